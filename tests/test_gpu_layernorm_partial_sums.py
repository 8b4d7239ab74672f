"""Layer norm's gradient by partial sums, the form of more rows than go by columns: a workspace that
held NaN, replays of a captured graph, a stream of its own, and NaN and infinities that stay where
they belong, also with row groups that have no row in the last turn. Each test first asserts that
its size takes this form, by the workspace that the call leaves written."""
import numpy as np
import pytest

from oracle import layernorm as ln
from tests.gpu_util import assert_within, note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NAN, INF = float("nan"), float("inf")

# a row in 16 lanes, in a wave of 8 and of 16 elements a lane, in two waves and more, in 32 elements
# a lane; rows that fill their last turn's groups and rows that do not; whole and cut-off widths
SIZES = [(2001, 100, "bf16"), (2048, 128, "f16"), (2501, 300, "bf16"), (2100, 640, "f16"),
         (1301, 701, "f32"), (3001, 1500, "bf16"), (1501, 1030, "f32"), (2050, 2048, "f32"),
         (2003, 5003, "f32"), (7, 20000, "bf16"), (6, 17001, "f32"), (5003, 4096, "bf16")]


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    m.load()
    return m


def host(t):
    return t.detach().cpu().double().numpy()


def inputs(lib, rows, cols, dt, seed=0):
    g = torch.Generator().manual_seed(rows + cols + seed)
    x, dy = ((torch.randn(rows, cols, generator=g) + 0.3).to(DT[dt]).cuda() for _ in range(2))
    gamma = (1 + 0.3 * torch.randn(cols, generator=g)).cuda()
    _, mean, rstd = lib.fp8_layernorm_fwd(x, gamma)
    return dy, x, mean, rstd, gamma


def with_workspace(lib, args):
    """The gradient in a workspace of NaN patterns; asserts that all of it was written (so this is
    the form of partial sums) and nothing past it."""
    need = lib.fp8_layernorm_bwd_workspace(*args[1].shape)
    ws = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")
    out = lib.fp8_layernorm_bwd(*args, workspace=ws)
    torch.cuda.synchronize()
    assert need > 0 and bool((ws[:need].view(torch.int32) != -1).all())
    assert bool((ws[need:] == 255).all())
    return out


@pytest.mark.parametrize("rows,cols,dt", SIZES)
def test_stale_workspace(lib, rows, cols, dt):
    args = inputs(lib, rows, cols, dt)
    note(f"layernorm_bwd by partial sums {rows}x{cols} {dt}")
    got = with_workspace(lib, args)
    h = tuple(host(t) for t in args)
    f = torch.finfo(DT[dt])
    half, tiny = f.eps / 2, f.smallest_normal * f.eps / 2
    for a, w, b, n in zip(got, ln.backward(*h), ln.backward_bounds(*h, half, 2.0 ** -24, tiny),
                          ("dx", "dgamma", "dbeta")):
        assert_within(host(a), w, b, n)
    plain = lib.fp8_layernorm_bwd(*args)
    for keep in range(3):
        want = {n: i == keep for i, n in enumerate(("want_dx", "want_dgamma", "want_dbeta"))}
        one = lib.fp8_layernorm_bwd(*args, **want)[keep]
        torch.cuda.synchronize()
        assert torch.equal(one, got[keep]) and torch.equal(plain[keep], got[keep])


@pytest.mark.parametrize("rows,cols,dt", SIZES)
def test_nan_and_infinity_stay_in_their_place(lib, rows, cols, dt):
    """One of dy spoils its row of dx and its column of the sums; one of x spoils its row of dx and,
    through the row's mean, all of dgamma. The last row is the one that idle groups work on."""
    dy, x, mean, rstd, gamma = inputs(lib, rows, cols, dt)
    clean = with_workspace(lib, (dy, x, mean, rstd, gamma))
    note(f"layernorm_bwd by partial sums with NaN {rows}x{cols} {dt}")
    for r, c, v in ((rows - 1, cols - 1, NAN), (rows // 2, 0, INF), (0, cols // 2, -INF)):
        d = dy.clone()
        d[r, c] = v
        dx, dgamma, dbeta = with_workspace(lib, (d, x, mean, rstd, gamma))
        rest = torch.arange(rows, device="cuda") != r
        assert torch.equal(dx[rest], clean[0][rest]) and not torch.isfinite(dx[r]).any()
        cols_rest = torch.arange(cols, device="cuda") != c
        for a, b in ((dgamma, clean[1]), (dbeta, clean[2])):
            assert torch.equal(a[cols_rest], b[cols_rest]) and not torch.isfinite(a[c])
        bad = x.clone()
        bad[r, c] = v
        _, m2, r2 = lib.fp8_layernorm_fwd(bad, gamma)
        dx, dgamma, dbeta = with_workspace(lib, (dy, bad, m2, r2, gamma))
        assert torch.equal(dx[rest], clean[0][rest]) and torch.isnan(dx[r]).all()
        assert torch.isnan(dgamma).all() and torch.equal(dbeta, clean[2])


@pytest.mark.parametrize("rows,cols,dt", [(3001, 1500, "bf16"), (1501, 1030, "f32"),
                                          (2001, 100, "bf16"), (6, 17001, "f32")])
def test_other_stream(lib, rows, cols, dt):
    """On a stream of its own the call takes workspace and outputs from that stream's pool."""
    args = inputs(lib, rows, cols, dt)
    want = with_workspace(lib, args)
    s = torch.cuda.Stream()
    note(f"layernorm_bwd by partial sums on another stream {rows}x{cols} {dt}")
    got = []
    for _ in range(4):
        got.append(lib.fp8_layernorm_bwd(*args, stream=s))
        torch.full((rows, cols), 3.0, device="cuda")          # other work on the current stream
        torch.full((1 << 20,), NAN, device="cuda")
    torch.cuda.synchronize()
    for grads in got:
        assert all(torch.equal(a, b) for a, b in zip(grads, want))


@pytest.mark.parametrize("rows,cols,dt", [(3001, 1500, "bf16"), (1501, 1030, "f32"),
                                          (2100, 640, "f16"), (7, 20000, "bf16")])
def test_graph_replays(lib, rows, cols, dt):
    dy, x, mean, rstd, gamma = inputs(lib, rows, cols, dt)
    with_workspace(lib, (dy, x, mean, rstd, gamma))
    grads = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    ws = torch.empty(lib.fp8_layernorm_bwd_workspace(rows, cols), dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    note(f"layernorm_bwd by partial sums, graph replays {rows}x{cols} {dt}")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.fp8_layernorm_fwd(x, gamma, y=y, mean=mean, rstd=rstd)
        lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma, *grads, workspace=ws)
    for k in range(4):
        new = inputs(lib, rows, cols, dt, seed=100 + k)
        dy.copy_(new[0])
        x.copy_(new[1])
        y0, m0, r0 = lib.fp8_layernorm_fwd(x, gamma)
        want = lib.fp8_layernorm_bwd(dy, x, m0, r0, gamma)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0) and torch.equal(mean, m0) and torch.equal(rstd, r0)
        assert all(torch.equal(a, b) for a, b in zip(grads, want)), k
