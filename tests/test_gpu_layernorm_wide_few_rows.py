"""The gradient of a few rows of more than 16384 columns, which one workgroup or a few take, and of
no rows at any width: against the float64 oracle, with every output wanted alone, in given buffers,
with a workspace of NaN, and again."""
import numpy as np
import pytest

from oracle import layernorm as ln
from tests.gpu_util import assert_within, note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    m.load()
    return m


def steps(dt):
    f = torch.finfo(dt)
    return f.eps / 2, f.smallest_normal * f.eps / 2      # the last: half the smallest subnormal


def host(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("cols", [16385, 20001, 24576, 32768])
@pytest.mark.parametrize("dt,pdt", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                    ("f32", "f32")])
def test_wide_rows(lib, rows, cols, dt, pdt):
    g = torch.Generator().manual_seed(rows * 11 + cols)
    wide = torch.randn(rows, cols + 5, generator=g).to(DT[dt]).cuda()
    x, dy = wide[:, 3:cols + 3], torch.randn(rows, cols, generator=g).to(DT[dt]).cuda()
    gamma = (1 + 0.3 * torch.randn(cols, generator=g)).to(DT[pdt]).cuda()
    note(f"layernorm_bwd wide rows {rows}x{cols} {dt}/{pdt}")
    _, mean, rstd = lib.fp8_layernorm_fwd(x, gamma)
    ws = torch.full((lib.fp8_layernorm_bwd_workspace(rows, cols) + 16,), 255, dtype=torch.uint8,
                    device="cuda")
    out = [torch.full(s, float("nan"), dtype=d, device="cuda")
           for s, d in (((rows, cols), DT[dt]), ((cols,), DT[pdt]), ((cols,), DT[pdt]))]
    got = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma, *out, workspace=ws)
    torch.cuda.synchronize()
    assert bool((ws[-16:] == 255).all())                          # nothing past what was asked
    args = (host(dy), host(x), host(mean), host(rstd), host(gamma))
    (half, tiny), (half_p, tiny_p) = steps(DT[dt]), steps(DT[pdt])
    for a, w, b, n in zip(got, ln.backward(*args),
                          ln.backward_bounds(*args, half, half_p, tiny, tiny_p),
                          ("dx", "dgamma", "dbeta")):
        assert_within(host(a), w, b, n)
    again = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    for keep in range(3):
        want = {n: i == keep for i, n in enumerate(("want_dx", "want_dgamma", "want_dbeta"))}
        one = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma, **want)[keep]
        torch.cuda.synchronize()
        assert torch.equal(one, got[keep]) and torch.equal(again[keep], got[keep])


@pytest.mark.parametrize("cols", [1, 7, 128, 129, 600, 1024, 2051, 16384, 16385, 32768])
@pytest.mark.parametrize("dt,pdt", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
def test_no_rows_give_zero_sums(lib, cols, dt, pdt):
    x = torch.empty((0, cols), dtype=DT[dt], device="cuda")
    stat = torch.empty(0, device="cuda")
    gamma = torch.ones(cols, dtype=DT[pdt], device="cuda")
    note(f"layernorm_bwd of no rows, cols={cols} {dt}/{pdt}")
    for dg, db in ((True, True), (True, False), (False, True)):
        flat = torch.full((2, cols + 2), 7.0, dtype=DT[pdt], device="cuda")
        a, b = (flat[i, 1:cols + 1] for i in range(2))
        dx, a2, b2 = lib.fp8_layernorm_bwd(x, x, stat, stat, gamma, want_dgamma=dg, want_dbeta=db,
                                           dgamma=a if dg else None, dbeta=b if db else None)
        torch.cuda.synchronize()
        assert dx.shape == (0, cols) and (a2 is a) == dg and (b2 is b) == db
        want = torch.full_like(flat, 7.0)
        want[0, 1:cols + 1] *= not dg
        want[1, 1:cols + 1] *= not db
        assert torch.equal(flat, want)
