"""GPU parity of layer norm and its gradient against the float64 oracle: every lane layout
and its borders, the types of rows and parameters, strides, ragged widths, single rows and
none, special values, streams, and replays of a captured graph. The tolerances are the
oracle's bounds of a float32 computation plus half a step of the stored type."""
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


def half(dt):
    return torch.finfo(dt).eps / 2


def host(t):
    return t.detach().cpu().double().numpy()


def draw(seed, rows, cols, dt, pdt, pad=0, offset=0.3):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols + pad, generator=g) + offset).to(dt)
    dy = (0.1 * torch.randn(rows, cols + pad, generator=g)).to(dt)
    gamma = (1 + 0.2 * torch.randn(cols, generator=g)).to(pdt)
    beta = (0.3 * torch.randn(cols, generator=g)).to(pdt)
    return [t.cuda() for t in (x, dy)] + [gamma.cuda(), beta.cuda()]


def check_forward(lib, x, gamma, beta, eps=1e-5, **kw):
    y, mean, rstd = lib.fp8_layernorm_fwd(x, gamma, beta, eps=eps, **kw)
    torch.cuda.synchronize()
    hx, hg, hb = host(x), None if gamma is None else host(gamma), None if beta is None else host(beta)
    want = ln.forward(hx, hg, hb, np.float64(np.float32(eps)))
    bounds = ln.forward_bounds(hx, hg, hb, np.float64(np.float32(eps)), half(x.dtype))
    for got, w, b, n in zip((y, mean, rstd), want, bounds, ("y", "mean", "rstd")):
        assert_within(host(got), w, b, n)
    return y, mean, rstd


def check_backward(lib, dy, x, mean, rstd, gamma, pdt, **kw):
    dx, dgamma, dbeta = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma, **kw)
    torch.cuda.synchronize()
    args = (host(dy), host(x), host(mean), host(rstd), None if gamma is None else host(gamma))
    want = ln.backward(*args)
    bounds = ln.backward_bounds(*args, half(x.dtype), half(pdt))
    for got, w, b, n in zip((dx, dgamma, dbeta), want, bounds, ("dx", "dgamma", "dbeta")):
        assert_within(host(got), w, b, n)
    return dx, dgamma, dbeta


# widths at and around the borders of the lane layouts, and odd ones
COLS = [1, 2, 7, 8, 9, 63, 127, 128, 129, 511, 512, 513, 1000, 1024, 1025, 2047, 2048, 2049, 4095,
        4096, 4097, 5003, 8192, 8193, 16384, 16385, 32767, 32768]


@pytest.mark.parametrize("cols", COLS)
def test_widths(lib, cols):
    for dt in ("bf16", "f32"):
        rows = 37 if cols <= 4097 else 5
        x, dy, gamma, beta = draw(cols, rows, cols, DT[dt], torch.float32)
        note(f"layernorm rows={rows} cols={cols} {dt}")
        _, mean, rstd = check_forward(lib, x, gamma, beta)
        check_backward(lib, dy, x, mean, rstd, gamma, torch.float32)


@pytest.mark.parametrize("dt,pdt", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"),
                                    ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("rows,cols,pad", [(1, 128, 0), (3, 77, 0), (64, 128, 0), (130, 500, 12),
                                           (517, 1027, 5), (1030, 96, 0), (2100, 640, 0),
                                           (600, 3000, 1)])
def test_types_rows_and_strides(lib, dt, pdt, rows, cols, pad):
    x, dy, gamma, beta = draw(rows + cols, rows, cols, DT[dt], DT[pdt], pad)
    x, dy = x[:, :cols], dy[:, pad:]               # a cut: odd strides, odd starts
    note(f"layernorm rows={rows} cols={cols} pad={pad} {dt}/{pdt}")
    _, mean, rstd = check_forward(lib, x, gamma, beta)
    check_backward(lib, dy, x, mean, rstd, gamma, DT[pdt])


def test_many_rows(lib):
    """More rows than the grids take at once, in every layout's kind."""
    for rows, cols in ((20011, 64), (9001, 520), (3001, 2056), (1501, 6000)):
        x, dy, gamma, beta = draw(rows, rows, cols, torch.bfloat16, torch.bfloat16)
        note(f"layernorm rows={rows} cols={cols}")
        _, mean, rstd = check_forward(lib, x, gamma, beta)
        check_backward(lib, dy, x, mean, rstd, gamma, torch.bfloat16)


def test_without_parameters_and_outputs(lib):
    x, dy, gamma, beta = draw(5, 33, 300, torch.bfloat16, torch.bfloat16)
    note("layernorm without gamma, beta, statistics or some gradients")
    _, mean, rstd = check_forward(lib, x, None, None)
    check_forward(lib, x, gamma, None)
    check_forward(lib, x, None, beta)
    y, m0, r0 = lib.fp8_layernorm_fwd(x, gamma, beta, want_stats=False)
    assert m0 is None and r0 is None
    assert torch.equal(y, lib.fp8_layernorm_fwd(x, gamma, beta)[0])
    full = check_backward(lib, dy, x, mean, rstd, gamma, torch.bfloat16)
    check_backward(lib, dy, x, mean, rstd, None, torch.float32, param_dtype=torch.float32)
    for keep in range(3):
        want = {n: i == keep for i, n in enumerate(("want_dx", "want_dgamma", "want_dbeta"))}
        got = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma, **want)
        assert [g is not None for g in got] == [i == keep for i in range(3)]
        assert torch.equal(got[keep], full[keep])


def test_no_rows(lib):
    x = torch.empty((0, 40), dtype=torch.bfloat16, device="cuda")
    g = torch.ones(40, device="cuda")
    y, mean, rstd = lib.fp8_layernorm_fwd(x, g, g)
    assert y.shape == (0, 40) and mean.numel() == 0
    dg, db = torch.full((40,), 7.0, device="cuda"), torch.full((40,), 7.0, device="cuda")
    dx, _, _ = lib.fp8_layernorm_bwd(x, x, mean, rstd, g, dgamma=dg, dbeta=db)
    torch.cuda.synchronize()
    assert dx.shape == (0, 40) and not dg.any() and not db.any()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_special_values(lib, dt):
    """A constant row gives beta (its variance is 0), a far offset keeps its variance, and a
    NaN or an infinity stays in its row."""
    cols = 264
    x, dy, gamma, beta = draw(9, 8, cols, DT[dt], torch.float32)
    x[1] = 3.0
    x[2] += 64.0
    note(f"layernorm special rows {dt}")
    y, mean, rstd = check_forward(lib, x, gamma, beta)
    assert torch.equal(y[1], beta.to(DT[dt]))
    clean = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)[0].clone()
    x[4, 5] = float("nan")
    x[6, 263] = float("inf")
    y2, m2, r2 = lib.fp8_layernorm_fwd(x, gamma, beta)
    dx2, dg2, db2 = lib.fp8_layernorm_bwd(dy, x, m2, r2, gamma)
    torch.cuda.synchronize()
    for r in range(8):
        if r in (4, 6):
            assert torch.isnan(y2[r]).all() and torch.isnan(dx2[r]).all()
        else:
            assert torch.equal(y2[r], y[r]) and torch.equal(dx2[r], clean[r])
    assert torch.isnan(dg2).all() and torch.isfinite(db2).all()


def test_f16_overflow_rounds_to_infinity(lib):
    x, _, _, beta = draw(11, 4, 64, torch.float16, torch.float32)
    gamma = torch.full((64,), 1e6, device="cuda")
    y, mean, rstd = lib.fp8_layernorm_fwd(x, gamma, beta)
    torch.cuda.synchronize()
    want = torch.from_numpy(ln.forward(host(x), host(gamma), host(beta), 1e-5)[0]).to(torch.float16)
    big = want.isinf()
    assert big.any() and torch.equal(y.cpu()[big], want[big])


def test_gradient_against_differences(lib):
    """Directional central differences of the float64 forward, against the kernel's gradient:
    off by the truncation (h^2 times the third derivative, below 1e-6 of the scale here) and
    the kernel's own bound."""
    rows, cols, eps = 6, 96, 1e-5
    x, dy, gamma, beta = draw(21, rows, cols, torch.float32, torch.float32)
    _, mean, rstd = lib.fp8_layernorm_fwd(x, gamma, beta, eps=eps)
    dx, dgamma, dbeta = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    torch.cuda.synchronize()
    hx, hd, hg, hb = host(x), host(dy), host(gamma), host(beta)
    rng = np.random.default_rng(3)
    e = np.float64(np.float32(eps))
    bounds = ln.backward_bounds(hd, hx, host(mean), host(rstd), hg, half(torch.float32),
                                half(torch.float32))
    # the kernel's gradient uses float32 statistics: relative changes of 1e-6 of mean and rstd
    stat = 4e-6
    h = 1e-4

    def loss(a, b, c):
        return (hd * ln.forward(a, b, c, e)[0]).sum()

    for _ in range(4):
        for name, grad, bound, args in (
                ("dx", dx, bounds[0], lambda s, v: (hx + s * v, hg, hb)),
                ("dgamma", dgamma, bounds[1], lambda s, v: (hx, hg + s * v, hb)),
                ("dbeta", dbeta, bounds[2], lambda s, v: (hx, hg, hb + s * v))):
            g = host(grad)
            v = rng.standard_normal(g.shape)
            diff = (loss(*args(h, v)) - loss(*args(-h, v))) / (2 * h)
            tol = (np.abs(v) * bound).sum() + (stat + 1e-5) * (np.abs(v) * np.abs(g)).sum() + 1e-7
            assert abs((g * v).sum() - diff) <= tol, (name, (g * v).sum(), diff, tol)


def test_repeats_and_given_buffers(lib):
    x, dy, gamma, beta = draw(31, 700, 1500, torch.bfloat16, torch.float32)
    y, mean, rstd = lib.fp8_layernorm_fwd(x, gamma, beta)
    first = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    ws = torch.empty(lib.fp8_layernorm_bwd_workspace(700, 1500), dtype=torch.uint8, device="cuda")
    assert ws.numel() > 0
    ws.fill_(255)                                    # NaN patterns: nothing stale is read
    out = [torch.full_like(t, float("nan")) for t in first]
    again = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma, *out, workspace=ws)
    torch.cuda.synchronize()
    for a, b, o in zip(first, again, out):
        assert b is o and torch.equal(a, b)
    with pytest.raises(ValueError, match="workspace"):
        lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma, workspace=ws[:-1])


def test_other_stream(lib):
    """A call on a stream of its own takes its buffers from that stream's pool."""
    x, dy, gamma, beta = draw(41, 900, 1100, torch.bfloat16, torch.float32)
    y0, mean, rstd = lib.fp8_layernorm_fwd(x, gamma, beta)
    ref = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(4):
        y, m, r = lib.fp8_layernorm_fwd(x, gamma, beta, stream=s)
        got.append((y, lib.fp8_layernorm_bwd(dy, x, m, r, gamma, stream=s)))
        torch.full((900, 1100), 3.0, device="cuda")          # other work on the current stream
    torch.cuda.synchronize()
    for y, grads in got:
        assert torch.equal(y, y0)
        assert all(torch.equal(a, b) for a, b in zip(grads, ref))


def test_graph_replays(lib):
    x, dy, gamma, beta = draw(51, 260, 1030, torch.bfloat16, torch.float32)
    y, mean, rstd = lib.fp8_layernorm_fwd(x, gamma, beta)
    grads = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    ws = torch.empty(lib.fp8_layernorm_bwd_workspace(260, 1030), dtype=torch.uint8, device="cuda")

    def step():
        lib.fp8_layernorm_fwd(x, gamma, beta, y=y, mean=mean, rstd=rstd)
        lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma, *grads, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(4):
        new = draw(60 + k, 260, 1030, torch.bfloat16, torch.float32)
        x.copy_(new[0])
        dy.copy_(new[1])
        y0, m0, r0 = lib.fp8_layernorm_fwd(x, gamma, beta)
        want = lib.fp8_layernorm_bwd(dy, x, m0, r0, gamma)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, y0)
        assert all(torch.equal(a, b) for a, b in zip(grads, want)), k
