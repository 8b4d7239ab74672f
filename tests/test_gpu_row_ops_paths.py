"""The paths that the row operators choose by size: waves to a row, rows that stream past the
caches or stay, the sort's steps, workgroups and scan, and the exchanges' pieces. Large tensors
are held against the same kernels on slices that take the other path (rows, columns and tokens
are independent, so those are equal bit for bit) and, for sums over the large dimension, against
64-bit sums with the oracle's bounds."""
import numpy as np
import pytest

from oracle import layernorm as ln
from oracle import moe
from tests.gpu_util import assert_within, note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24


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


# rows of 2 to 16 waves, whole and cut off, and of two pieces more a lane
@pytest.mark.parametrize("cols", [1032, 2056, 5120, 5121, 6143, 7168, 7169, 9215, 9216, 10241,
                                  11264, 13312, 15359, 15368, 16383, 17408, 20001])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_layernorm_row_waves(lib, cols, dt):
    g = torch.Generator().manual_seed(cols)
    rows = 19
    x = (torch.randn(rows, cols, generator=g) + 0.3).to(DT[dt]).cuda()
    dy = torch.randn(rows, cols, generator=g).to(DT[dt]).cuda()
    gamma = (1 + 0.2 * torch.randn(cols, generator=g)).cuda()
    beta = torch.randn(cols, generator=g).cuda()
    note(f"layernorm waves of a row cols={cols} {dt}")
    y, mean, rstd = lib.fp8_layernorm_fwd(x, gamma, beta)
    grads = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    torch.cuda.synchronize()
    hx, hg, hb, eps = host(x), host(gamma), host(beta), np.float64(np.float32(1e-5))
    for got, w, b, n in zip((y, mean, rstd), ln.forward(hx, hg, hb, eps),
                            ln.forward_bounds(hx, hg, hb, eps, half(DT[dt])), ("y", "mean", "rstd")):
        assert_within(host(got), w, b, n)
    args = (host(dy), hx, host(mean), host(rstd), hg)
    for got, w, b, n in zip(grads, ln.backward(*args),
                            ln.backward_bounds(*args, half(DT[dt]), U), ("dx", "dgamma", "dbeta")):
        assert_within(host(got), w, b, n)


@pytest.mark.parametrize("rows,cols,dt", [(4000, 4096, "bf16"), (7001, 2051, "f16"),
                                          (3000, 17000, "f16"), (13000, 4100, "bf16"),
                                          (2100, 12290, "f32")])
def test_layernorm_of_large_tensors(lib, rows, cols, dt):
    """Tensors of 28 to 106 MB: their rows stream, those of the slices are kept."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, cols, generator=g, device="cuda").to(DT[dt])
    dy = torch.randn(rows, cols, generator=g, device="cuda").to(DT[dt])
    gamma = torch.randn(cols, generator=g, device="cuda")
    beta = torch.randn(cols, generator=g, device="cuda")
    note(f"layernorm of a large tensor {rows}x{cols} {dt}")
    y, mean, rstd = lib.fp8_layernorm_fwd(x, gamma, beta)
    dx, dgamma, dbeta = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    for a in (0, rows // 2, rows - 37):
        s = slice(a, a + 37)
        y2, m2, r2 = lib.fp8_layernorm_fwd(x[s], gamma, beta)
        dx2, _, _ = lib.fp8_layernorm_bwd(dy[s], x[s], m2, r2, gamma)
        torch.cuda.synchronize()
        assert torch.equal(y[s], y2) and torch.equal(mean[s], m2) and torch.equal(rstd[s], r2)
        assert torch.equal(dx[s], dx2)
    chain = ln.col_chain(rows)
    for c in range(0, cols, 1024):
        cs = slice(c, min(c + 1024, cols))
        d = dy[:, cs].double()
        xh = (x[:, cs].double() - mean[:, None].double()) * rstd[:, None].double()
        for got, terms in ((dgamma, d * xh), (dbeta, d)):
            want, mag = terms.sum(0), terms.abs().sum(0)
            tol = (chain + 3) * U * mag + U * want.abs() + 1e-30
            assert bool(((got[cs].double() - want).abs() <= tol).all())


def routing(seed, tokens, topk, experts):
    rng = np.random.default_rng(seed)
    idx = rng.integers(-1, experts, size=(tokens, topk))
    idx[rng.random((tokens, topk)) < 0.3] = experts // 2          # one expert is liked
    return idx


# one step, four steps, counted chunks, and the scan, at and around their borders
@pytest.mark.parametrize("pairs", [1023, 1024, 1025, 4095, 4096, 4097, 131071, 131072, 131073,
                                   140000])
@pytest.mark.parametrize("experts,multiple", [(1, 16), (2, 1), (64, 16), (65, 16), (512, 16),
                                              (7, 100)])
def test_sort_borders(lib, pairs, experts, multiple):
    idx = routing(pairs + experts, pairs, 1, experts)
    t = torch.from_numpy(idx).cuda()
    rows = lib.fp8_moe_rows(pairs, 1, experts, multiple)
    note(f"moe_sort pairs={pairs} experts={experts} multiple={multiple}")
    ws = torch.full((lib.fp8_moe_sort_workspace(pairs, 1, experts) + 4,), 255, dtype=torch.uint8,
                    device="cuda")
    bufs = [torch.full(s, -99, dtype=torch.int32, device="cuda")
            for s in ((pairs, 1), (rows,), (experts,), (experts + 1,))]
    got = lib.fp8_moe_sort(t, experts, multiple, *bufs, workspace=ws)
    torch.cuda.synchronize()
    for g, w, n in zip(got, moe.sort(idx, experts, multiple, rows),
                       ("slot", "source", "counts", "offsets")):
        assert np.array_equal(g.cpu().numpy(), w), n
    assert bool((ws[-4:] == 255).all())                           # nothing past what was asked


@pytest.mark.parametrize("tokens,topk,cols,dt", [(9000, 2, 4100, "bf16"), (6000, 5, 2052, "f16"),
                                                 (3000, 9, 1300, "f32"), (20000, 3, 130, "bf16")])
def test_exchanges_of_large_tensors(lib, tokens, topk, cols, dt):
    """Buffers above 96 MiB stream; slices of columns are kept, and are equal bit for bit. The
    router's gradient sums over the columns: a 64-bit sum with the oracle's bound."""
    experts = 24
    slot, source, _, _ = lib.fp8_moe_sort(torch.from_numpy(routing(9, tokens, topk, experts)).cuda(),
                                          experts)
    rows = source.numel()
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x = torch.randn(tokens, cols, generator=g, device="cuda").to(DT[dt])
    ys = torch.randn(rows, cols, generator=g, device="cuda").to(DT[dt])
    w = torch.rand(tokens, topk, generator=g, device="cuda")
    note(f"moe exchanges of large tensors tokens={tokens} topk={topk} cols={cols} {dt}")
    xs = lib.fp8_moe_dispatch(x, slot, source)
    y, dx = lib.fp8_moe_combine(ys, slot, w), lib.fp8_moe_dispatch_bwd(ys, slot)
    dys, dw = lib.fp8_moe_combine_bwd(x, ys, slot, source, w)
    live = source >= 0
    assert torch.equal(xs[live], x[(source[live] // topk).long()]) and not xs[~live].any()
    for a, b in ((0, 17), (cols // 2, cols // 2 + 64), (cols - 33, cols)):
        s = slice(a, b)
        y2, dx2 = lib.fp8_moe_combine(ys[:, s], slot, w), lib.fp8_moe_dispatch_bwd(ys[:, s], slot)
        dys2, _ = lib.fp8_moe_combine_bwd(x[:, s], ys[:, s], slot, source, w)
        torch.cuda.synchronize()
        assert torch.equal(y[:, s], y2) and torch.equal(dx[:, s], dx2)
        assert torch.equal(dys[:, s], dys2)
    for j in range(topk):
        kept = slot[:, j] >= 0
        want, mag = torch.zeros(tokens, dtype=torch.float64, device="cuda"), None
        prod = x[kept].double() * ys[slot[kept, j].long()].double()
        want[kept] = prod.sum(1)
        mag = torch.zeros_like(want)
        mag[kept] = prod.abs().sum(1)
        tol = (8 * np.ceil(cols / 256) + 24) * U * mag + 1e-30
        assert bool(((dw[:, j].double() - want).abs() <= tol).all())


@pytest.mark.parametrize("tokens,topk,cols,dt,skip", [(2500, 3, 2049, "bf16", 1),
                                                      (2500, 4, 2080, "f16", 7),
                                                      (1500, 3, 1999, "f32", 5),
                                                      (300, 3, 77, "bf16", 3)])
def test_dispatch_into_a_cut_of_a_buffer(lib, tokens, topk, cols, dt, skip):
    """An output that starts anywhere in a line, its rows ending anywhere: every element of it is
    written, and nothing beside it."""
    experts = 11
    slot, source, _, _ = lib.fp8_moe_sort(torch.from_numpy(routing(5, tokens, topk, experts)).cuda(),
                                          experts)
    rows = source.numel()
    x = torch.randn(tokens, cols + 3, device="cuda").to(DT[dt])[:, 2:cols + 2]
    flat = torch.full((rows * cols + 200,), 7.0, dtype=DT[dt], device="cuda")
    xs = flat[skip:skip + rows * cols].view(rows, cols)
    note(f"moe_dispatch into a cut, tokens={tokens} cols={cols} {dt} skip={skip}")
    lib.fp8_moe_dispatch(x, slot, source, xs=xs)
    torch.cuda.synchronize()
    live = source >= 0
    assert torch.equal(xs[live], x[(source[live] // topk).long()]) and not xs[~live].any()
    assert bool((flat[:skip] == 7).all()) and bool((flat[skip + rows * cols:] == 7).all())
