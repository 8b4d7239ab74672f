"""GPU parity of the expert exchange: the sort against a pair-by-pair oracle (all integers
equal), dispatch and the gradient of the experts' outputs bit for bit, combine, dispatch's
gradient and the router's gradient within the oracle's float32 bounds."""
import numpy as np
import pytest

from oracle import moe
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


def route(seed, tokens, topk, experts, drop, kind="any"):
    rng = np.random.default_rng(seed)
    if kind == "one":                                # every pair to the last expert
        idx = np.full((tokens, topk), experts - 1)
    elif kind == "none":                             # every pair dropped, in several ways
        idx = rng.choice([-1, -7, experts, experts + 100, -2 ** 31], size=(tokens, topk))
    else:                                            # skewed, some experts empty
        p = rng.random(experts) ** 3
        p[rng.random(experts) < 0.2] = 0
        p = p / p.sum() if p.sum() > 0 else np.full(experts, 1 / experts)
        idx = rng.choice(experts, size=(tokens, topk), p=p)
        idx[rng.random((tokens, topk)) < drop] = -1
        if tokens > 2:
            idx[1] = -1                              # a token that kept nothing
    return idx


def check_sort(lib, idx, experts, multiple, dtype=torch.int64):
    tokens, topk = idx.shape
    t = torch.from_numpy(np.ascontiguousarray(idx)).to(dtype).cuda()
    rows = lib.fp8_moe_rows(tokens, topk, experts, multiple)
    bufs = [torch.full(s, -99, dtype=torch.int32, device="cuda")
            for s in ((tokens, topk), (rows,), (experts,), (experts + 1,))]
    got = lib.fp8_moe_sort(t, experts, multiple, *bufs)
    torch.cuda.synchronize()
    want = moe.sort(idx, experts, multiple, rows)
    for g, w, n in zip(got, want, ("slot", "source", "counts", "offsets")):
        assert np.array_equal(g.cpu().numpy(), w), n
    return got


SORT = [(0, 1, 1, 16), (0, 3, 8, 16), (1, 1, 1, 1), (1, 2, 8, 16), (3, 64, 5, 16), (64, 2, 8, 16),
        (333, 4, 16, 16), (1000, 1, 512, 16), (77, 7, 511, 3), (2048, 8, 64, 16),
        (2049, 8, 64, 128), (5000, 5, 3, 1), (20000, 6, 129, 16)]


@pytest.mark.parametrize("tokens,topk,experts,multiple", SORT)
def test_sort(lib, tokens, topk, experts, multiple):
    for kind in ("any", "one", "none"):
        idx = route(tokens + topk, tokens, topk, experts, 0.1, kind)
        note(f"moe_sort tokens={tokens} topk={topk} experts={experts} multiple={multiple} {kind}")
        check_sort(lib, idx, experts, multiple)
        check_sort(lib, idx, experts, multiple, torch.int32)


def test_sort_long(lib):
    """More pairs than the workgroups take one chunk each of: 4.3 million."""
    tokens, topk, experts = 2_150_000, 2, 6
    idx = route(5, tokens, topk, experts, 0.05)
    note("moe_sort of 4.3 million pairs")
    check_sort(lib, idx, experts, 16, torch.int32)


def test_sort_index_beyond_32_bits(lib):
    idx = np.array([[2 ** 32 + 1, 1], [-2 ** 40, 0], [2 ** 62, 2]])
    check_sort(lib, idx, 3, 16)


def setup(lib, seed, tokens, topk, experts, cols, dt, drop=0.1, pad=0, multiple=16, kind="any"):
    idx = route(seed, tokens, topk, experts, drop, kind)
    slot, source, counts, offsets = check_sort(lib, idx, experts, multiple)
    g = torch.Generator().manual_seed(seed)
    rows = source.numel()
    x = torch.randn(tokens, cols + pad, generator=g).to(dt)[:, :cols].cuda() if not pad else \
        torch.randn(tokens, cols + pad, generator=g).to(dt).cuda()[:, pad:]
    ys = torch.randn(rows, cols + pad, generator=g).to(dt).cuda()[:, :cols]
    # what the experts left in the padding rows must not matter
    ys[source < 0] = float("nan")
    w = torch.rand(tokens, topk, generator=g).cuda()
    w[slot < 0] = float("nan")                       # nor a dropped pair's weight
    return x, ys, w, slot, source


SHAPES = [(1, 2, 8, 4096, 0), (1, 1, 1, 1, 0), (5, 3, 4, 7, 0), (64, 2, 8, 128, 0),
          (77, 3, 10, 1027, 3), (100, 8, 64, 513, 0), (130, 9, 12, 2049, 5), (40, 4, 16, 8192, 0),
          (33, 64, 70, 130, 1), (300, 1, 6, 2048, 8), (17, 2, 4, 20001, 0), (600, 6, 32, 24, 0)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,topk,experts,cols,pad", SHAPES)
def test_exchanges(lib, tokens, topk, experts, cols, pad, dt):
    note(f"moe exchanges tokens={tokens} topk={topk} experts={experts} cols={cols} pad={pad} {dt}")
    x, ys, w, slot, source = setup(lib, tokens + cols, tokens, topk, experts, cols, DT[dt], pad=pad)
    rows, hs = source.numel(), slot.cpu().numpy()
    nan = float("nan")
    xs = lib.fp8_moe_dispatch(x, slot, source,
                              xs=torch.full((rows, cols), nan, dtype=DT[dt], device="cuda"))
    y = lib.fp8_moe_combine(ys, slot, w)
    dx = lib.fp8_moe_dispatch_bwd(ys, slot)
    dys, dw = lib.fp8_moe_combine_bwd(
        x, ys, slot, source, w, dys=torch.full((rows, cols), nan, dtype=DT[dt], device="cuda"))
    torch.cuda.synchronize()
    assert np.array_equal(host(xs), moe.dispatch(host(x), hs, rows))
    for got, weights, n in ((y, host(w), "y"), (dx, None, "dx")):
        want, bound = moe.combine(host(ys), hs, weights)
        assert_within(host(got), want,
                      bound * (1 + 2 * half(DT[dt])) + half(DT[dt]) * np.abs(want) + 1e-7 * (dt == "f16"),
                      n)
        assert np.all(host(got)[(hs < 0).all(1)] == 0)
    _, wdw, bound = moe.combine_bwd(host(x), host(ys), hs, host(w), rows)
    assert_within(host(dw), wdw, bound, "dw")
    # one float32 product, one rounding: the same bits
    live = source.cpu() >= 0
    src = source.cpu()[live].long()
    want = torch.zeros((rows, cols), dtype=DT[dt])
    want[live] = (w.cpu().reshape(-1)[src][:, None] * x.cpu().float()[src // topk]).to(DT[dt])
    assert torch.equal(dys.cpu(), want)


@pytest.mark.parametrize("kind", ["one", "none"])
def test_all_to_one_and_all_dropped(lib, kind):
    x, ys, w, slot, source = setup(lib, 3, 50, 2, 7, 200, torch.bfloat16, kind=kind)
    hs = slot.cpu().numpy()
    xs = lib.fp8_moe_dispatch(x, slot, source)
    y = lib.fp8_moe_combine(ys, slot, w)
    dys, dw = lib.fp8_moe_combine_bwd(x, ys, slot, source, w)
    torch.cuda.synchronize()
    assert np.array_equal(host(xs), moe.dispatch(host(x), hs, source.numel()))
    if kind == "none":
        assert not xs.any() and not y.any() and not dys.any() and not dw.any()


def test_wrong_slots_are_skipped(lib):
    """Entries of slot outside the sorted buffer are never used as addresses."""
    x, ys, w, slot, source = setup(lib, 4, 20, 2, 4, 96, torch.float32, drop=0.0)
    ys = torch.nan_to_num(ys)
    rows = source.numel()
    bad = slot.clone()
    bad[3, 0], bad[4, 1], bad[5, 0] = rows, 2 ** 31 - 1, -2 ** 31
    ref = bad.clone()
    ref[3, 0] = ref[4, 1] = ref[5, 0] = -1
    w = torch.rand_like(w)
    note("moe exchanges with slots outside the buffer")
    for f in (lambda s: lib.fp8_moe_combine(ys, s, w), lambda s: lib.fp8_moe_dispatch_bwd(ys, s),
              lambda s: lib.fp8_moe_combine_bwd(x, ys, s, source, w)[1]):
        a, b = f(bad), f(ref)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
    xs = torch.full((rows, 96), 5.0, device="cuda")
    lib.fp8_moe_dispatch(x, bad, source, xs=xs)
    torch.cuda.synchronize()
    assert torch.equal(xs[slot[0, 0].item()], x[0]) and bool((xs[slot[3, 0].item()] == 5.0).all())


def test_infinite_rows_stay_with_their_tokens(lib):
    x, ys, w, slot, source = setup(lib, 6, 40, 2, 4, 72, torch.bfloat16, drop=0.0)
    ys = torch.nan_to_num(ys)
    w = torch.rand_like(w)
    clean = lib.fp8_moe_combine(ys, slot, w)
    r = int(slot[7, 1])
    ys[r, 3] = float("inf")
    y = lib.fp8_moe_combine(ys, slot, w)
    torch.cuda.synchronize()
    assert torch.isinf(y[7, 3]) and int((y != clean).sum()) == 1


def test_offsets_past_32_bits(lib):
    """Sorted and token buffers of more than 2^32 bytes, and of more than 2^31 elements."""
    tokens, cols, experts = 140_000, 16_384, 3
    idx = route(8, tokens, 1, experts, 0.0)
    slot, source, _, _ = check_sort(lib, idx, experts, 16, torch.int32)
    x = torch.empty((tokens, cols), dtype=torch.bfloat16, device="cuda")
    x.copy_(torch.arange(tokens, device="cuda")[:, None] % 251)
    note("moe exchanges over 4.6 GB")
    xs = lib.fp8_moe_dispatch(x, slot, source)
    back = lib.fp8_moe_dispatch_bwd(xs, slot)
    torch.cuda.synchronize()
    kept = slot[:, 0] >= 0
    assert torch.equal(back[kept], x[kept]) and not back[~kept].any()
    live = source >= 0
    assert torch.equal(xs[live][:, ::4099], x[source[live].long()][:, ::4099])
    assert not xs[~live].any()


def test_gradients_against_differences(lib):
    """combine is linear in ys and in w, dispatch in x: central differences of the float64
    forms are exact but for rounding, so they meet the kernels' bounds."""
    tokens, topk, cols = 12, 3, 40
    x, ys, w, slot, source = setup(lib, 10, tokens, topk, 5, cols, torch.float32)
    ys, w = torch.nan_to_num(ys), torch.nan_to_num(w)
    hs, rows = slot.cpu().numpy(), source.numel()
    dys, dw = lib.fp8_moe_combine_bwd(x, ys, slot, source, w)
    dx = lib.fp8_moe_dispatch_bwd(ys, slot)
    torch.cuda.synchronize()
    hx, hy, hw = host(x), host(ys), host(w)
    rng = np.random.default_rng(1)
    _, _, b_dw = moe.combine_bwd(hx, hy, hs, hw, rows)
    _, b_dx = moe.combine(hy, hs, None)
    for _ in range(4):
        for g, b, loss, at in (
                (host(dys), 2 * moe.U * np.abs(host(dys)),
                 lambda v: (hx * moe.combine(v, hs, hw)[0]).sum(), hy),
                (host(dw), b_dw, lambda v: (hx * moe.combine(hy, hs, v)[0]).sum(), hw),
                (host(dx), b_dx + moe.U * np.abs(host(dx)),
                 lambda v: (hy * moe.dispatch(v, hs, rows)).sum(), hx)):
            v = rng.standard_normal(at.shape)
            diff = (loss(at + v) - loss(at - v)) / 2
            tol = (np.abs(v) * b).sum() + 1e-11 * (np.abs(v) * np.abs(g)).sum() + 1e-11
            assert abs((g * v).sum() - diff) <= tol


def test_other_stream_and_graph_replays(lib):
    tokens, topk, experts, cols = 3000, 6, 24, 264
    x, ys, w, slot, source = setup(lib, 12, tokens, topk, experts, cols, torch.bfloat16)
    ys, w = torch.nan_to_num(ys), torch.nan_to_num(w)
    idx = torch.from_numpy(route(12, tokens, topk, experts, 0.1)).cuda()

    def step(**kw):
        sl, so, c, o = lib.fp8_moe_sort(idx, experts, **kw)
        xs = lib.fp8_moe_dispatch(x, sl, so, **kw)
        y = lib.fp8_moe_combine(ys, sl, w, **kw)
        dys, dw = lib.fp8_moe_combine_bwd(x, ys, sl, so, w, **kw)
        dx = lib.fp8_moe_dispatch_bwd(dys, sl, **kw)
        return [sl, so, c, o, xs, y, dys, dw, dx]

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = step(stream=s)
        torch.full((4000, cols), 2.0, device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        idx.copy_(torch.from_numpy(route(20 + k, tokens, topk, experts, 0.1)))
        x.copy_(torch.randn(x.shape, device="cuda"))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), k
