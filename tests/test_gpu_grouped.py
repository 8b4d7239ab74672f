"""GPU parity of the experts' products: every expert's rows within the block recipe's float32
bound, 0 in all other rows, whatever the counts and strides."""
import numpy as np
import pytest

from oracle import block
from tests.gpu_util import assert_within, host_bf16_f64, note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U = 2.0 ** -23


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    m.load()
    return m


def codes(g, *shape):
    """Codes of normal values, some of them small, none NaN."""
    v = torch.randn(*shape, generator=g) * 100
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def scales(g, *shape):
    return torch.exp(torch.randn(*shape, generator=g)) / 448


def layout(counts, multiple, extra=0, lead=0):
    offsets = [lead]
    for c in counts:
        offsets.append(offsets[-1] + -(-c // multiple) * multiple)
    return offsets, offsets[-1] + extra


def bound_of(qa, qb, sa, sb, b_rows):
    """The oracle's, and a rounding for each block whose sums another wave may have begun."""
    d, b = block.block_fp32_bound(qa, qb, sa, sb, b_rows)
    mag = np.abs(block.dequant_rows(qa, sa, 1)) @ np.abs(block.dequant_rows(qb, sb, b_rows)).T
    return d, b + U * (qa.shape[1] // 128 + 8) * mag


def dev(t):
    return t.cuda()


def check_products(lib, counts, N, K, multiple, extra=0, lead=0, max_rows=None, dgrad=False, seed=0,
                   given=None, strides=False):
    g = torch.Generator().manual_seed(seed)
    E = len(counts)
    offsets, rows = layout(counts, multiple, extra, lead)
    x, sx = codes(g, rows, K), scales(g, rows, K // 128)
    x[:, 3] = 0x7F                                    # rows of no expert may hold anything
    for e, c in enumerate(counts):
        x[offsets[e]:offsets[e] + c, 3] = 0x31
    w, sw = codes(g, E, N, K), scales(g, E, N // 128, K // 128)
    if strides:                                       # experts side by side along the columns
        wd = w.permute(1, 0, 2).contiguous().cuda().permute(1, 0, 2)
        swd = sw.permute(1, 0, 2).contiguous().cuda().permute(1, 0, 2)
    else:
        wd, swd = w.cuda(), sw.cuda()
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    cnt = torch.tensor(counts if given is None else given, dtype=torch.int32).cuda()
    y = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    f = lib.fp8_grouped_linear_dgrad if dgrad else lib.fp8_grouped_linear_fwd
    f(x.cuda(), wd, sx.cuda(), swd, off, cnt, y, max_rows=max_rows)
    torch.cuda.synchronize()
    got = host_bf16_f64(y)
    live = np.zeros(rows, bool)
    for e, c in enumerate(counts):
        r = slice(offsets[e], offsets[e] + c)
        live[r] = True
        if c:
            d, b = bound_of(x[r].numpy(), w[e].numpy(), sx[r].numpy(), sw[e].numpy(), 128)
            assert_within(got[r], d, b, f"expert {e}")
    assert (got[~live] == 0).all()
    return y


COUNTS = [[1], [0], [0, 3, 0, 17, 1], [16, 32, 33, 64, 65], [128, 0, 129, 255, 256, 257],
          [1] * 40, [0] * 20 + [5] + [0] * 30]
SIZES = [(128, 128), (256, 640), (384, 128), (128, 2048), (896, 1152)]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_products(lib, counts):
    for n, (N, K) in enumerate(SIZES):
        for max_rows in (None, max(counts)):
            note(f"grouped counts={counts} N={N} K={K} max_rows={max_rows}")
            check_products(lib, counts, N, K, 128, extra=128 * (n % 2), max_rows=max_rows, seed=n)


@pytest.mark.parametrize("multiple,extra,lead", [(1, 0, 0), (1, 5, 3), (16, 0, 16), (3, 1, 0)])
def test_rows_at_any_place(lib, multiple, extra, lead):
    for counts in ([7, 0, 40, 1, 130], [300, 2]):
        for max_rows in (None, max(counts)):
            note(f"grouped multiple={multiple} extra={extra} lead={lead} counts={counts}")
            check_products(lib, counts, 256, 384, multiple, extra, lead, max_rows=max_rows)


def test_dgrad_of_stacked_transposed_weights(lib):
    for counts in ([3, 0, 70], [200, 129, 1]):
        for max_rows in (None, max(counts)):
            note(f"grouped dgrad {counts} {max_rows}")
            check_products(lib, counts, 384, 640, 128, dgrad=True, strides=True, max_rows=max_rows)


def test_a_wrong_bound_costs_speed_only(lib):
    note("grouped with a bound below the counts")
    a = check_products(lib, [300, 10, 90], 256, 256, 128, max_rows=1)
    b = check_products(lib, [300, 10, 90], 256, 256, 128, max_rows=10 ** 9)
    assert a.shape == b.shape


@pytest.mark.parametrize("off,cnt", [([0, 5000, -3, 40], [10, 10, 10]), ([-7, 2 ** 31 - 1, 128, 256], [1, 2, 3]),
                                     ([0, 128, 256, 384], [-5, 2 ** 31 - 1, 128]),
                                     ([300, 200, 100, 0], [50, 50, 50])])
def test_offsets_outside_the_tensors_are_clamped(lib, off, cnt):
    """Nothing outside y is written, whatever the offsets and counts say."""
    note(f"grouped offsets {off} {cnt}")
    g = torch.Generator().manual_seed(1)
    rows, N, K = 384, 128, 256
    room = torch.full((rows + 256, N), 3.0, dtype=torch.bfloat16, device="cuda")
    o = torch.tensor(off, dtype=torch.int32).cuda()
    c = torch.tensor(cnt, dtype=torch.int32).cuda()
    for max_rows in (16, None):
        lib.fp8_grouped_linear_fwd(codes(g, rows, K).cuda(), codes(g, 3, N, K).cuda(),
                                   scales(g, rows, 2).cuda(), scales(g, 3, 1, 2).cuda(), o, c,
                                   room[128:128 + rows], max_rows=max_rows)
        torch.cuda.synchronize()
        assert (room[:128] == 3).all() and (room[128 + rows:] == 3).all()
    droom = torch.full((5, N, K), 3.0, dtype=torch.bfloat16, device="cuda")
    lib.fp8_grouped_linear_wgrad(codes(g, N, rows).cuda(), codes(g, K, rows).cuda(),
                                 scales(g, N, 3).cuda(), scales(g, K, 3).cuda(), o, c, droom[1:4])
    torch.cuda.synchronize()
    assert (droom[0] == 3).all() and (droom[4] == 3).all()


def check_wgrad(lib, counts, N, K, extra=0, lead=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    E = len(counts)
    offsets, rows = layout(counts, 128, extra, lead)
    live = torch.zeros(rows, dtype=torch.uint8)
    for e, c in enumerate(counts):
        live[offsets[e]:offsets[e] + c] = 1
    gq, xq = codes(g, N, rows) * live, codes(g, K, rows) * live
    gs, xs = scales(g, N, rows // 128), scales(g, K, rows // 128)
    gd, xd = gq.clone(), xq.clone()
    gd[:, offsets[-1]:], xd[:, offsets[-1]:] = 0x7F, 0x7F       # blocks of no expert are not read
    gd[:, :lead], xd[:, :lead] = 0x7F, 0x7F
    dw = torch.full((E, N, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    lib.fp8_grouped_linear_wgrad(gd.cuda(), xd.cuda(), gs.cuda(), xs.cuda(),
                                 torch.tensor(offsets, dtype=torch.int32).cuda(),
                                 torch.tensor(counts, dtype=torch.int32).cuda(), dw)
    torch.cuda.synchronize()
    got = host_bf16_f64(dw)
    for e, c in enumerate(counts):
        if not c:
            assert (got[e] == 0).all()
            continue
        b = slice(offsets[e] // 128, offsets[e + 1] // 128)
        r = slice(offsets[e], offsets[e + 1])
        d, bound = bound_of(gq[:, r].numpy(), xq[:, r].numpy(), gs[:, b].numpy(), xs[:, b].numpy(), 1)
        assert_within(got[e], d, bound, f"expert {e}")


@pytest.mark.parametrize("counts", COUNTS + [[640, 1, 0, 1025], [512] * 3, [130, 400, 600, 897]],
                         ids=lambda c: f"{len(c)}x{max(c)}")
def test_wgrad(lib, counts):
    for n, (N, K) in enumerate([(128, 128), (256, 640), (384, 256), (640, 128)]):
        note(f"grouped wgrad counts={counts} N={N} K={K}")
        check_wgrad(lib, counts, N, K, extra=128 * (n % 2), lead=128 * (n // 2), seed=n)


# outputs of one round of tiles and more, whose tiles are 128 or 256 rows high, and of few of them
@pytest.mark.parametrize("counts,N,K", [([300, 1, 0, 129], 4352, 384), ([1100, 0, 130], 5120, 640),
                                        ([2000, 130, 0], 8448, 128), ([4096], 6144, 256),
                                        ([20, 0, 31, 1], 4352, 128), ([250, 90], 1024, 2176)],
                         ids=lambda v: str(v))
def test_products_of_many_tiles(lib, counts, N, K):
    note(f"grouped counts={counts} N={N} K={K}")
    check_products(lib, counts, N, K, 128, extra=128)
    if N * K < 2 ** 21:
        check_products(lib, counts, N, K, 8, extra=8, lead=8)


@pytest.mark.parametrize("counts,N,K", [([130, 0, 400], 1152, 896), ([300, 0, 129, 640], 1664, 1920),
                                        ([128, 0, 1], 2688, 2688), ([128, 0, 130, 1], 3200, 2048),
                                        ([2000, 3], 256, 384)], ids=lambda v: str(v))
def test_wgrad_of_many_tiles(lib, counts, N, K):
    note(f"grouped wgrad counts={counts} N={N} K={K}")
    check_wgrad(lib, counts, N, K, extra=128, lead=128)


@pytest.mark.parametrize("experts", [62, 63, 130, 300])
def test_many_experts(lib, experts):
    """Spans of more than one wave's lanes, the last of them without rows."""
    counts = [(7 * e * e + 3) % 41 if e % 5 else 0 for e in range(experts - 3)] + [0, 130, 0]
    for max_rows in (8, None):
        note(f"grouped {experts} experts max_rows={max_rows}")
        check_products(lib, counts, 128, 256, 16, max_rows=max_rows)
    note(f"grouped wgrad {experts} experts")
    check_wgrad(lib, counts, 128, 256)


def test_more_tiles_than_a_list(lib):
    """A workgroup's tiles come in lists of some. A block of K alone has the same float32 products
    whatever the order, so the forms for many rows and for few have to agree to the bit."""
    note("grouped: 64 tiles a workgroup")
    g = torch.Generator("cuda").manual_seed(5)
    E, N, K, each = 512, 8192, 128, 34
    x = torch.randint(0, 120, (E * each, K), generator=g, device="cuda", dtype=torch.uint8)
    w = torch.randint(0, 120, (E, N, K), generator=g, device="cuda", dtype=torch.uint8)
    sx = torch.rand(E * each, 1, generator=g, device="cuda")
    sw = torch.rand(E, N // 128, 1, generator=g, device="cuda")
    off = torch.arange(0, E * each + 1, each, device="cuda", dtype=torch.int32)
    cnt = torch.full((E,), each, device="cuda", dtype=torch.int32)
    cnt[7], cnt[300] = 0, 5
    tiles = lib.fp8_grouped_linear_fwd(x, w, sx, sw, off, cnt)
    few = lib.fp8_grouped_linear_fwd(x, w, sx, sw, off, cnt, max_rows=8)
    assert torch.equal(tiles, few) and (tiles != 0).any()

    note("grouped wgrad: 129 tiles a workgroup")
    E, N, K = 65, 8192, 4096
    gq = torch.randint(0, 120, (N, E * 128), generator=g, device="cuda", dtype=torch.uint8)
    xq = torch.randint(0, 120, (K, E * 128), generator=g, device="cuda", dtype=torch.uint8)
    gs = torch.rand(N, E, generator=g, device="cuda")
    xs = torch.rand(K, E, generator=g, device="cuda")
    off = torch.arange(0, E * 128 + 1, 128, device="cuda", dtype=torch.int32)
    cnt = torch.full((E,), 128, device="cuda", dtype=torch.int32)
    cnt[64] = 1
    dw = lib.fp8_grouped_linear_wgrad(gq, xq, gs, xs, off, cnt)
    for e in (0, 31, 63, 64):
        r = slice(128 * e, 128 * e + 128)
        alone = lib.fp8_grouped_linear_wgrad(gq[:, r].contiguous(), xq[:, r].contiguous(),
                                             gs[:, e:e + 1].contiguous(), xs[:, e:e + 1].contiguous(),
                                             off[:2], cnt[e:e + 1].clone())
        assert torch.equal(dw[e:e + 1], alone) and (alone != 0).any()


def test_no_rows(lib):
    note("grouped without rows")
    g = torch.Generator().manual_seed(0)
    off, cnt = torch.zeros(4, dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    y = lib.fp8_grouped_linear_fwd(codes(g, 0, 128).cuda(), codes(g, 3, 256, 128).cuda(),
                                   scales(g, 0, 1).cuda(), scales(g, 3, 2, 1).cuda(), off, cnt)
    assert y.shape == (0, 256)
    dw = lib.fp8_grouped_linear_wgrad(codes(g, 128, 0).cuda(), codes(g, 256, 0).cuda(),
                                      scales(g, 128, 0).cuda(), scales(g, 256, 0).cuda(), off, cnt)
    assert dw.shape == (3, 128, 256) and (dw == 0).all()


def test_nan_stays_in_its_row(lib):
    note("grouped nan")
    g = torch.Generator().manual_seed(2)
    counts = [40, 200]
    offsets, rows = layout(counts, 128)
    x = codes(g, rows, 256)
    x[7, 9] = 0x7F
    x[128 + 150, 200] = 0xFF
    args = [t.cuda() for t in (x, codes(g, 2, 128, 256), scales(g, rows, 2), scales(g, 2, 1, 2),
                               torch.tensor(offsets, dtype=torch.int32),
                               torch.tensor(counts, dtype=torch.int32))]
    for max_rows in (40, None):
        y = lib.fp8_grouped_linear_fwd(*args, max_rows=max_rows)
        nan = torch.isnan(y)
        assert nan[7].all() and nan[128 + 150].all() and nan.sum().item() == 2 * 128


@pytest.mark.parametrize("max_rows", [16, None])
def test_streams_and_replays(lib, max_rows):
    note(f"grouped streams and replays {max_rows}")
    g = torch.Generator().manual_seed(3)
    rows, N, K, E = 512, 256, 512, 4
    x, w = codes(g, rows, K).cuda(), codes(g, E, N, K).cuda()
    sx, sw = scales(g, rows, K // 128).cuda(), scales(g, E, N // 128, K // 128).cuda()
    off = torch.arange(0, 513, 128, dtype=torch.int32).cuda()
    cnt = torch.tensor([16, 5, 0, 9], dtype=torch.int32).cuda()
    want = lib.fp8_grouped_linear_fwd(x, w, sx, sw, off, cnt, max_rows=max_rows)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lib.fp8_grouped_linear_fwd(x, w, sx, sw, off, cnt, max_rows=max_rows, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y = lib.fp8_grouped_linear_fwd(x, w, sx, sw, off, cnt, max_rows=max_rows)
    for c in ([16, 5, 0, 9], [0, 128, 3, 1], [16, 5, 0, 9]):
        cnt.copy_(torch.tensor(c, dtype=torch.int32))
        y.fill_(7.0)
        gr.replay()
        torch.cuda.synchronize()
        eager = lib.fp8_grouped_linear_fwd(x, w, sx, sw, off, cnt, max_rows=max_rows)
        assert torch.equal(y, eager)
    assert torch.equal(y, want)


def test_weights_past_32_bits(lib):
    """Experts' weights of 4.3 GB: the last expert's against the same weights alone."""
    note("grouped weights of 4.3 GB")
    g = torch.Generator().manual_seed(4)
    E, N, K = 128, 4096, 8192
    w = torch.zeros(E, N, K, dtype=torch.uint8, device="cuda")
    sw = scales(g, E, N // 128, K // 128).cuda()
    for e in (0, 63, 127):
        w[e] = torch.randint(0, 120, (N, K), generator=torch.Generator("cuda").manual_seed(e),
                             device="cuda", dtype=torch.uint8)
    counts = [0] * E
    counts[0], counts[63], counts[127] = 20, 130, 3
    offsets, rows = layout(counts, 128)
    x, sx = codes(g, rows, K).cuda(), scales(g, rows, K // 128).cuda()
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    cnt = torch.tensor(counts, dtype=torch.int32).cuda()
    for max_rows in (130, 3):
        y = lib.fp8_grouped_linear_fwd(x, w, sx, sw, off, cnt, max_rows=max_rows)
        for e in (0, 63, 127):
            r = slice(offsets[e], offsets[e + 1])
            alone = lib.fp8_grouped_linear_fwd(
                x[r].contiguous(), w[e:e + 1].clone(), sx[r].contiguous(), sw[e:e + 1].clone(),
                torch.tensor([0, offsets[e + 1] - offsets[e]], dtype=torch.int32).cuda(),
                cnt[e:e + 1].clone(), max_rows=max_rows)
            assert torch.equal(y[r], alone) and (y[r] != 0).any()
