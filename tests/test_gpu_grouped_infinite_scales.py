"""Grouped products of a few K blocks with infinite scales: an infinity where the formula has one, and
none elsewhere (codes are positive, so that no sum is 0 times infinity).

Bound of the finite ones: terms of one sign, so the float32 sums are within 2^-9 of the value (the
block oracle's bound) and their rounding to bf16 within 2^-8 of that."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

U8, I32 = torch.uint8, torch.int32
INF = float("inf")
BOUND = 2.0 ** -9 + 2.0 ** -8 * (1 + 2.0 ** -9)


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    m.load()
    return m


def codes(*shape):
    return torch.randint(0x20, 0x50, shape, device="cuda", dtype=U8)


def value(q):
    return q.view(torch.float8_e4m3fn).double()


def compare(got, want):
    got = got.double()
    inf = torch.isinf(want)
    assert not torch.isnan(got).any() and torch.equal(torch.isinf(got), inf)
    assert (got[inf] == want[inf]).all() and inf.any() and not inf.all()
    assert ((got - want)[~inf].abs() <= BOUND * want[~inf]).all()


# tiles of 128 x 256, of 256 x 256, and streams of 32 and of 8 rows
@pytest.mark.parametrize("rows,n,k,most", [(4096, 1024, 128, None), (4096, 1024, 256, None),
                                           (4096, 1024, 384, None), (4096, 1024, 640, None),
                                           (32768, 2048, 128, None), (32768, 2048, 256, None),
                                           (384, 256, 128, None), (384, 256, 384, None),
                                           (384, 256, 256, 8)])
def test_product(lib, rows, n, k, most):
    note(f"grouped product, infinite scales, {rows} rows {n} x {k} max_rows={most}")
    torch.manual_seed(k)
    x, w = codes(rows, k), codes(1, n, k)
    sx = torch.rand(rows, k // 128, device="cuda") + 0.5
    sw = torch.rand(1, n // 128, k // 128, device="cuda") + 0.5
    sx[::5, -1] = INF
    sx[2] = 1e30                                 # times this the product of two finite scales is one
    sw[0, 1, 0] = 1e30
    sw[0, 0, -1] = INF
    counts = torch.tensor([rows - 77], device="cuda", dtype=I32)
    offsets = torch.tensor([0, rows], device="cuda", dtype=I32)
    y = lib.fp8_grouped_linear_fwd(x, w, sx, sw, offsets, counts, max_rows=most)
    want = sum(sx[:, b, None].double() * sw[0, :, b].double().repeat_interleave(128) *
               (value(x[:, 128 * b:128 * b + 128]) @ value(w[0, :, 128 * b:128 * b + 128]).T)
               for b in range(k // 128))
    want[rows - 77:] = 0
    want[want > torch.finfo(torch.bfloat16).max] = INF       # far above what rounds to the largest
    assert (y[rows - 77:] == 0).all()
    compare(y[:rows - 77], want[:rows - 77])


# tiles of 128 x 128, of 256 x 256, and streams
@pytest.mark.parametrize("n", [2048, 4096, 256])
def test_weight_gradient(lib, n):
    note(f"grouped weight gradient, infinite scales, {n} x {n}")
    torch.manual_seed(n)
    counts, offsets, rows = [128, 300, 100], [0, 128, 512, 640], 640
    g, x = codes(n, rows), codes(n, rows)
    for e in range(3):
        for q in (g, x):
            q[:, offsets[e] + counts[e]:offsets[e + 1]] = 0
    sg = torch.rand(n, 5, device="cuda") + 0.5
    sx = torch.rand(n, 5, device="cuda") + 0.5
    sg[3::7, 0], sg[5::9, 4], sg[6::11, 2] = INF, INF, INF
    sx[2::13, 0], sx[2::17, 4] = INF, INF
    dw = lib.fp8_grouped_linear_wgrad(g, x, sg, sx, torch.tensor(offsets, device="cuda", dtype=I32),
                                      torch.tensor(counts, device="cuda", dtype=I32))
    for e in range(3):
        want = sum(sg[:, b, None].double() * sx[:, b].double() *
                   (value(g[:, 128 * b:128 * b + 128]) @ value(x[:, 128 * b:128 * b + 128]).T)
                   for b in range(offsets[e] // 128, offsets[e + 1] // 128))
        compare(dw[e], want)
