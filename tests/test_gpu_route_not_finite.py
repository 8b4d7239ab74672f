"""Rows of the router with NaN or infinity beside masked experts: no choice (-1) has weight 0, a masked
expert and padding have gradient 0, and other rows are as they are without them."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    m.load()
    return m


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("experts", [5, 12, 30, 60, 100, 200, 400])
@pytest.mark.parametrize("normalize", [True, False])
def test_masked_beside_not_finite(lib, dt, experts, normalize):
    note(f"route, not finite, {dt} {experts} experts normalize={normalize}")
    torch.manual_seed(experts)
    x = torch.randn(9, experts, device="cuda").to(dt)
    x[1:5] = -INF
    x[1, 3] = NAN                                # one choice left: NaN, +inf, both, a number
    x[2, 2] = INF
    x[3, 1], x[3, 4] = INF, NAN
    x[4, 0] = 1.0
    x[5, 3] = NAN                                # nothing masked
    x[6, ::2] = -INF                             # finite
    x[7] = -INF                                  # nothing left
    valid = 8
    x[8] = NAN                                   # padding
    idx, w, lse, counts, losses = lib.fp8_moe_route(x, 4, valid, normalize)
    left = [[3], [2], [4, 1], [0]]
    for row, want in zip(idx[1:5].tolist(), left):
        assert row == want + [-1] * (4 - len(want))
    assert (w[idx < 0] == 0).all()
    assert torch.isnan(w[1:4][idx[1:4] >= 0]).all() and w[4, 0] == 1 and torch.isnan(w[5]).all()
    assert torch.isnan(lse[[1, 2, 3, 5]]).all() and torch.isfinite(lse[[0, 4, 6]]).all()
    assert lse[7] == -INF and lse[8] == 0
    assert torch.isnan(losses).all()
    dw = torch.randn(9, 4, device="cuda")
    masked = x == -INF
    for dl in (None, torch.tensor([1.0, 0.5], device="cuda"), torch.tensor([NAN, NAN], device="cuda"),
               losses, torch.tensor([INF, -INF], device="cuda")):
        for g in (dw, None):
            d = lib.fp8_moe_route_bwd(x, lse, idx, w, counts, g, dl, valid, normalize)
            assert (d[masked] == 0).all() and (d[valid:] == 0).all()
            if dl is None or torch.isfinite(dl).all():
                ok = [0, 4, 6, 7]
                assert torch.isfinite(d[ok]).all()
                # a row's gradient is its own
                y = x.clone()
                y[[1, 2, 3, 5]] = 0
                l2, w2, i2 = lse.clone(), w.clone(), idx.clone()
                l2[[1, 2, 3, 5]], w2[[1, 2, 3, 5]], i2[[1, 2, 3, 5]] = 1, 0, -1
                d2 = lib.fp8_moe_route_bwd(y, l2, i2, w2, counts, g, dl, valid, normalize)
                assert torch.equal(d[ok], d2[ok])
