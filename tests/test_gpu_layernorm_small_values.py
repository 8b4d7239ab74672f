"""Layer norm and its gradient where the stored values fall below the normal range of float16, with
bounds that count the steps of the type there: one row of any width (its dgamma is a single
product) and small gradients of many rows, by either form of the backward."""
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


@pytest.mark.parametrize("rows,cols", [(1, 16384), (1, 16400), (1, 77), (2, 5003), (40, 1000),
                                       (1600, 264), (1203, 1030)])
@pytest.mark.parametrize("pdt", ["f16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -12])
def test_f16_below_its_normal_range(lib, rows, cols, pdt, scale):
    g = torch.Generator().manual_seed(rows * 7 + cols)
    wide = torch.randn(rows, cols + 9, generator=g).half().cuda()
    x, dy = wide[:, 4:cols + 4], (scale * torch.randn(rows, cols, generator=g)).half().cuda()
    gamma = (scale * torch.randn(cols, generator=g)).to(DT[pdt]).cuda()
    beta = (scale * torch.randn(cols, generator=g)).to(DT[pdt]).cuda()
    note(f"layernorm of small f16 values {rows}x{cols} {pdt} {scale}")
    y, mean, rstd = lib.fp8_layernorm_fwd(x, gamma, beta)
    got = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    torch.cuda.synchronize()
    half, tiny = steps(torch.float16)
    half_p, tiny_p = steps(DT[pdt])
    fwd = (host(x), host(gamma), host(beta), np.float64(np.float32(1e-5)))
    assert_within(host(y), ln.forward(*fwd)[0], ln.forward_bounds(*fwd, half, tiny)[0], "y")
    args = (host(dy), host(x), host(mean), host(rstd), host(gamma))
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
