"""Rows whose values are all the same and so large that mean * rstd leaves float32: their normalised
values are 0, so the gradient is finite, whatever the lanes past the row's end hold. Widths that fill
their lanes and pieces and widths that do not, in both forms of the backward."""
import numpy as np
import pytest

from oracle import layernorm as ln
from tests.gpu_util import assert_within, note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def host(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("rows,cols", [(6, 1), (6, 3), (6, 5), (6, 24), (6, 23), (6, 100), (6, 700),
                                       (6, 1500), (6, 1501), (6, 16385), (2001, 3), (2001, 7),
                                       (2001, 101), (2501, 301), (2501, 1000), (3001, 1501),
                                       (1501, 5003)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_constant_rows(rows, cols, dt):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    g = torch.Generator().manual_seed(rows + cols)
    x = torch.randn(rows, cols, generator=g)
    far = [0, rows // 2, rows - 1]
    x[far] = torch.tensor([2.0 ** 110, -2.0 ** 110, 2.0 ** 110])[:, None]   # their sums are exact
    x = x.to(DT[dt]).cuda()
    dy = (1e-3 * torch.randn(rows, cols, generator=g)).to(DT[dt]).cuda()
    gamma = (1 + 0.3 * torch.randn(cols, generator=g)).cuda()
    note(f"layernorm_bwd large constant rows {rows}x{cols} {dt}")
    y, mean, rstd = m.fp8_layernorm_fwd(x, gamma, eps=1e-12)
    got = m.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    torch.cuda.synchronize()
    assert torch.equal(mean[far], x[far, 0].float()) and not y[far].any()
    assert bool((mean[far].double() * rstd[far].double()).abs().min() > 2.0 ** 128)
    args = (host(dy), host(x), host(mean), host(rstd), host(gamma))
    half = torch.finfo(DT[dt]).eps / 2
    for a, w, b, n in zip(got, ln.backward(*args), ln.backward_bounds(*args, half, 2.0 ** -24),
                          ("dx", "dgamma", "dbeta")):
        assert_within(host(a), w, b, n)
