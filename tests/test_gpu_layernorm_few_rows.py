"""The gradient of few rows (dx by rows, the parameters' gradients by columns) at and around the
sizes where it gives way to partial sums, against the float64 oracle; what is wanted does not
change what comes out; results repeat."""
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


def host(t):
    return t.detach().cpu().double().numpy()


# sizes of one turn of a workgroup and one row more, and around earlier and present limits
@pytest.mark.parametrize("rows,cols", [(1, 5), (64, 100), (65, 100), (16, 600), (17, 601), (8, 2000),
                                       (9, 2001), (2, 5003), (268, 193), (524, 100), (525, 100),
                                       (262, 97), (263, 97), (672, 1280), (673, 1280), (416, 2561),
                                       (1, 16384), (2, 16384), (130, 12301)])
@pytest.mark.parametrize("dt,pdt", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                    ("f32", "f32")])
def test_few_rows(lib, rows, cols, dt, pdt):
    if (rows, cols, pdt) == (1, 16384, "f16"):
        pytest.skip("a product below float16's normal range (6.1e-5) is rounded by up to 2^-25, "
                    "which this bound, relative to the value, leaves out; "
                    "test_single_rows_of_f16 counts it")
    g = torch.Generator().manual_seed(rows * 7 + cols)
    wide = torch.randn(rows, cols + 9, generator=g).to(DT[dt]).cuda()
    x, dy = wide[:, 4:cols + 4], torch.randn(rows, cols, generator=g).to(DT[dt]).cuda()
    gamma = (1 + 0.3 * torch.randn(cols, generator=g)).to(DT[pdt]).cuda()
    note(f"layernorm_bwd few rows {rows}x{cols} {dt}/{pdt}")
    _, mean, rstd = lib.fp8_layernorm_fwd(x, gamma)
    got = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    torch.cuda.synchronize()
    args = (host(dy), host(x), host(mean), host(rstd), host(gamma))
    half, half_p = torch.finfo(DT[dt]).eps / 2, torch.finfo(DT[pdt]).eps / 2
    for a, w, b, n in zip(got, ln.backward(*args), ln.backward_bounds(*args, half, half_p),
                          ("dx", "dgamma", "dbeta")):
        assert_within(host(a), w, b, n)
    again = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    for keep in range(3):
        want = {n: i == keep for i, n in enumerate(("want_dx", "want_dgamma", "want_dbeta"))}
        one = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma, **want)[keep]
        torch.cuda.synchronize()
        assert torch.equal(one, got[keep]) and torch.equal(again[keep], got[keep])


def test_a_nan_stays_in_its_row_and_column_sums(lib):
    g = torch.Generator().manual_seed(3)
    x, dy = torch.randn(40, 1100, generator=g).cuda(), torch.randn(40, 1100, generator=g).cuda()
    _, mean, rstd = lib.fp8_layernorm_fwd(x)
    clean = lib.fp8_layernorm_bwd(dy, x, mean, rstd)
    dy[7, 1099] = float("nan")
    dx, dgamma, dbeta = lib.fp8_layernorm_bwd(dy, x, mean, rstd)
    torch.cuda.synchronize()
    rows = torch.arange(40, device="cuda") != 7
    assert torch.equal(dx[rows], clean[0][rows]) and torch.isnan(dx[7]).all()
    assert torch.equal(dgamma[:-1], clean[1][:-1]) and torch.isnan(dgamma[-1])
    assert torch.equal(dbeta[:-1], clean[2][:-1]) and torch.isnan(dbeta[-1])


@pytest.mark.parametrize("cols", [16384, 7001, 129])
def test_single_rows_of_f16(lib, cols):
    """dgamma of one row is a single product, as small as the row's values are near the mean. Half
    a step of float16 is 2^-11 of the value, and never below 2^-25."""
    g = torch.Generator().manual_seed(cols)
    x, dy = (torch.randn(1, cols, generator=g).half().cuda() for _ in range(2))
    gamma = torch.randn(cols, generator=g).half().cuda()
    note(f"layernorm_bwd one row of f16, cols={cols}")
    _, mean, rstd = lib.fp8_layernorm_fwd(x, gamma)
    got = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    torch.cuda.synchronize()
    args = (host(dy), host(x), host(mean), host(rstd), host(gamma))
    for a, w, b, n in zip(got, ln.backward(*args), ln.backward_bounds(*args, 2.0 ** -11, 2.0 ** -11),
                          ("dx", "dgamma", "dbeta")):
        assert_within(host(a), w, b + 2.0 ** -25, n)


# the largest number of rows by columns and one more: 2-byte types up to 1000 + cols / 4 rows,
# float32 half of that
@pytest.mark.parametrize("rows,cols,dt", [(1025, 100, "bf16"), (1026, 100, "bf16"),
                                          (1503, 2015, "f16"), (1504, 2015, "f16"),
                                          (512, 97, "f32"), (513, 97, "f32"), (1125, 5003, "f32"),
                                          (1126, 5003, "f32"), (2048, 8192, "bf16"),
                                          (2049, 8192, "bf16")])
def test_limits_of_few_rows(lib, rows, cols, dt):
    g = torch.Generator().manual_seed(rows + cols)
    x, dy = (torch.randn(rows, cols, generator=g).to(DT[dt]).cuda() for _ in range(2))
    gamma = (1 + 0.3 * torch.randn(cols, generator=g)).cuda()
    note(f"layernorm_bwd at the limit of few rows {rows}x{cols} {dt}")
    _, mean, rstd = lib.fp8_layernorm_fwd(x, gamma)
    got = lib.fp8_layernorm_bwd(dy, x, mean, rstd, gamma)
    torch.cuda.synchronize()
    args = (host(dy), host(x), host(mean), host(rstd), host(gamma))
    for a, w, b, n in zip(got, ln.backward(*args),
                          ln.backward_bounds(*args, torch.finfo(DT[dt]).eps / 2, 2.0 ** -24),
                          ("dx", "dgamma", "dbeta")):
        tol = b + 2.0 ** -25 if dt == "f16" and n == "dx" else b      # float16's subnormal step
        assert_within(host(a), w, tol, n)
