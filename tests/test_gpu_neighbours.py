"""Outputs that lie next to the inputs, or between an input's rows, without sharing a byte are no
shared memory: the same results as in tensors of their own."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    m.load()
    return m


def in_one_buffer(*likes):
    """Tensors like these, one right behind the other."""
    sizes = [t.numel() * t.element_size() for t in likes]
    assert all(n % 16 == 0 for n in sizes)
    buffer, at, out = torch.empty(sum(sizes), dtype=U8, device="cuda"), 0, []
    for t, n in zip(likes, sizes):
        out.append(buffer[at:at + n].view(t.dtype).view(t.shape))
        at += n
    return out


@pytest.mark.parametrize("gated", [False, True])
def test_act_back_to_back(lib, gated):
    note(f"activation, tensors back to back, gated={gated}")
    torch.manual_seed(0)
    h = torch.randn(256, 512 if gated else 256, device="cuda").to(BF)
    want = lib.fp8_act_quantize(h, "gelu", gated)
    q, s, hh, q_t, s_t, hq, hs = in_one_buffer(*want[:2], h, *want[2:])
    hh.copy_(h)
    lib.fp8_act_quantize(hh, "gelu", gated, None, q, s, q_t, s_t, hq, hs)
    assert all(torch.equal(a, b) for a, b in zip((q, s, q_t, s_t, hq, hs), want))
    da = torch.randn(256, 256, device="cuda").to(BF)
    back = lib.fp8_act_quantize_bwd(da, *want[4:], "gelu", gated, want_dh=True)
    dh, hq2, q, s, d, q_t, s_t, hs2 = in_one_buffer(back[4], hq, *back[:2], da, *back[2:4], hs)
    d.copy_(da), hq2.copy_(hq), hs2.copy_(hs)
    lib.fp8_act_quantize_bwd(d, hq2, hs2, "gelu", gated, None, q, s, q_t, s_t, dh)
    assert all(torch.equal(a, b) for a, b in zip((q, s, q_t, s_t, dh), back))


def test_act_gradient_between_rows(lib):
    """dh in the gap between two rows of da."""
    note("activation gradient between rows")
    torch.manual_seed(1)
    rows, cols = 128, 128
    h = torch.randn(rows, cols, device="cuda").to(BF)
    hq, hs = lib.fp8_act_quantize(h, "silu", False)[4:]
    ld = cols + rows * cols
    buffer = torch.zeros(2 * ld + (rows - 2) * ld + cols, dtype=BF, device="cuda")
    da = buffer.as_strided((rows, cols), (ld, 1))
    da.copy_(torch.randn(rows, cols, device="cuda"))
    want = lib.fp8_act_quantize_bwd(da.contiguous(), hq, hs, "silu", False, want_dh=True)[4]
    for row in (0, 1, rows - 2):
        dh = buffer[row * ld + cols:(row + 1) * ld].view(rows, cols)
        lib.fp8_act_quantize_bwd(da, hq, hs, "silu", False, want_q=False, want_q_t=False, dh=dh)
        assert torch.equal(dh, want)


def test_products_back_to_back(lib):
    note("grouped products, tensors back to back")
    torch.manual_seed(2)
    e, n, k = 3, 256, 384
    idx = torch.randint(0, e, (150, 2), device="cuda")
    plan = lib.expert_plan(idx, e, 128)
    x = lib.expert_dispatch(torch.randn(150, k, device="cuda").to(BF), plan)
    g = lib.expert_dispatch(torch.randn(150, n, device="cuda").to(BF), plan)
    w = torch.randn(e * n, k, device="cuda").to(BF)
    B = lib.FP8_BLOCK_1x128
    qx, qx_t, _, sx, sx_t = lib.fp8_quantize_amax(x, gran=B, want_amax=False)
    qg, qg_t, _, sg, sg_t = lib.fp8_quantize_amax(g, gran=B, want_amax=False)
    q, _, _, s, _ = lib.fp8_quantize_amax(w, gran=lib.FP8_BLOCK_128x128, want_amax=False)
    qw, sw = q.view(e, n, k), s.view(e, n // 128, k // 128)
    y = lib.fp8_grouped_linear_fwd(qx, qw, sx, sw, plan.offsets, plan.counts)
    x2, y2, w2 = in_one_buffer(qx, y, qw)
    x2.copy_(qx), w2.copy_(qw)
    lib.fp8_grouped_linear_fwd(x2, w2, sx, sw, plan.offsets, plan.counts, y2)
    assert torch.equal(y2, y)
    # y between the rows that two experts' weights alternate in
    wide = torch.zeros(n, e * k + 2 * y.numel(), dtype=U8, device="cuda")
    alt = wide[:, :e * k].view(n, e, k).transpose(0, 1)
    alt.copy_(qw)
    y3 = wide[7, e * k:].view(BF).view(y.shape)
    lib.fp8_grouped_linear_fwd(qx, alt, sx, sw, plan.offsets, plan.counts, y3)
    assert torch.equal(y3, y)
    dw = lib.fp8_grouped_linear_wgrad(qg_t, qx_t, sg_t, sx_t, plan.offsets, plan.counts)
    g2, dw2, x2 = in_one_buffer(qg_t, dw, qx_t)
    g2.copy_(qg_t), x2.copy_(qx_t)
    lib.fp8_grouped_linear_wgrad(g2, x2, sg_t, sx_t, plan.offsets, plan.counts, dw2)
    assert torch.equal(dw2, dw)
