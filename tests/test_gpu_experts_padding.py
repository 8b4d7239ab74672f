"""What the padding rows of a plan hold inside an expert of two linears: zeros without biases, the
activation of the bias with them (which the second linear's amax then includes), and gradients of
exactly zero at every place either way, in bf16 and in FP8."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_padding_rows_inside_an_expert(bias, fp8):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    torch.manual_seed(3)
    tokens, cols, hidden = 37, 64, 96
    up = m.Fp8Linear(cols, hidden, bias=bias, device="cuda")
    down = m.Fp8Linear(hidden, cols, bias=bias, device="cuda")
    if bias:                                     # one that stands out of the rows' own values
        with torch.no_grad():
            up.bias[5] = 64.0
    plan = m.expert_plan(torch.zeros((tokens, 1), dtype=torch.int64, device="cuda"), 1)
    pad = plan.source < 0
    x = torch.randn(tokens, cols, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    w = torch.rand(tokens, 1, device="cuda")
    note(f"padding rows inside an expert, bias={bias} fp8={fp8}")
    m.fp8_state().reset()
    with m.fp8_autocast(enabled=fp8):
        xs = m.expert_dispatch(x, plan)
        h = up(xs)
        a = torch.relu(h)
        ys = down(a)
        for t in (xs, h, a, ys):
            t.retain_grad()
        y = m.expert_combine(ys, w, plan)
    y.backward(torch.randn_like(y))
    torch.cuda.synchronize()
    m.fp8_state().reset()
    assert int(pad.sum()) == 48 - tokens and not xs[pad].any()
    if bias:
        assert torch.equal(a[pad], torch.relu(up.bias).expand(48 - tokens, hidden))
        assert bool((a[pad][:, 5] == 64).all())
    else:
        assert not h[pad].any() and not ys[pad].any()
    for t in (xs, h, a, ys):
        assert not t.grad[pad].any() and bool(t.grad[~pad].any())
    assert torch.isfinite(x.grad).all()
