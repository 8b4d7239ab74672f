"""A stack of experts' weights whose transposed rows are 2^23 codes apart, more than the products take."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16


def test_mlp_of_many_wide_experts():
    """512 experts of a gated hidden size of 8192, against the first 256 of them alone, to which all
    tokens go: the same bits of outputs and gradients, which are 0 for the rest."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    note("expert_mlp, 512 experts, 128 x 8192 gated")
    e, cols, hidden, tokens = 512, 128, 8192, 8
    torch.manual_seed(0)
    up = torch.empty(e, 2 * hidden, cols, device="cuda", dtype=BF).uniform_(-0.1, 0.1)
    down = torch.empty(e, cols, hidden, device="cuda", dtype=BF).uniform_(-0.02, 0.02)
    idx = torch.randperm(e // 2, device="cuda")[:2 * tokens].view(tokens, 2)
    x = torch.randn(tokens, cols, device="cuda").to(BF)
    dy = torch.randn(tokens, cols, device="cuda").to(BF)
    got = []
    for n in (e, e // 2):
        plan = m.expert_plan(idx, n, 128)
        xs, dys = m.expert_dispatch(x, plan), m.expert_dispatch(dy, plan)
        leaves = [t.detach().requires_grad_(True) for t in (xs, up[:n], down[:n])]
        ys = m.expert_mlp(*leaves, plan)
        ys.backward(dys)
        got.append([ys.detach()] + [t.grad for t in leaves])
    whole, half = got
    assert torch.equal(whole[0], half[0]) and torch.equal(whole[1], half[1])
    assert (whole[1] != 0).any()
    for a, b in zip(whole[2:], half[2:]):
        assert torch.equal(a[:e // 2], b) and (b != 0).any()
        assert not a[e // 2:].any()
