"""Plans of expert_mlp on the device: what an expert's gradients would get of another's rows, plans
made of the index tensors alone, and captures."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    m.load()
    return m


def setup(lib, multiple):
    """150 and 50 tokens to two experts."""
    torch.manual_seed(0)
    idx = (torch.arange(200, device="cuda") >= 150).long().view(200, 1)
    plan = lib.expert_plan(idx, 2, multiple)
    xs = lib.expert_dispatch(torch.randn(200, 128, device="cuda").to(BF), plan)
    up = (torch.randn(2, 512, 128, device="cuda") / 11).to(BF).requires_grad_(True)
    down = (torch.randn(2, 128, 256, device="cuda") / 16).to(BF).requires_grad_(True)
    return plan, xs, up, down


def test_mixed_blocks_are_refused(lib):
    note("expert_mlp, plan with multiple 96")
    plan, xs, up, down = setup(lib, 96)
    assert plan.offsets.tolist() == [0, 192, 288] and xs.shape[0] == 384
    for p in (plan, lib.ExpertPlan(*plan)):
        with pytest.raises(ValueError, match="mix experts"):
            lib.expert_mlp(xs, up, down, p)


def test_plan_of_the_tensors_alone(lib):
    """The same bits as the plan itself; in a capture only without weight gradients."""
    note("expert_mlp, plan made of the tensors")
    plan, xs, up, down = setup(lib, 128)
    bare = lib.ExpertPlan(*plan)
    got = []
    for p in (plan, bare):
        up.grad = down.grad = None
        y = lib.expert_mlp(xs, up, down, p)
        y.backward(xs)
        got.append((y, up.grad, down.grad))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    torch.cuda.synchronize()
    with torch.no_grad():
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = lib.expert_mlp(xs, up, down, bare)
        for scale in (1.0, 2.0, 1.0):
            xs.mul_(scale)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, lib.expert_mlp(xs, up, down, plan))
    refused = []
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = xs + 1                               # a graph of something
        try:
            lib.expert_mlp(xs, up, down, bare)
        except ValueError as e:
            refused.append(str(e))
    assert refused and "capture" in refused[0]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, xs + 1)
