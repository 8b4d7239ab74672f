"""A training step of the grouped expert block, forward and backward, captured once and replayed with
other tokens: every gradient bit for bit that of the eager step, with eager work between replays."""
import pytest

from tests.gpu_util import note

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BF = torch.bfloat16


def test_training_step_in_a_graph():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import scaled_fp8_linear_amd as m
    m.load()
    note("GroupedExpertBlock, a training step in a graph")
    torch.manual_seed(0)
    block = m.GroupedExpertBlock(256, 384, 8, 2, device="cuda")
    shadow = m.GroupedExpertBlock(256, 384, 8, 2, device="cuda")     # eager steps have leaves of their own
    shadow.load_state_dict(block.state_dict())
    x = torch.randn(300, 256, device="cuda", dtype=BF)
    dy = torch.randn(300, 256, device="cuda", dtype=BF)

    def step(b):
        y, r = b(x)
        torch.autograd.backward([y, r.balance_loss, r.z_loss],
                                [dy, torch.full_like(r.balance_loss, 0.5),
                                 torch.full_like(r.z_loss, 0.25)])
        return y.detach(), r.counts

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):                       # library handles are made here
            step(block)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for p in block.parameters():
        p.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, counts = step(block)
    for seed in (1, 2, 3, 1):
        torch.manual_seed(seed)
        x.copy_(torch.randn(300, 256, device="cuda") * seed)
        dy.copy_(torch.randn(300, 256, device="cuda"))
        for p in block.parameters():
            p.grad.zero_()                       # a replay adds or sets; from zero both are the same
        g.replay()
        torch.cuda.synchronize()
        for p in shadow.parameters():
            p.grad = None
        want, wc = step(shadow)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(counts, wc)
        for (n, p), q in zip(block.named_parameters(), shadow.parameters()):
            assert torch.equal(p.grad, q.grad), n
            assert (p.grad != 0).any(), n
