"""Layer norm, dispatch and combine under autograd, and the expert block: gradients bit for bit
those of the direct calls, an expert block against the same chain of plain operations, masked
experts, no tokens, and a run that trains in FP8."""
import numpy as np
import pytest

from oracle import moe
from tests.gpu_util import assert_within, note

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


def host(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("dt,pdt", [(BF, torch.float32), (BF, BF), (torch.float32, torch.float32)])
def test_layer_norm_gradients_are_the_direct_calls(lib, dt, pdt):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 17, 200, generator=g).to(dt).cuda().requires_grad_(True)
    dy = torch.randn(3, 17, 200, generator=g).to(dt).cuda()
    norm = lib.LayerNorm(200, device="cuda", dtype=pdt)
    with torch.no_grad():
        norm.weight.copy_(torch.randn(200, generator=g))
        norm.bias.copy_(torch.randn(200, generator=g))
    note(f"LayerNorm autograd {dt} {pdt}")
    y = norm(x)
    y.backward(dy)
    w, b = norm.weight.detach(), norm.bias.detach()
    y2, mean, rstd = lib.fp8_layernorm_fwd(x.detach().view(51, 200), w, b)
    dx, dg, db = lib.fp8_layernorm_bwd(dy.view(51, 200), x.detach().view(51, 200), mean, rstd, w)
    torch.cuda.synchronize()
    assert torch.equal(y.view(51, 200), y2) and torch.equal(x.grad.view(51, 200), dx)
    assert torch.equal(norm.weight.grad, dg) and torch.equal(norm.bias.grad, db)


def test_layer_norm_odd_gradients_and_partial_needs(lib):
    """Expanded and transposed output gradients, strided inputs, and each input alone."""
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(20, 90, generator=g).cuda()
    gamma, beta = torch.randn(70, generator=g).cuda(), torch.randn(70, generator=g).cuda()
    dys = {"expanded": torch.ones((), device="cuda").expand(20, 70),
           "transposed": torch.randn(70, 20, generator=g).cuda().t()}
    x0 = wide[:, 11:81]
    _, mean, rstd = lib.fp8_layernorm_fwd(x0, gamma, beta)
    for kind, dy in dys.items():
        want = lib.fp8_layernorm_bwd(dy.contiguous(), x0, mean, rstd, gamma)
        for need in range(3):
            ins = [t.detach().requires_grad_(i == need) for i, t in enumerate((x0, gamma, beta))]
            note(f"layer_norm {kind} gradient, input {need}")
            lib.layer_norm(*ins).backward(dy)
            torch.cuda.synchronize()
            assert torch.equal(ins[need].grad, want[need])
            assert all(t.grad is None for i, t in enumerate(ins) if i != need)


def test_dispatch_and_combine_gradients(lib):
    g = torch.Generator().manual_seed(3)
    tokens, topk, experts, cols = 50, 3, 7, 136
    idx = torch.randint(-1, experts, (tokens, topk), generator=g).cuda()
    plan = lib.expert_plan(idx, experts)
    x = torch.randn(tokens, cols, generator=g).to(BF).cuda().requires_grad_(True)
    w = torch.rand(tokens, topk, generator=g).cuda().requires_grad_(True)
    note("expert_dispatch and expert_combine autograd")
    xs = lib.expert_dispatch(x, plan)
    ys = (xs * 2).detach().requires_grad_(True)
    y = lib.expert_combine(ys, w, plan)
    dy = torch.randn(tokens, cols, generator=g).to(BF).cuda()
    y.backward(dy)
    dxs = torch.randn(xs.shape, generator=g).to(BF).cuda()
    xs.backward(dxs)
    dys, dw = lib.fp8_moe_combine_bwd(dy, ys.detach(), plan.slot, plan.source, w.detach())
    dx = lib.fp8_moe_dispatch_bwd(dxs, plan.slot)
    torch.cuda.synchronize()
    assert torch.equal(ys.grad, dys) and torch.equal(w.grad, dw) and torch.equal(x.grad, dx)


def test_block_against_plain_operations(lib):
    """The block with its exchange replaced by indexing in float32: the experts see the same rows
    (bit for bit) and only the combine's last roundings and float32 sums may differ. So the
    output is off by at most a step of bf16 (two roundings of half a step each, of nearly equal
    values) plus the float32 bound, and the sum with x by half a step more."""
    torch.manual_seed(4)
    tokens, cols, hidden, experts, topk = 120, 96, 160, 6, 2
    lib.fp8_state().reset()
    block = lib.ExpertBlock(cols, hidden, experts, topk, device="cuda")
    x = torch.randn(tokens, cols, device="cuda", dtype=BF)
    note("ExpertBlock forward against indexing")
    out = block(x)
    with torch.no_grad():
        h = block.norm(x)
        idx, w = block.route(h)
        slot, source, _, offsets = lib.fp8_moe_sort(idx, experts)
        hs, at = slot.cpu().numpy(), offsets.tolist()
        xs = torch.zeros((source.numel(), cols), device="cuda", dtype=BF)
        live = source >= 0
        xs[live] = h[(source[live] // topk).long()]
        ys = torch.zeros_like(xs)
        for e in range(experts):
            if at[e + 1] > at[e]:
                r = slice(at[e], at[e + 1])
                ys[r] = block.down[e](torch.relu(block.up[e](xs[r])))
    torch.cuda.synchronize()
    want, bound = moe.combine(host(ys), hs, host(w))
    half = torch.finfo(BF).eps / 2
    total = host(x) + want
    tol = bound * 1.01 + half * np.abs(want) + half * (np.abs(total) + half * np.abs(want) + bound)
    assert_within(host(out), total, tol, "block output")


def test_block_trains_and_repeats(lib):
    """FP8 steps lower the loss, twice with the same numbers (nothing depends on timing)."""
    from examples.expert_block import train
    note("ExpertBlock trains in FP8")
    kw = dict(tokens=500, cols=128, hidden=256, experts=4, topk=2, steps=6, log=lambda *_: None)
    a, b = train(**kw), train(**kw)
    assert a == b and a[-1] < 0.9 * a[0]
    lib.fp8_state().reset()


def test_block_masked_experts_and_no_tokens(lib):
    torch.manual_seed(5)
    lib.fp8_state().reset()
    block = lib.ExpertBlock(64, 96, 4, 2, device="cuda")
    x = torch.randn(33, 64, device="cuda", dtype=BF, requires_grad=True)
    note("ExpertBlock with one expert, none, and no tokens")
    one = torch.tensor([False, False, True, False], device="cuda")
    y = block(x, expert_mask=one)
    y.float().sum().backward()
    assert torch.isfinite(x.grad).all() and block.up[2].weight.grad is not None
    assert block.up[0].weight.grad is None
    idx, w = block.route(block.norm(x), one)
    assert bool((idx[:, 0] == 2).all()) and bool((idx[:, 1] == -1).all())
    assert bool((w[:, 0] == 1).all()) and not w[:, 1].any()
    none = torch.zeros(4, dtype=torch.bool, device="cuda")
    assert torch.equal(block(x, expert_mask=none), x)
    empty = torch.empty((0, 64), device="cuda", dtype=BF)
    assert block(empty).shape == (0, 64)
    torch.cuda.synchronize()
