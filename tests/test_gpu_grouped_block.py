"""The router, the experts' products and the activation run together: under autograd bit for bit the
direct calls, the experts' MLP and its gradients against float64 with bounds carried through every
step, the whole block trained for a step, captured, masked, and without tokens."""
import numpy as np
import pytest

from oracle import act as oact
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


def host(t):
    return t.detach().cpu().double().numpy()


def setup(lib, tokens, cols, hidden, experts, topk, gated, seed=0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(tokens, experts, generator=g)
    if experts > topk:
        logits[:, experts // 2] = -float("inf")              # an expert without rows
    r = lib.expert_route(logits.cuda(), topk)
    plan = lib.expert_plan(r.expert_idx, experts, 128)
    x = torch.randn(tokens, cols, generator=g).to(BF).cuda()
    width = 2 * hidden if gated else hidden
    up = (torch.randn(experts, width, cols, generator=g) / cols ** 0.5).to(BF).cuda()
    down = (torch.randn(experts, cols, hidden, generator=g) / hidden ** 0.5).to(BF).cuda()
    xs = lib.expert_dispatch(x, plan)
    dys = lib.expert_dispatch(torch.randn(tokens, cols, generator=g).to(BF).cuda(), plan)
    return r, plan, xs, up, down, dys


def test_route_gradients_are_the_direct_calls(lib):
    g = torch.Generator().manual_seed(1)
    for normalize in (True, False):
        x = torch.randn(50, 20, generator=g).to(BF).cuda().requires_grad_(True)
        note(f"expert_route autograd normalize={normalize}")
        r = lib.expert_route(x, 4, normalize=normalize, tokens_valid=47)
        assert not r.expert_idx.requires_grad and not r.counts.requires_grad
        dw = torch.randn(50, 4, generator=g).cuda()
        ((r.weights * dw).sum() + 3 * r.balance_loss - 2 * r.z_loss).backward()
        idx, w, lse, counts, losses = lib.fp8_moe_route(x.detach(), 4, 47, normalize)
        want = lib.fp8_moe_route_bwd(x.detach(), lse, idx, w, counts, dw,
                                     torch.tensor([3.0, -2.0]).cuda(), 47, normalize)
        assert torch.equal(x.grad, want) and torch.equal(r.weights, w)
        x.grad = None
        lib.expert_route(x, 4, normalize=normalize).balance_loss.backward()   # one output alone
        assert torch.isfinite(x.grad).all() and (x.grad != 0).any()


@pytest.mark.parametrize("gated,act", [(True, "silu"), (False, "relu"), (False, "gelu")])
def test_mlp_is_the_direct_calls(lib, gated, act):
    r, plan, xs, up, down, dys = setup(lib, 200, 256, 384, 6, 2, gated)
    for t in (xs, up, down):
        t.requires_grad_(True)
    note(f"expert_mlp autograd {act} gated={gated}")
    ys = lib.expert_mlp(xs, up, down, plan, act, gated)
    ys.backward(dys)
    o, c, B = plan.offsets, plan.counts, (lib.FP8_BLOCK_1x128, lib.FP8_BLOCK_128x128)
    e, w1, k1 = up.shape

    def rows(t):
        q, qt, _, s, st = lib.fp8_quantize_amax(t.detach(), gran=B[0])
        return q, s, qt, st

    def weights(w):
        n, n1, n2 = w.shape
        q, qt, _, s, st = lib.fp8_quantize_amax(w.detach().reshape(n * n1, n2), gran=B[1])
        return (q.view(n, n1, n2), s.view(n, n1 // 128, n2 // 128),
                qt.view(n2, n, n1).transpose(0, 1).contiguous(),
                st.view(n2 // 128, n, n1 // 128).transpose(0, 1).contiguous())

    x_, u_, d_ = rows(xs), weights(up), weights(down)
    h = lib.fp8_grouped_linear_fwd(x_[0], u_[0], x_[1], u_[1], o, c, max_rows=200)
    a = lib.fp8_act_quantize(h, act, gated)
    assert torch.equal(ys, lib.fp8_grouped_linear_fwd(a[0], d_[0], a[1], d_[1], o, c, max_rows=200))
    g_ = rows(dys)
    assert torch.equal(down.grad, lib.fp8_grouped_linear_wgrad(g_[2], a[2], g_[3], a[3], o, c))
    da = lib.fp8_grouped_linear_dgrad(g_[0], d_[2], g_[1], d_[3], o, c, max_rows=200)
    h_ = lib.fp8_act_quantize_bwd(da, a[4], a[5], act, gated)
    assert torch.equal(up.grad, lib.fp8_grouped_linear_wgrad(h_[2], x_[2], h_[3], x_[3], o, c))
    assert torch.equal(xs.grad, lib.fp8_grouped_linear_dgrad(h_[0], u_[2], h_[1], u_[3], o, c,
                                                             max_rows=200))
    # each gradient alone
    grads = [t.grad for t in (xs, up, down)]
    for want, was in zip((xs, up, down), grads):
        for t in (xs, up, down):
            t.requires_grad_(t is want)
            t.grad = None
        lib.expert_mlp(xs, up, down, plan, act, gated).backward(dys)
        assert torch.equal(want.grad, was)
    with torch.no_grad():
        assert torch.equal(lib.expert_mlp(xs, up, down, plan, act, gated), ys)


class Near:
    """A float64 value and how far the computed one may be from it, elementwise."""

    def __init__(self, v, e=None):
        self.v, self.e = v, np.zeros_like(v) if e is None else e

    def __matmul__(self, o):
        return Near(self.v @ o.v, np.abs(self.v) @ o.e + self.e @ np.abs(o.v) + self.e @ o.e)

    def __mul__(self, o):
        return Near(self.v * o.v, np.abs(self.v) * o.e + self.e * np.abs(o.v) + self.e * o.e)

    @property
    def T(self):
        return Near(self.v.T, self.e.T)

    def cols(self, a, b):
        return Near(self.v[:, a:b], self.e[:, a:b])


def coded(n):
    """Quantized in 8 bits, whatever the tiles: half a step of the code, 2^-4 of the value or 2^-10
    of the scale, which is at most the largest magnitude / 448; float32's own errors, below 2^-16
    of both, with it."""
    size = np.abs(n.v) + n.e
    return Near(n.v, n.e + size * (2.0 ** -4 + 2.0 ** -16)
                + size.max(initial=0) / 448 * (2.0 ** -10 + 2.0 ** -16))


def stored(n):
    """A bf16 product of codes: float32 sums, whose error (the oracle's bound for a block of 128 is
    below 2^-9 of the terms' magnitudes; here of the largest sum of magnitudes) and one rounding."""
    return Near(n.v, n.e + (np.abs(n.v) + n.e) * 2.0 ** -8)


def product(a, b):
    p = a @ b
    mag = np.abs(a.v) @ np.abs(b.v) + p.e
    return stored(Near(p.v, p.e + mag * 2.0 ** -9))


def silu(n, derivative=False):
    v = oact.dact(n.v, "silu")[0] if derivative else oact.act(n.v, "silu")
    # silu' lies within 1.1, silu'' within 0.5
    return Near(v, n.e * (0.5 if derivative else 1.1) + np.abs(v) * 2.0 ** -18 + 1e-30)


def test_mlp_against_float64(lib):
    """Every expert's output and gradients within bounds that follow each quantization through the
    chain: x, W and a in 8 bits, h kept in 8 bits for the backward, sums in float32."""
    hidden, cols = 256, 128
    r, plan, xs, up, down, dys = setup(lib, 150, cols, hidden, 4, 2, True, seed=3)
    for t in (xs, up, down):
        t.requires_grad_(True)
    note("expert_mlp against float64")
    ys = lib.expert_mlp(xs, up, down, plan)
    ys.backward(dys)
    torch.cuda.synchronize()
    off, cnt = plan.offsets.tolist(), plan.counts.tolist()
    got = {n: host(t) for n, t in (("ys", ys), ("dx", xs.grad), ("dup", up.grad),
                                   ("ddown", down.grad))}
    hx, hd, hu, hw = host(xs), host(dys), host(up), host(down)
    loose = 0.0
    for e in range(4):
        s = slice(off[e], off[e] + cnt[e])
        x, dy = coded(Near(hx[s])), coded(Near(hd[s]))
        w1, w2 = coded(Near(hu[e])), coded(Near(hw[e]))
        h = product(x, w1.T)
        a = silu(h.cols(0, hidden)) * h.cols(hidden, 2 * hidden)
        y = product(coded(a), w2.T)
        kept = coded(h)
        g, u = kept.cols(0, hidden), kept.cols(hidden, 2 * hidden)
        da = product(dy, w2)
        dg, du = da * u * silu(g, True), da * silu(g)
        dh = coded(Near(np.concatenate([dg.v, du.v], 1), np.concatenate([dg.e, du.e], 1)))
        for name, want, at in (("ys", y, s), ("dx", product(dh, w1), s),
                               ("dup", product(dh.T, x), e), ("ddown", product(dy.T, coded(a)), e)):
            err = np.abs(got[name][at] - want.v)
            assert (err <= want.e + 1e-30).all(), (name, e, (err / (want.e + 1e-30)).max())
            # and far nearer than the worst case on the whole: 8-bit codes of 4 factors are each
            # 2^-4 off at most, so their products' norms are within a quarter
            norm = np.linalg.norm(want.v)
            if norm:
                loose = max(loose, np.linalg.norm(err) / norm)
        if cnt[e] == 0:
            assert (got["dup"][e] == 0).all() and (got["ddown"][e] == 0).all()
    assert loose < 0.25
    live = np.zeros(hx.shape[0], bool)
    for e in range(4):
        live[off[e]:off[e] + cnt[e]] = True
    assert (got["ys"][~live] == 0).all() and (got["dx"][~live] == 0).all()


@pytest.mark.parametrize("gated,act", [(True, "silu"), (False, "relu")])
def test_block(lib, gated, act):
    """Runs and gives every parameter a finite gradient; without a graph the same tokens; masked
    experts get nothing; a mask of all experts leaves the tokens as they are."""
    torch.manual_seed(0)
    block = lib.GroupedExpertBlock(256, 384, 6, 2, device="cuda", act=act, gated=gated)
    x = torch.randn(3, 70, 256, device="cuda", dtype=BF, requires_grad=True)
    note(f"GroupedExpertBlock {act} gated={gated}")
    y, r = block(x)
    (y.float().square().mean() + 0.01 * r.balance_loss + 0.001 * r.z_loss).backward()
    for n, p in [("x", x)] + list(block.named_parameters()):
        assert p.grad is not None and torch.isfinite(p.grad).all() and (p.grad != 0).any(), n
    with torch.no_grad():
        assert torch.equal(block(x)[0], y)
    mask = torch.tensor([True, False, True, False, True, True], device="cuda")
    with torch.no_grad():
        _, r = block(x, mask)
        assert (r.counts[~mask] == 0).all() and r.counts.sum().item() == 2 * 210
        y, r = block(x, torch.zeros(6, dtype=torch.bool, device="cuda"))
        assert torch.equal(y, x) and (r.expert_idx == -1).all() and (r.counts == 0).all()
        y, r = block(x[:, :0])
        assert y.shape == (3, 0, 256) and (r.counts == 0).all()


def test_block_without_tokens_has_gradients(lib):
    note("GroupedExpertBlock without tokens")
    block = lib.GroupedExpertBlock(128, 128, 4, 2, device="cuda")
    y, r = block(torch.empty(0, 128, device="cuda", dtype=BF))
    (y.sum().float() + r.balance_loss).backward()
    assert (block.w_up.grad == 0).all() and (block.w_down.grad == 0).all()


def test_block_in_a_graph(lib):
    """A forward with nothing read back can be captured; every replay is the eager result, also
    for tokens that go elsewhere."""
    torch.manual_seed(1)
    block = lib.GroupedExpertBlock(128, 256, 8, 2, device="cuda")
    x = torch.randn(200, 128, device="cuda", dtype=BF)
    note("GroupedExpertBlock in a graph")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.no_grad(), torch.cuda.stream(s):
        block(x)                                             # library handles are made here
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(g):
        y, r = block(x)
    for seed in (2, 3, 2):
        torch.manual_seed(seed)
        x.copy_(torch.randn(200, 128, device="cuda", dtype=BF) * seed)
        g.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            want, rw = block(x)
        assert torch.equal(y, want) and torch.equal(r.counts, rw.counts)
        assert torch.equal(r.balance_loss, rw.balance_loss)


def test_two_streams_at_once(lib):
    """Two blocks' calls under way at the same time do not share anything."""
    note("two streams")
    torch.manual_seed(2)
    blocks = [lib.GroupedExpertBlock(128, 256, 8, 2, device="cuda") for _ in range(2)]
    xs = [torch.randn(300, 128, device="cuda", dtype=BF) for _ in range(2)]
    with torch.no_grad():
        want = [b(x)[0] for b, x in zip(blocks, xs)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):
            got = []
            for b, x, s in zip(blocks, xs, streams):
                with torch.cuda.stream(s):
                    got.append(b(x)[0])
            torch.cuda.synchronize()
            assert all(torch.equal(a, w) for a, w in zip(got, want))


def test_example_trains(lib):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "expert_block.py")
    spec = importlib.util.spec_from_file_location("expert_block_example", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    note("example, grouped")
    losses = ex.train(tokens=300, cols=128, hidden=256, experts=4, topk=2, steps=3, grouped=True,
                      log=lambda s: None)
    assert len(losses) == 3 and all(np.isfinite(losses))
