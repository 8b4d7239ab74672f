"""GPU parity of the router: choices and counts equal to the oracle's, weights, losses and the
gradient within its float32 bounds."""
import numpy as np
import pytest

from oracle import route
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


def make(seed, tokens, experts, dt, kind="any", pad=0):
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn(tokens, experts + pad, generator=g)
    if kind == "ties":                                # few different values, both zeros
        x = (x.round() * 0.5) * torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0)
    if kind == "masked":
        x[torch.rand(x.shape, generator=g) < 0.4] = -float("inf")
        x[::3, :] = -float("inf")                     # rows without any expert
        x[1::3, pad:pad + 1] = 0.25
    if kind == "lowest":
        x[torch.rand(x.shape, generator=g) < 0.4] = torch.finfo(DT[dt]).min
        x[1::3, :] = torch.finfo(DT[dt]).min
    return x.to(DT[dt]).cuda()[:, pad:]


def check(lib, x, topk, normalize, valid=None, seed=0, losses=True):
    tokens, experts = x.shape
    got = lib.fp8_moe_route(x, topk, tokens_valid=valid, normalize=normalize)
    torch.cuda.synchronize()
    idx, w, lse, counts, loss, _ = route.forward(host(x), topk, normalize, valid)
    assert np.array_equal(got[0].cpu().numpy(), idx), "expert_idx"
    assert np.array_equal(got[3].cpu().numpy(), counts), "counts"
    bw, bl, bloss = route.forward_bounds(host(x), w, lse, loss)
    assert_within(host(got[1]), w, bw, "weights")
    g = host(got[2])
    gone = np.isneginf(lse)
    assert np.array_equal(np.isneginf(g), gone)
    assert_within(np.where(gone, 0, g), np.where(gone, 0, lse), np.broadcast_to(bl, lse.shape), "lse")
    if losses:
        assert_within(host(got[4]), loss, bloss, "losses")
    # the gradient, from what the kernel's forward gave
    gen = torch.Generator().manual_seed(seed)
    dw = torch.randn(tokens, topk, generator=gen)
    dw[torch.from_numpy(idx) < 0] = float("nan")      # not used
    dw = dw.cuda()
    dl = torch.tensor([0.7, 0.3 if losses else 0.0]).cuda()
    args = [host(x), g, idx, host(got[1]), counts]
    dt = x.dtype
    half, tiny = torch.finfo(dt).eps / 2, torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
    for a, b in ((dw, dl), (None, dl), (dw, None), (None, None)):
        d = lib.fp8_moe_route_bwd(x, got[2], got[0], got[1], got[3], a, b, valid, normalize)
        torch.cuda.synchronize()
        want, mag = route.backward(*args, None if a is None else host(a),
                                   None if b is None else host(b), normalize, valid)
        assert_within(host(d), want, route.backward_bound(host(x), g, want, mag, half, tiny), "dlogits")
    return got


SHAPES = [(1, 1, 1, 0), (1, 8, 2, 0), (3, 8, 8, 0), (40, 7, 3, 2), (65, 16, 16, 0), (130, 20, 4, 1),
          (300, 32, 5, 0), (77, 60, 3, 5), (500, 64, 8, 0), (33, 64, 64, 0), (50, 100, 40, 3),
          (64, 128, 64, 0), (90, 200, 10, 1), (257, 256, 8, 0), (31, 300, 64, 7), (20, 512, 10, 0),
          (2, 511, 1, 0)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,experts,topk,pad", SHAPES)
def test_route(lib, tokens, experts, topk, pad, dt):
    for kind in ("any", "ties", "masked"):
        note(f"route tokens={tokens} experts={experts} topk={topk} pad={pad} {dt} {kind}")
        x = make(tokens + experts, tokens, experts, dt, kind, pad)
        check(lib, x, topk, True)
        check(lib, x, topk, False, valid=max(0, tokens - 3))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_route_lowest_values(lib, dt):
    """A mask of the type's lowest value is a number: chosen when nothing else is left."""
    note(f"route lowest {dt}")
    x = make(5, 40, 12, dt, "lowest")
    idx, w, *_ = check(lib, x, 9, True, losses=dt == "f16")
    assert (idx >= 0).all() and torch.isfinite(w).all()


def test_route_no_tokens(lib):
    note("route without tokens")
    x = torch.empty(0, 8, device="cuda")
    idx, w, lse, counts, losses = lib.fp8_moe_route(x, 2)
    assert idx.shape == (0, 2) and counts.tolist() == [0] * 8 and losses.tolist() == [0, 0]
    x = torch.full((5, 8), float("nan"), device="cuda")
    idx, w, lse, counts, losses = lib.fp8_moe_route(x, 2, tokens_valid=0)
    assert (idx == -1).all() and (w == 0).all() and losses.tolist() == [0, 0]
    d = lib.fp8_moe_route_bwd(x, lse, idx, w, counts, w, losses, tokens_valid=0)
    assert (d == 0).all()
    assert lib.fp8_moe_route_bwd(x[:0], lse[:0], idx[:0], w[:0], counts).shape == (0, 8)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_route_nan_and_infinity(lib, dt):
    """NaN ranks first and stays in its row."""
    note(f"route nan {dt}")
    x = torch.zeros(6, 70, dtype=DT[dt], device="cuda")
    x[1, 33] = float("nan")
    x[2, 5] = -float("nan")
    x[3, 60] = float("inf")
    idx, w, lse, counts, losses = lib.fp8_moe_route(x, 3)
    assert idx[1].tolist() == [33, 0, 1] and idx[2].tolist() == [5, 0, 1]
    assert idx[3].tolist() == [60, 0, 1] and idx[0].tolist() == [0, 1, 2]
    assert torch.isnan(w[1:4, 0]).all() and torch.isfinite(w[[0, 4, 5]]).all()
    assert torch.isfinite(lse[[0, 4, 5]]).all() and torch.isnan(losses).all()
    assert counts.sum().item() == 18


@pytest.mark.parametrize("tokens,experts,topk,dt", [(40000, 64, 8, "bf16"), (9000, 256, 8, "f32"),
                                                    (70000, 8, 2, "f16"), (5000, 500, 4, "bf16")])
def test_route_many_tokens(lib, tokens, experts, topk, dt):
    """Several workgroups and steps: against torch in float64, and the same bits every time."""
    note(f"route many tokens={tokens} experts={experts} topk={topk} {dt}")
    x = make(1, tokens, experts, dt)
    got = lib.fp8_moe_route(x, topk)
    again = lib.fp8_moe_route(x, topk)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    v, i = torch.sort(x.double(), dim=1, descending=True, stable=True)
    assert torch.equal(got[0].long(), i[:, :topk])
    counts = torch.bincount(i[:, :topk].reshape(-1), minlength=experts)
    assert torch.equal(got[3].long(), counts)
    p = torch.softmax(x.double(), 1)
    lse = torch.logsumexp(x.double(), 1)
    w = torch.softmax(v[:, :topk], 1)
    loss = torch.stack([experts / (tokens * topk) * (counts * p.mean(0)).sum(), lse.square().mean()])
    bw, bl, bloss = route.forward_bounds(host(x), host(w), host(lse), host(loss))
    assert_within(host(got[1]), host(w), bw, "weights")
    assert_within(host(got[2]), host(lse), np.broadcast_to(bl, lse.shape), "lse")
    assert_within(host(got[4]), host(loss), bloss, "losses")
    sl = slice(tokens - 50, tokens)
    d = lib.fp8_moe_route_bwd(x, got[2], got[0], got[1], got[3], got[1], loss.float())
    want, mag = route.backward(host(x)[sl], host(got[2])[sl], host(got[0])[sl].astype(int),
                               host(got[1])[sl], host(counts) * (50 / tokens) ** 2, host(got[1])[sl],
                               host(loss.float()) * [1, 50 / tokens])
    half = torch.finfo(x.dtype).eps / 2
    tiny = torch.finfo(x.dtype).smallest_normal * half
    assert_within(host(d)[sl], want, route.backward_bound(host(x)[sl], host(got[2])[sl], want, mag,
                                                          half, tiny), "dlogits")


def test_route_streams_and_replays(lib):
    """On another stream, with buffers of the caller's that hold something else, and captured."""
    note("route streams and replays")
    x = make(3, 700, 64, "bf16")
    want = lib.fp8_moe_route(x, 8)
    dwant = lib.fp8_moe_route_bwd(x, want[2], want[0], want[1], want[3], want[1], want[4])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = torch.full((lib.fp8_moe_route_workspace(700, 64),), 255, dtype=torch.uint8, device="cuda")
    out = [torch.full_like(t, 77) for t in want]
    torch.cuda.synchronize()
    lib.fp8_moe_route(x, 8, expert_idx=out[0], weights=out[1], lse=out[2], counts=out[3],
                      losses=out[4], workspace=ws, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    g = torch.cuda.CUDAGraph()
    held = x.clone()
    with torch.cuda.graph(g):
        got = lib.fp8_moe_route(held, 8)
        d = lib.fp8_moe_route_bwd(held, got[2], got[0], got[1], got[3], got[1], got[4])
    for seed in (3, 4, 3):
        y = make(seed, 700, 64, "bf16")
        held.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        eager = lib.fp8_moe_route(y, 8)
        assert all(torch.equal(a, b) for a, b in zip(got, eager))
        assert torch.equal(d, lib.fp8_moe_route_bwd(y, eager[2], eager[0], eager[1], eager[3],
                                                    eager[1], eager[4]))
    assert torch.equal(d, dwant)
