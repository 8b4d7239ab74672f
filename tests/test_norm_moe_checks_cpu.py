"""Refusals of the layer norm and expert exchange entry points, without a GPU: the C ABI's
host checks (made-up addresses that no check lets through to a kernel; only where no GPU is
visible) and the binding's checks of tensors. And the oracle's own pins."""
import ctypes
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import scaled_fp8_linear_amd as m  # noqa: E402
from oracle import layernorm as ln  # noqa: E402
from oracle import moe  # noqa: E402

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "scaled_fp8_linear_amd", "libfp8lin.so")
bf, f16, f32, i32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
P = ctypes.c_void_p(64)
ODD = ctypes.c_void_p(65)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.skip("libfp8lin.so not built (python -m scaled_fp8_linear_amd.build)")
    return m.load()


no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes made-up addresses")


# ---------------------------------------------------------------------- C ABI

@no_gpu
def test_layernorm_fwd_argument_checks(lib):
    def f(x=P, ldx=64, g=P, b=P, rows=4, cols=64, dt=0, pdt=0, eps=1e-5, y=ctypes.c_void_p(128),
          mean=P, rstd=P):
        return lib.fp8_layernorm_fwd(x, ldx, g, b, rows, cols, dt, pdt, eps, y, mean, rstd, None)

    assert f(rows=-1) == 2 and f(cols=0) == 2 and f(ldx=63) == 2
    assert f(cols=32769, ldx=40000) == 4 and f(rows=1 << 31) == 4
    assert f(dt=3) == 4 and f(dt=0, pdt=1) == 4 and f(dt=2, pdt=0) == 4
    assert f(eps=-1e-9) == 2 and f(eps=float("nan")) == 2 and f(eps=float("inf")) == 2
    assert f(x=None) == 1 and f(y=None) == 1 and f(y=P) == 4
    assert f(x=ODD) == 3 and f(y=ODD) == 3 and f(mean=ODD) == 3 and f(rstd=ODD) == 3
    assert f(g=ODD) == 3 and f(b=ctypes.c_void_p(66), pdt=2) == 3
    assert f(x=ctypes.c_void_p(66), dt=2, pdt=2) == 3
    assert f(rows=1 << 30, ldx=1 << 40) == 2
    assert f(rows=0, x=None, y=None) == 0                    # nothing to do


@no_gpu
def test_layernorm_bwd_argument_checks(lib):
    q = ctypes.c_void_p(128)

    def f(dy=P, lddy=64, x=P, ldx=64, mean=P, rstd=P, g=P, rows=4000, cols=64, dt=0, pdt=0, dx=q,
          dg=q, db=q, ws=q, n=1 << 30):
        return lib.fp8_layernorm_bwd(dy, lddy, x, ldx, mean, rstd, g, rows, cols, dt, pdt, dx, dg,
                                     db, ws, n, None)

    assert f(rows=-1) == 2 and f(cols=0) == 2 and f(cols=32769, ldx=1 << 20, lddy=1 << 20) == 4
    assert f(lddy=63) == 2 and f(ldx=63) == 2
    assert f(dy=None) == 1 and f(x=None) == 1 and f(mean=None) == 1 and f(rstd=None) == 1
    assert f(ws=None) == 1 and f(n=8) == 2 and f(ws=ctypes.c_void_p(130)) == 3
    assert f(dx=P) == 4 and f(dt=7) == 4 and f(pdt=1) == 4
    assert f(dx=ODD) == 3 and f(dg=ODD) == 3 and f(db=ODD) == 3 and f(g=ODD) == 3
    assert f(dx=None, dg=None, db=None) == 0
    assert f(rows=0, dg=None, db=None) == 0
    out = ctypes.c_int64(-1)
    assert lib.fp8_layernorm_bwd_workspace(10, 10, None) == 1
    assert lib.fp8_layernorm_bwd_workspace(10, 0, ctypes.byref(out)) == 2
    assert lib.fp8_layernorm_bwd_workspace(1, 10, ctypes.byref(out)) == 0 and out.value == 0


@no_gpu
def test_sort_argument_checks(lib):
    def f(idx=P, nb=8, tokens=4, topk=2, experts=8, multiple=16, slot=P, source=P, counts=P,
          offsets=P, ws=None, n=0):
        return lib.fp8_moe_sort(idx, nb, tokens, topk, experts, multiple, slot, source, counts,
                                offsets, ws, n, None)

    assert f(tokens=-1) == 2 and f(topk=0) == 2 and f(topk=65) == 2
    assert f(experts=0) == 2 and f(experts=513) == 2 and f(multiple=0) == 2
    assert f(nb=2) == 4 and f(tokens=1 << 30, topk=2) == 4 and f(multiple=1 << 30) == 4
    assert f(idx=None) == 1 and f(slot=None) == 1 and f(source=None) == 1
    assert f(counts=None) == 1 and f(offsets=None) == 1
    assert f(idx=ctypes.c_void_p(68)) == 3 and f(slot=ctypes.c_void_p(66)) == 3
    assert f(tokens=1 << 20) == 1                            # needs a workspace
    assert f(tokens=1 << 20, ws=P, n=16) == 2
    out = ctypes.c_int64(-1)
    assert lib.fp8_moe_rows(4, 2, 8, 16, None) == 1
    assert lib.fp8_moe_sort_workspace(4, 2, 8, None) == 1
    assert lib.fp8_moe_sort_workspace(4, 2, 0, ctypes.byref(out)) == 2


@no_gpu
def test_exchange_argument_checks(lib):
    q = ctypes.c_void_p(128)

    def d(x=P, ldx=64, slot=P, source=P, tokens=4, topk=2, rows=32, cols=64, dt=0, xs=q):
        return lib.fp8_moe_dispatch(x, ldx, slot, source, tokens, topk, rows, cols, dt, xs, None)

    def c(ys=P, ld=64, slot=P, w=P, tokens=4, topk=2, rows=32, cols=64, dt=0, y=q):
        return lib.fp8_moe_combine(ys, ld, slot, w, tokens, topk, rows, cols, dt, y, None)

    def g(ys=P, ld=64, slot=P, tokens=4, topk=2, rows=32, cols=64, dt=0, dx=q):
        return lib.fp8_moe_dispatch_bwd(ys, ld, slot, tokens, topk, rows, cols, dt, dx, None)

    def b(dy=P, lddy=64, ys=P, ldys=64, slot=P, source=P, w=P, tokens=4, topk=2, rows=32, cols=64,
          dt=0, dys=q, dw=q):
        return lib.fp8_moe_combine_bwd(dy, lddy, ys, ldys, slot, source, w, tokens, topk, rows,
                                       cols, dt, dys, dw, None)

    for f in (d, c, g, b):
        assert f(tokens=-1) == 2 and f(topk=0) == 2 and f(topk=65) == 2 and f(rows=-1) == 2
        assert f(cols=-1) == 2 and f(dt=3) == 4 and f(dt=-1) == 4
        assert f(slot=None) == 1 and f(slot=ctypes.c_void_p(66)) == 3
        assert f(tokens=1 << 24) == 4 and f(rows=1 << 24) == 4
        assert "2^24" in lib.fp8_last_error().decode()
        assert f(tokens=1 << 30, topk=2) == 4
    for f in (d, b):
        assert f(source=None) == 1 and f(source=ctypes.c_void_p(66)) == 3
    for f in (c, b):
        assert f(w=None) == 1 and f(w=ctypes.c_void_p(66)) == 3
    assert d(x=None) == 1 and d(xs=None) == 1 and d(ldx=63) == 2 and d(xs=P) == 4
    assert d(x=ODD) == 3 and d(xs=ODD) == 3 and d(x=ctypes.c_void_p(66), dt=2) == 3
    assert c(ys=None) == 1 and c(y=None) == 1 and c(ld=63) == 2 and c(y=P) == 4
    assert g(ys=None) == 1 and g(dx=None) == 1 and g(ld=63) == 2 and g(dx=P) == 4
    assert b(dy=None) == 1 and b(ys=None) == 1 and b(dys=None) == 1 and b(dw=None) == 1
    assert b(lddy=63) == 2 and b(ldys=63) == 2 and b(dys=P) == 4 and b(dw=ctypes.c_void_p(66)) == 3
    assert d(rows=0, tokens=0) == 0 and c(tokens=0) == 0 and g(tokens=0, cols=0) == 0


def test_moe_rows_against_the_worst_routing(lib):
    for tokens in (0, 1, 3, 17, 64):
        for topk in (1, 2, 5):
            for experts in (1, 4, 11):
                for multiple in (1, 3, 16):
                    got = m.fp8_moe_rows(tokens, topk, experts, multiple)
                    assert got == moe.rows_of(tokens, topk, experts, multiple)


# ---------------------------------------------------------------------- the binding

def _raises(fn, *words):
    with pytest.raises(ValueError) as e:
        fn()
    for w in words:
        assert w in str(e.value), (w, str(e.value))


def test_layernorm_buffers(lib):
    x, g, s = torch.zeros((6, 40), dtype=bf), torch.ones(40, dtype=bf), torch.zeros(6)
    _raises(lambda: m.fp8_layernorm_fwd(x[0]), "2-D")
    _raises(lambda: m.fp8_layernorm_fwd(x.double()), "dtype")
    _raises(lambda: m.fp8_layernorm_fwd(x.t()), "contiguous")
    _raises(lambda: m.fp8_layernorm_fwd(x[:1].expand(6, 40)), "overlap")
    _raises(lambda: m.fp8_layernorm_fwd(x, g[:39]), "gamma")
    _raises(lambda: m.fp8_layernorm_fwd(x, g.to(f16)), "gamma")
    _raises(lambda: m.fp8_layernorm_fwd(x, g, g.float()), "beta")
    _raises(lambda: m.fp8_layernorm_fwd(x, g, g, y=x.float()), "y ")
    _raises(lambda: m.fp8_layernorm_fwd(x, g, g, mean=s[:5]), "mean")
    _raises(lambda: m.fp8_layernorm_fwd(x, g, g, rstd=s.to(bf)), "rstd")
    _raises(lambda: m.fp8_layernorm_fwd(x, g, g), "device")
    _raises(lambda: m.fp8_layernorm_bwd(x[:5], x, s, s, g), "dy")
    _raises(lambda: m.fp8_layernorm_bwd(x.float(), x, s, s, g), "dy")
    _raises(lambda: m.fp8_layernorm_bwd(x, x, s, None, g), "rstd")
    _raises(lambda: m.fp8_layernorm_bwd(x, x, s[:2], s, g), "mean")
    _raises(lambda: m.fp8_layernorm_bwd(x, x, s, s, g, dgamma=g.float()), "dgamma")
    _raises(lambda: m.fp8_layernorm_bwd(x, x, s, s, g, dx=x[:, :39]), "dx")
    _raises(lambda: m.fp8_layernorm_bwd(x, x, s, s, param_dtype=f16), "param_dtype")
    _raises(lambda: m.fp8_layernorm_bwd(x, x, s, s, g), "device")


def test_exchange_buffers(lib):
    idx = torch.zeros((6, 2), dtype=torch.int64)
    slot, source = torch.zeros((6, 2), dtype=i32), torch.zeros(42, dtype=i32)
    x, ys, w = torch.zeros((6, 40), dtype=bf), torch.zeros((42, 40), dtype=bf), torch.zeros((6, 2))
    assert m.fp8_moe_rows(6, 2, 2, 16) == 32
    _raises(lambda: m.fp8_moe_sort(idx[0], 2), "2-D")
    _raises(lambda: m.fp8_moe_sort(idx.float(), 2), "expert_idx")
    _raises(lambda: m.fp8_moe_sort(idx.t(), 2), "contiguous")
    _raises(lambda: m.fp8_moe_sort(idx, 2, slot=slot[:5]), "slot")
    _raises(lambda: m.fp8_moe_sort(idx, 2, source=source), "source")
    _raises(lambda: m.fp8_moe_sort(idx, 2, counts=source[:3]), "counts")
    _raises(lambda: m.fp8_moe_sort(idx, 2, offsets=source[:2]), "offsets")
    _raises(lambda: m.fp8_moe_sort(idx, 2), "device")
    with pytest.raises(m.Fp8Error):
        m.fp8_moe_sort(idx, 0)
    _raises(lambda: m.fp8_moe_dispatch(x[:5], slot, source), "tokens")
    _raises(lambda: m.fp8_moe_dispatch(x, slot.long(), source), "slot")
    _raises(lambda: m.fp8_moe_dispatch(x, slot[0], source), "2-D")
    _raises(lambda: m.fp8_moe_dispatch(x, slot, source[None]), "1-D")
    _raises(lambda: m.fp8_moe_dispatch(x, slot, source.long()), "source")
    _raises(lambda: m.fp8_moe_dispatch(x, slot, source, xs=ys[:41]), "xs")
    _raises(lambda: m.fp8_moe_dispatch(x, slot, source), "device")
    _raises(lambda: m.fp8_moe_dispatch_bwd(ys, slot, dx=x.float()), "dx")
    _raises(lambda: m.fp8_moe_dispatch_bwd(ys, slot), "device")
    _raises(lambda: m.fp8_moe_combine(ys, slot, w.to(bf)), "weights")
    _raises(lambda: m.fp8_moe_combine(ys, slot, w[:, :1]), "weights")
    _raises(lambda: m.fp8_moe_combine(ys, slot, w, y=x[:, :8]), "y ")
    _raises(lambda: m.fp8_moe_combine(ys, slot, w), "device")
    _raises(lambda: m.fp8_moe_combine_bwd(x, ys[:41], slot, source, w), "ys")
    _raises(lambda: m.fp8_moe_combine_bwd(x[:5], ys, slot, source, w), "dy")
    _raises(lambda: m.fp8_moe_combine_bwd(x, ys, slot, source, w, dys=x), "dys")
    _raises(lambda: m.fp8_moe_combine_bwd(x, ys, slot, source, w, dw=w.to(bf)), "dw")
    _raises(lambda: m.fp8_moe_combine_bwd(x, ys, slot, source, w), "device")


# ---------------------------------------------------------------------- the oracle

def test_oracle_layernorm_against_torch():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(7, 33, generator=g, dtype=torch.float64, requires_grad=True)
    gamma = torch.randn(33, generator=g, dtype=torch.float64, requires_grad=True)
    beta = torch.randn(33, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(7, 33, generator=g, dtype=torch.float64)
    y = torch.nn.functional.layer_norm(x, (33,), gamma, beta, eps=1e-5)
    y.backward(dy)
    n = [t.detach().numpy() for t in (x, gamma, beta, dy)]
    wy, mean, rstd = ln.forward(n[0], n[1], n[2], 1e-5)
    wx, wg, wb = ln.backward(n[3], n[0], mean, rstd, n[1])
    for a, b in ((y.detach(), wy), (x.grad, wx), (gamma.grad, wg), (beta.grad, wb)):
        assert np.allclose(a.numpy(), b, rtol=1e-11, atol=1e-12)


def test_oracle_bounds_hold_for_float32_and_catch_mistakes():
    """numpy's float32 forms stay inside the bounds; a missing mean term, a variance over
    cols - 1 and a dropped row do not."""
    rng = np.random.default_rng(2)
    half = 2.0 ** -24
    x = (rng.standard_normal((9, 700)) + 0.5).astype(np.float32)
    dy = rng.standard_normal((9, 700)).astype(np.float32)
    gamma = (1 + 0.1 * rng.standard_normal(700)).astype(np.float32)
    beta = rng.standard_normal(700).astype(np.float32)
    want = ln.forward(x, gamma, beta, 1e-5)
    bound = ln.forward_bounds(x, gamma, beta, 1e-5, half)
    mean = x.mean(1, dtype=np.float32)
    d = x - mean[:, None]
    rstd = (1 / np.sqrt((d * d).mean(1) + np.float32(1e-5))).astype(np.float32)
    y = d * rstd[:, None] * gamma + beta
    for got, w, b in zip((y, mean, rstd), want, bound):
        assert np.all(np.abs(got - w) <= b)
    wrong = 1 / np.sqrt(d.var(1, ddof=1) + 1e-5)
    assert np.any(np.abs(wrong - want[2]) > bound[2])
    wx, wg, wb = ln.backward(dy, x, mean, rstd, gamma)
    bx, bg, bb = ln.backward_bounds(dy, x, mean, rstd, gamma, half, half)
    xh, g = d * rstd[:, None], dy * gamma
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    assert np.all(np.abs(dx - wx) <= bx)
    assert np.all(np.abs((dy * xh).sum(0) - wg) <= bg) and np.all(np.abs(dy.sum(0) - wb) <= bb)
    assert np.any(np.abs(rstd[:, None] * (g - xh * (g * xh).mean(1, keepdims=True)) - wx) > bx)
    assert np.any(np.abs(dy[1:].sum(0) - wb) > bb)


def test_oracle_moe():
    idx = np.array([[2, 0], [0, -1], [5, 2], [2, 2]])
    slot, source, counts, offsets = moe.sort(idx, 4, 4, 16)
    assert counts.tolist() == [2, 0, 4, 0] and offsets.tolist() == [0, 4, 4, 8, 8]
    assert slot.tolist() == [[4, 0], [1, -1], [-1, 5], [6, 7]]
    assert source.tolist() == [1, 2, -1, -1, 0, 5, 6, 7] + [-1] * 8
    x = np.arange(8.0).reshape(4, 2)
    xs = moe.dispatch(x, slot, 16)
    assert xs[7].tolist() == x[3].tolist() and not xs[2:4].any() and not xs[8:].any()
    w = np.full((4, 2), 0.5)
    y, _ = moe.combine(xs, slot, w)
    assert np.allclose(y, x * np.array([1, 0.5, 0.5, 1])[:, None])
    dys, dw, _ = moe.combine_bwd(x, xs, slot, w, 16)
    assert np.allclose(dys[5], 0.5 * x[2]) and dw[1, 1] == 0 and np.isclose(dw[3, 0], (x[3] ** 2).sum())


# ---------------------------------------------------------------------- the native binding

def test_binding_refuses_what_is_no_tensor(lib):
    x, s = torch.zeros((4, 8)), torch.zeros(4)
    slot = torch.zeros((4, 1), dtype=i32)
    _raises(lambda: m.fp8_layernorm_fwd([1.0, 2.0]), "x must be a tensor")
    _raises(lambda: m.fp8_layernorm_fwd(None), "x is needed")
    _raises(lambda: m.fp8_layernorm_bwd(None, x, s, s), "dy is needed")
    _raises(lambda: m.fp8_moe_sort(None, 4), "expert_idx is needed")
    _raises(lambda: m.fp8_moe_dispatch(x, slot, None), "source is needed")
    _raises(lambda: m.fp8_moe_combine(x, slot, None), "weights is needed")
    _raises(lambda: m.fp8_moe_combine_bwd(x, x, slot, torch.zeros(4, dtype=i32), None),
            "weights is needed")
    _raises(lambda: m.fp8_layernorm_fwd(x, 3), "gamma must be a tensor")
    _raises(lambda: m.fp8_moe_sort(slot, 1 << 40), "32 bits")
    with pytest.raises(TypeError):
        m.fp8_moe_sort(slot, "four")
    with pytest.raises(TypeError):
        m.fp8_layernorm_fwd(x, eps="small")


def test_expert_block_argument_checks():
    for topk in (0, 5):
        with pytest.raises(ValueError):
            m.ExpertBlock(16, 32, 4, topk)
    block = m.ExpertBlock(16, 32, 4, 2)
    _raises(lambda: block(torch.zeros((3, 16))), "bfloat16")
    _raises(lambda: block(torch.zeros((3, 15), dtype=bf)), "width 16")
