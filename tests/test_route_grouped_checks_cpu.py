"""Refusals of the router, activation and grouped product entry points, without a GPU: the C ABI's
host checks (made-up addresses that no check lets through to a kernel; only where no GPU is visible),
the binding's checks of tensors, the modules'. And the oracles' own pins."""
import ctypes
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import scaled_fp8_linear_amd as m  # noqa: E402
from oracle import act as oact  # noqa: E402
from oracle import route  # noqa: E402

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "scaled_fp8_linear_amd", "libfp8lin.so")
bf, f16, f32, i32, u8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8
P = ctypes.c_void_p(64)
Q = ctypes.c_void_p(128)
ODD = ctypes.c_void_p(65)
ODD4 = ctypes.c_void_p(68)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.skip("libfp8lin.so not built (python -m scaled_fp8_linear_amd.build)")
    return m.load()


no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes made-up addresses")


# ---------------------------------------------------------------------- C ABI

@no_gpu
def test_route_argument_checks(lib):
    def f(x=P, ld=64, t=1000, v=1000, e=64, k=8, dt=0, i=P, w=P, lse=P, c=P, lo=P, ws=P, n=1 << 30):
        return lib.fp8_moe_route(x, ld, t, v, e, k, dt, 1, i, w, lse, c, lo, ws, n, None)

    assert f(t=-1, v=0) == 2 and f(ld=63) == 2 and f(e=0, ld=0) == 2 and f(e=513, ld=513) == 2
    assert f(k=0) == 2 and f(k=65) == 2 and f(e=4, k=5) == 2 and f(v=1001) == 2 and f(v=-1) == 2
    assert f(dt=3) == 4 and f(t=1 << 31, v=0, k=1) == 4
    assert f(x=None) == 1 and f(i=None) == 1 and f(w=None) == 1 and f(lse=None) == 1
    assert f(c=None) == 1 and f(lo=None) == 1 and f(ws=None) == 1 and f(n=100) == 2
    assert f(x=ODD) == 3 and f(i=ODD) == 3 and f(w=ODD) == 3 and f(lse=ODD) == 3
    assert f(c=ODD) == 3 and f(lo=ODD) == 3 and f(ws=ODD) == 3 and f(x=ctypes.c_void_p(66), dt=2) == 3
    out = ctypes.c_int64(-1)
    assert lib.fp8_moe_route_workspace(1000, 64, None) == 1
    assert lib.fp8_moe_route_workspace(-1, 64, ctypes.byref(out)) == 2
    assert lib.fp8_moe_route_workspace(1, 513, ctypes.byref(out)) == 2
    assert lib.fp8_moe_route_workspace(1, 8, ctypes.byref(out)) == 0 and out.value == 0
    assert lib.fp8_moe_route_workspace(100000, 64, ctypes.byref(out)) == 0 and out.value > 0


@no_gpu
def test_route_bwd_argument_checks(lib):
    def f(x=P, ld=64, lse=P, i=P, w=P, c=P, dw=P, dl=P, t=100, v=100, e=64, k=8, dt=0, d=Q):
        return lib.fp8_moe_route_bwd(x, ld, lse, i, w, c, dw, dl, t, v, e, k, dt, 1, d, None)

    assert f(t=-1, v=0) == 2 and f(ld=63) == 2 and f(k=65) == 2 and f(v=101) == 2
    assert f(dt=7) == 4 and f(d=P) == 4
    assert f(x=None) == 1 and f(lse=None) == 1 and f(i=None) == 1 and f(w=None) == 1
    assert f(c=None) == 1 and f(d=None) == 1
    assert f(dw=ODD) == 3 and f(dl=ODD) == 3 and f(d=ODD) == 3 and f(lse=ODD) == 3
    assert f(t=0, v=0, x=None, lse=None, i=None, w=None, d=None) == 0


@no_gpu
def test_act_argument_checks(lib):
    def f(h=P, ld=512, r=256, v=256, c=256, act=1, gated=1, dt=0, q=Q, s=Q, qt=Q, st=Q, hq=Q, hs=Q):
        return lib.fp8_act_quantize(h, ld, r, v, c, act, gated, dt, q, s, qt, st, hq, hs, None)

    assert f(r=-1, v=0) == 2 and f(c=0) == 2 and f(c=100) == 2 and f(ld=511) == 2
    assert f(gated=0, ld=255) == 2 and f(v=257) == 2 and f(v=-1) == 2 and f(r=200, v=200) == 2
    assert f(r=1 << 23, v=0) == 4 and f(c=1 << 17, ld=1 << 18) == 4 and f(act=3) == 4 and f(dt=3) == 4
    assert f(h=None) == 1 and f(q=None) == 1 and f(s=None) == 1 and f(st=None) == 1 and f(hs=None) == 1
    assert f(q=ODD4) == 3 and f(qt=ODD4) == 3 and f(hq=ODD4) == 3 and f(s=ODD) == 3 and f(h=ODD) == 3
    assert f(q=None, s=None, qt=None, st=None, hq=None, hs=None) == 0
    assert f(r=0, v=0, h=None) == 0

    def b(da=P, ld=256, hq=P, hs=P, r=256, v=256, c=256, act=1, gated=1, dt=0, q=Q, s=Q, qt=Q, st=Q,
          dh=Q):
        return lib.fp8_act_quantize_bwd(da, ld, hq, hs, r, v, c, act, gated, dt, q, s, qt, st, dh, None)

    assert b(ld=255) == 2 and b(c=64) == 2 and b(v=300) == 2 and b(r=100, v=100) == 2
    assert b(act=-1) == 4 and b(dt=5) == 4 and b(dh=P) == 4 and b(q=P) == 4
    assert b(da=None) == 1 and b(hq=None) == 1 and b(hs=None) == 1 and b(s=None) == 1
    assert b(hq=ODD4) == 3 and b(dh=ODD) == 3 and b(qt=ODD4) == 3
    assert b(q=None, s=None, qt=None, st=None, dh=None) == 0


@no_gpu
@pytest.mark.parametrize("dgrad", [False, True])
def test_grouped_argument_checks(lib, dgrad):
    fn = lib.fp8_grouped_linear_dgrad if dgrad else lib.fp8_grouped_linear_fwd

    def f(x=P, w=P, ldw=256, sew=1 << 16, sx=P, sw=P, ldsw=2, ses=4, off=P, cnt=P, e=4, r=512, n=384,
          k=256, most=512, y=Q):
        a, b = (k, n) if dgrad else (n, k)
        return fn(x, w, ldw, sew, sx, sw, ldsw, ses, off, cnt, e, r, a, b, most, y, None)

    assert f(e=0) == 2 and f(e=513) == 2 and f(r=-1) == 2 and f(n=100) == 2 and f(k=0) == 2
    assert f(ldw=255) == 2 and f(ldw=264) == 2 and f(sew=8) == 2 and f(sew=-16) == 2
    assert f(ldsw=1) == 2 and f(ses=-1) == 2 and f(most=-1) == 2
    assert f(r=1 << 23) == 4 and f(n=1 << 17) == 4 and f(k=1 << 17, ldw=1 << 17) == 4
    assert f(ldw=1 << 23) == 4 and f(ldsw=1 << 23) == 4 and f(sew=1 << 60) == 4 and f(ses=1 << 60) == 4
    assert f(off=None) == 1 and f(cnt=None) == 1 and f(x=None) == 1 and f(w=None) == 1
    assert f(sx=None) == 1 and f(sw=None) == 1 and f(y=None) == 1
    assert f(off=ODD) == 3 and f(x=ODD4) == 3 and f(w=ODD4) == 3 and f(y=ODD4) == 3 and f(sx=ODD) == 3
    assert f(r=0, x=None, y=None) == 0


@no_gpu
def test_grouped_wgrad_argument_checks(lib):
    def f(g=P, x=P, sg=P, sx=P, off=P, cnt=P, e=4, r=512, n=384, k=256, dw=Q):
        return lib.fp8_grouped_linear_wgrad(g, x, sg, sx, off, cnt, e, r, n, k, dw, None)

    assert f(e=0) == 2 and f(r=100) == 2 and f(r=-128) == 2 and f(n=64) == 2 and f(k=1) == 2
    assert f(r=1 << 23) == 4 and f(n=1 << 17) == 4
    assert f(g=None) == 1 and f(x=None) == 1 and f(sg=None) == 1 and f(sx=None) == 1
    assert f(dw=None) == 1 and f(off=None) == 1 and f(cnt=None) == 1
    assert f(g=ODD4) == 3 and f(x=ODD4) == 3 and f(dw=ODD4) == 3 and f(sg=ODD) == 3 and f(cnt=ODD) == 3


# ---------------------------------------------------------------------- tensors

def bad(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


def test_route_tensor_checks(lib):
    x = torch.zeros(5, 8)
    bad("device tensors", m.fp8_moe_route, x, 2)
    bad("2-D", m.fp8_moe_route, torch.zeros(8), 2)
    bad("dtype", m.fp8_moe_route, x.double(), 2)
    bad("topk", m.fp8_moe_route, x, 0)
    bad("contiguous", m.fp8_moe_route, torch.zeros(8, 5).t(), 2)
    bad("tokens_valid", m.fp8_moe_route, x, 2, tokens_valid=6)
    bad("expert_idx has dtype", m.fp8_moe_route, x, 2, expert_idx=torch.zeros(5, 2, dtype=torch.int64))
    bad("weights has shape", m.fp8_moe_route, x, 2, weights=torch.zeros(5, 3))
    bad("losses has shape", m.fp8_moe_route, x, 2, losses=torch.zeros(3))
    idx, w, lse, c = torch.zeros(5, 2, dtype=i32), torch.zeros(5, 2), torch.zeros(5), \
        torch.zeros(8, dtype=i32)
    bad("device tensors", m.fp8_moe_route_bwd, x, lse, idx, w, c)
    bad("lse has shape", m.fp8_moe_route_bwd, x, lse[:4], idx, w, c)
    bad("expert_idx must be 2-D", m.fp8_moe_route_bwd, x, lse, idx.view(-1), w, c)
    bad("counts has shape", m.fp8_moe_route_bwd, x, lse, idx, w, c[:7])
    bad("dweights has shape", m.fp8_moe_route_bwd, x, lse, idx, w, c, dweights=w[:4])
    bad("dlosses has dtype", m.fp8_moe_route_bwd, x, lse, idx, w, c, dlosses=torch.zeros(2).double())
    bad("dlogits has dtype", m.fp8_moe_route_bwd, x, lse, idx, w, c, dlogits=x.half())
    bad("lse is needed", m.fp8_moe_route_bwd, x, None, idx, w, c)


def test_act_tensor_checks(lib):
    h = torch.zeros(128, 512, dtype=bf)
    bad("device tensors", m.fp8_act_quantize, h)
    bad("act must be", m.fp8_act_quantize, h, act="tanh")
    bad("odd width", m.fp8_act_quantize, torch.zeros(128, 257))
    bad("multiple of 128", m.fp8_act_quantize, torch.zeros(128, 200))
    bad("multiple of 128", m.fp8_act_quantize, h[:100])
    bad("rows_valid", m.fp8_act_quantize, h, rows_valid=129)
    bad("both be given", m.fp8_act_quantize, h, q=torch.zeros(128, 256, dtype=u8))
    bad("q has shape", m.fp8_act_quantize, h, q=torch.zeros(128, 512, dtype=u8),
        scale=torch.zeros(128, 2))
    bad("scale_t has shape", m.fp8_act_quantize, h, q_t=torch.zeros(256, 128, dtype=u8),
        scale_t=torch.zeros(256, 2))
    bad("hq has dtype", m.fp8_act_quantize, h, hq=torch.zeros(128, 512), hscale=torch.zeros(128, 4))
    da, hq, hs = h[:, :256], torch.zeros(128, 512, dtype=u8), torch.zeros(128, 4)
    bad("device tensors", m.fp8_act_quantize_bwd, da, hq, hs)
    bad("hq has shape", m.fp8_act_quantize_bwd, da, hq, hs, gated=False)
    bad("hscale has shape", m.fp8_act_quantize_bwd, da, hq, hs[:, :2])
    bad("is needed", m.fp8_act_quantize_bwd, da, None, hs)
    bad("dh has dtype", m.fp8_act_quantize_bwd, da, hq, hs, dh=torch.zeros(128, 512))
    bad("act must be", m.fp8_act_quantize_bwd, da, hq, hs, act=1)


def test_grouped_tensor_checks(lib):
    x, sx = torch.zeros(256, 256, dtype=u8), torch.zeros(256, 2)
    w, sw = torch.zeros(3, 384, 256, dtype=u8), torch.zeros(3, 3, 2)
    off, cnt = torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32)
    for f in (m.fp8_grouped_linear_fwd, m.fp8_grouped_linear_dgrad):
        bad("device tensors", f, x, w, sx, sw, off, cnt)
        bad("device tensors", f, x.view(torch.float8_e4m3fn), w, sx, sw, off, cnt)
        bad("has dtype", f, x.float(), w, sx, sw, off, cnt)
        bad("has shape", f, x, w, sx[:, :1], sw, off, cnt)
        bad("must be 3-D", f, x, w[0], sx, sw, off, cnt)
        bad("has shape", f, x, w[:2], sx, sw, off, cnt)
        bad("has shape", f, x, w, sx, sw[:, :2], off, cnt)
        bad("rows must be contiguous", f, x, w.transpose(1, 2)[:, :, :256].transpose(1, 2)
            .permute(0, 2, 1)[:, :, :256], sx, torch.zeros(3, 2, 2), off, cnt)
        bad("offsets has shape", f, x, w, sx, sw, cnt, cnt)
        bad("counts has dtype", f, x, w, sx, sw, off, cnt.long())
        bad("is needed", f, x, w, None, sw, off, cnt)
        bad("negative", f, x, w, sx, sw, off, cnt, max_rows=-1)
        bad("has dtype", f, x, w, sx, sw, off, cnt, torch.zeros(256, 384))
    g, sg = torch.zeros(384, 256, dtype=u8), torch.zeros(384, 2)
    bad("device tensors", m.fp8_grouped_linear_wgrad, g, x, sg, sx, off, cnt)
    bad("rows of tokens", m.fp8_grouped_linear_wgrad, g, x[:, :128].contiguous(), sg,
        torch.zeros(256, 1), off, cnt)
    bad("dw has shape", m.fp8_grouped_linear_wgrad, g, x, sg, sx, off, cnt,
        torch.zeros(3, 256, 384, dtype=bf))


def test_module_checks(lib):
    bad("topk", m.GroupedExpertBlock, 128, 128, 4, 5)
    bad("multiples of 128", m.GroupedExpertBlock, 100, 128, 4, 2)
    block = m.GroupedExpertBlock(128, 256, 4, 2)
    bad("bfloat16 tokens", block, torch.zeros(3, 128))
    bad("bfloat16 tokens", block, torch.zeros(3, 64, dtype=bf))
    plan = m.ExpertPlan(torch.zeros(3, 2, dtype=i32), torch.zeros(256, dtype=i32),
                        torch.zeros(4, dtype=i32), torch.zeros(5, dtype=i32))
    xs = torch.zeros(256, 128, dtype=bf)
    bad("multiple of 128", m.expert_mlp, xs[:48], block.w_up, block.w_down, plan)
    bad("w_up has shape", m.expert_mlp, xs, block.w_up[:, :256], block.w_down, plan)
    bad("the plan is for", m.expert_mlp, xs, block.w_up[:3], block.w_down[:3], plan)
    bad("bfloat16", m.expert_mlp, xs.float(), block.w_up, block.w_down, plan)
    # 3 tokens to 2 of 4 experts padded to 128 need 512 rows: these were padded to less
    bad("with multiple=128 it has 512", m.expert_mlp, xs, block.w_up, block.w_down, plan)


# ---------------------------------------------------------------------- the oracles

def test_route_oracle_against_differences():
    """The gradient against differences of the loss it is the gradient of."""
    rng = np.random.default_rng(0)
    for normalize in (True, False):
        x = rng.normal(size=(7, 9))
        x[2, 4], x[3] = -np.inf, -np.inf
        idx, w, lse, counts, _, _ = route.forward(x, 3, normalize, valid=6)
        dw, dl = rng.normal(size=(7, 3)), (0.7, 0.3)

        def loss(v):
            _, w2, l2, _, _, p = route.forward(v, 3, normalize, valid=6)
            bal = 9 / (6 * 3) * (counts * p[:6].sum(0)).sum() / 6
            z = (np.where(np.isfinite(l2[:6]), l2[:6], 0) ** 2).sum() / 6
            return (w2 * dw)[:6].sum() + dl[0] * bal + dl[1] * z

        d, _ = route.backward(x, lse, idx, w, counts, dw, dl, normalize, valid=6)
        for t in range(7):
            for e in range(9):
                if not np.isfinite(x[t, e]):
                    assert d[t, e] == 0
                    continue
                hi, lo = x.copy(), x.copy()
                hi[t, e] += 1e-6
                lo[t, e] -= 1e-6
                # differences of order 1e-6 of values of order 1 are good to about 1e-9
                assert abs((loss(hi) - loss(lo)) / 2e-6 - d[t, e]) < 1e-7
        assert (d[6] == 0).all()


def test_route_oracle_by_hand():
    x = np.array([[0.0, np.log(2.0), np.log(2.0), -np.inf]])
    idx, w, lse, counts, losses, p = route.forward(x, 3, False)
    assert idx.tolist() == [[1, 2, 0]] and np.allclose(w, [[0.4, 0.4, 0.2]])
    assert np.isclose(lse[0], np.log(5)) and counts.tolist() == [1, 1, 1, 0]
    # 4 experts, 1 token, 3 choices: 4/3 sum_e counts[e] p[e] = 4/3
    assert np.allclose(losses, [4 / 3, np.log(5) ** 2])
    idx, w, *_ = route.forward(x, 2, True)
    assert idx.tolist() == [[1, 2]] and np.allclose(w, [[0.5, 0.5]])


def test_act_oracle_against_torch_and_differences():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(4, 256)) * 3
    t = torch.from_numpy(x)
    for kind, f in (("silu", torch.nn.functional.silu), ("relu", torch.relu),
                    ("gelu", lambda v: torch.nn.functional.gelu(v, approximate="tanh"))):
        assert np.allclose(oact.act(x, kind), f(t).numpy(), rtol=1e-12, atol=1e-14)
        d = (oact.act(x + 1e-6, kind) - oact.act(x - 1e-6, kind)) / 2e-6
        assert np.abs(d - oact.dact(x, kind)[0]).max() < 1e-8
    g = torch.from_numpy(x).requires_grad_(True)
    da = rng.normal(size=(4, 128))
    (torch.nn.functional.silu(g[:, :128]) * g[:, 128:]).backward(torch.from_numpy(da))
    assert np.allclose(oact.backward(da, x, "silu", True)[0], g.grad.numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(oact.scales(x), np.abs(x.reshape(4, 2, 128)).max(2) / 448)
