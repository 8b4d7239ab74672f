"""GPU parity of the quantized activation and of its gradient: scales and the values that the
codes stand for within the oracle's bounds, rows and columns alike."""
import numpy as np
import pytest

from oracle import act as oact
from oracle import e4m3
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


def rows_of(rows, width, seed, dt, pad=0, std=1.5):
    g = torch.Generator().manual_seed(seed)
    x = std * torch.randn(rows, width + pad, generator=g)
    x *= torch.exp(2 * torch.randn(rows, 1, generator=g))      # rows of different sizes
    if rows > 2:
        x[1] = 0                                               # a padding row of an expert
    return x.to(DT[dt]).cuda()[:, pad:]


def check_tiles(q, scale, v, err, what):
    """Codes q with scales against the values v (tiles along v's rows)."""
    q, scale = q.view(torch.uint8).cpu().numpy(), host(scale)
    assert_within(scale, oact.scales(v), oact.scale_bound(v, err), what + " scale")
    got = e4m3.decode(q) * np.repeat(scale, 128, axis=1)
    assert_within(got, v, oact.value_bound(v, err, scale), what)


SHAPES = [(128, 128, 0, 128), (256, 384, 0, 200), (128, 1024, 8, 0), (384, 256, 3, 384),
          (128, 2176, 1, 127)]
KINDS = [("relu", False), ("relu", True), ("silu", False), ("silu", True), ("gelu", False),
         ("gelu", True)]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind,gated", KINDS)
def test_forward(lib, kind, gated, dt):
    for rows, cols, pad, valid in SHAPES:
        note(f"act_quantize {kind} gated={gated} {rows}x{cols} valid={valid} pad={pad} {dt}")
        h = rows_of(rows, cols * (2 if gated else 1), rows + cols, dt, pad)
        q, s, qt, st, hq, hs = lib.fp8_act_quantize(h, kind, gated, rows_valid=valid)
        torch.cuda.synchronize()
        hh = host(h)
        hh[valid:] = 0
        a, err = oact.forward(hh, kind, gated)
        check_tiles(q, s, a, err, "q")
        check_tiles(qt, st, a.T, err.T, "q_t")
        check_tiles(hq, hs, hh, 0 * hh, "hq")
        assert (q[valid:] == 0).all() and (hq[valid:] == 0).all() and (qt[:, valid:] == 0).all()
        # the outputs one at a time are the same bits
        only = lib.fp8_act_quantize(h, kind, gated, rows_valid=valid, want_q_t=False,
                                    want_checkpoint=False)
        assert torch.equal(only[0], q) and torch.equal(only[1], s) and only[2:] == (None,) * 4
        only = lib.fp8_act_quantize(h, kind, gated, rows_valid=valid, want_q=False,
                                    want_checkpoint=False)
        assert torch.equal(only[2], qt) and torch.equal(only[3], st)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind,gated", KINDS)
def test_backward(lib, kind, gated, dt):
    for rows, cols, pad, valid in SHAPES:
        note(f"act_quantize_bwd {kind} gated={gated} {rows}x{cols} valid={valid} pad={pad} {dt}")
        h = rows_of(rows, cols * (2 if gated else 1), rows, dt)
        da = rows_of(rows, cols, cols, dt, pad, 0.3)
        _, _, _, _, hq, hs = lib.fp8_act_quantize(h, kind, gated, want_q=False, want_q_t=False)
        q, s, qt, st, dh = lib.fp8_act_quantize_bwd(da, hq, hs, kind, gated, rows_valid=valid,
                                                    want_dh=True)
        torch.cuda.synchronize()
        hh = e4m3.decode(hq.cpu().numpy()) * np.repeat(host(hs), 128, axis=1)
        hda = host(da)
        hda[valid:], hh[valid:] = 0, 0
        want, err = oact.backward(hda, hh, kind, gated)
        half = torch.finfo(DT[dt]).eps / 2
        tiny = torch.finfo(DT[dt]).smallest_normal * half
        biggest = torch.finfo(DT[dt]).max
        fits = np.abs(want) < biggest                    # f16 may overflow to infinity
        assert_within(np.where(fits, host(dh), 0), np.where(fits, want, 0),
                      err + half * (np.abs(want) + err) + tiny, "dh")
        check_tiles(q, s, want, err, "q")
        check_tiles(qt, st, want.T, err.T, "q_t")
        # a gradient of the function itself, by differences in float64, where it is smooth
        if kind != "relu":
            step = 1e-6 * np.maximum(1.0, np.abs(hh))
            for part in ([0] if not gated else [0, 1]):
                d = np.zeros_like(hh)
                d[:, part * cols:(part + 1) * cols] = step[:, part * cols:(part + 1) * cols]
                hi, _ = oact.forward(hh + d, kind, gated)
                lo, _ = oact.forward(hh - d, kind, gated)
                at = slice(part * cols, (part + 1) * cols)
                diff = hda * (hi - lo) / (2 * d[:, at])
                size = np.abs(hda) * (1 + np.abs(hh[:, -cols:]) if gated else 1.0)
                assert (np.abs(diff - want[:, at]) <= 1e-5 * (np.abs(want[:, at]) + size)).all()


@pytest.mark.parametrize("rows", [1, 2, 5, 127, 129, 300])
def test_rows_that_are_no_whole_tile(lib, rows):
    note(f"act_quantize rows={rows}")
    h = rows_of(rows, 512, rows, "bf16", 4)
    room = torch.full((rows + 1, 256), 77, dtype=torch.uint8, device="cuda")
    sroom = torch.full((rows + 1, 2), -1.0, device="cuda")
    q, s, _, _, hq, hs = lib.fp8_act_quantize(h, "silu", True, q=room[:rows], scale=sroom[:rows],
                                              want_q_t=False)
    a, err = oact.forward(host(h), "silu", True)
    check_tiles(q, s, a, err, "q")
    check_tiles(hq, hs, host(h), 0 * host(h), "hq")
    assert (room[rows] == 77).all() and (sroom[rows] == -1).all()
    da = rows_of(rows, 256, rows + 1, "bf16")
    *_, dh = lib.fp8_act_quantize_bwd(da, hq, hs, "silu", True, want_q_t=False, want_dh=True)
    assert dh.shape == (rows, 512) and torch.isfinite(dh).all()
    with pytest.raises(ValueError, match="multiple of 128"):
        lib.fp8_act_quantize(h)


def test_no_rows(lib):
    note("act_quantize without rows")
    h = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    q, s, qt, st, hq, hs = lib.fp8_act_quantize(h, "gelu", False)
    assert q.shape == (0, 256) and qt.shape == (256, 0) and hq.shape == (0, 256)
    out = lib.fp8_act_quantize_bwd(h, hq, hs, "gelu", False, want_dh=True)
    assert out[0].shape == (0, 256) and out[4].shape == (0, 256)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_and_small_values(lib, dt):
    """A tile's largest value takes the code of 448; zeros, subnormal tiles and values up to the
    type's largest stay finite."""
    note(f"act_quantize extremes {dt}")
    h = rows_of(128, 256, 3, dt)
    h[3], h[4], h[5] = 0, 1e-30, -1e-30
    h[6, 7] = torch.finfo(torch.bfloat16).max
    h[7, 9] = -torch.finfo(torch.bfloat16).max
    for kind in ("relu", "silu", "gelu"):
        q, s, qt, st, hq, hs = lib.fp8_act_quantize(h, kind, False)
        for codes, scale in ((q, s), (qt, st), (hq, hs)):
            v = e4m3.decode(codes.cpu().numpy())
            assert np.isfinite(v).all() and torch.isfinite(scale).all(), kind
            top = np.abs(v).reshape(v.shape[0], -1, 128).max(2)
            live = host(scale) > 1e-12 / 448 * 1.01
            assert (top[live] == 448).all()
        out = lib.fp8_act_quantize_bwd(torch.ones_like(h), hq, hs, kind, False, want_dh=True)
        assert torch.isfinite(out[4]).all(), kind


def test_nan_and_infinity(lib):
    note("act_quantize nan")
    h = rows_of(128, 256, 4, "f32")
    clean = lib.fp8_act_quantize(h, "relu", False)
    h[9, 130] = float("nan")
    q, s, qt, st, hq, hs = lib.fp8_act_quantize(h, "relu", False)
    for codes, was, at in ((q, clean[0], (9, 130)), (qt, clean[2], (130, 9)), (hq, clean[4], (9, 130))):
        v, w = e4m3.decode(codes.cpu().numpy()), e4m3.decode(was.cpu().numpy())
        assert np.isnan(v[at]) and np.isnan(v).sum() == 1
        v, w = np.delete(v, at[0], 0), np.delete(w, at[0], 0)
        assert np.array_equal(v, w)                      # other rows are as they were
    h[9, 130] = float("inf")
    q, s, qt, st, hq, hs = lib.fp8_act_quantize(h, "relu", False)
    assert torch.isinf(s[9, 1]) and torch.isinf(st[130, 0]) and torch.isinf(hs[9, 1])
    assert torch.isfinite(s[8]).all() and torch.isfinite(s[9, 0])


def test_streams_and_replays(lib):
    note("act_quantize streams and replays")
    h = rows_of(256, 1024, 1, "bf16")
    da = rows_of(256, 512, 2, "bf16")
    want = lib.fp8_act_quantize(h)
    dwant = lib.fp8_act_quantize_bwd(da, want[4], want[5])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = lib.fp8_act_quantize(h, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    held = h.clone()
    with torch.cuda.graph(g):
        out = lib.fp8_act_quantize(held)
        dout = lib.fp8_act_quantize_bwd(da, out[4], out[5])
    for seed in (1, 5, 1):
        held.copy_(rows_of(256, 1024, seed, "bf16"))
        g.replay()
        torch.cuda.synchronize()
        eager = lib.fp8_act_quantize(held)
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
        deager = lib.fp8_act_quantize_bwd(da, eager[4], eager[5])
        assert all(torch.equal(a, b) for a, b in zip(dout[:4], deager[:4]))
    assert all(torch.equal(a, b) for a, b in zip(dout[:4], dwant[:4]))


def test_large_tensor_against_slices(lib):
    """2.2 G elements of h: offsets past 32 bits."""
    note("act_quantize of 2.2 G elements")
    rows, cols = 38400, 28672
    h = torch.zeros(rows, 2 * cols, dtype=torch.bfloat16, device="cuda")
    at = [0, 128 * 147, rows - 128]
    for i in at:
        h[i:i + 128] = rows_of(128, 2 * cols, i, "bf16")
    q, s, qt, st, hq, hs = lib.fp8_act_quantize(h)
    del h
    da = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    for i in at:
        da[i:i + 128] = rows_of(128, cols, i + 1, "bf16")
    out = lib.fp8_act_quantize_bwd(da, hq, hs)
    for i in at:
        r = slice(i, i + 128)
        part = lib.fp8_act_quantize(rows_of(128, 2 * cols, i, "bf16"))
        assert torch.equal(part[0], q[r]) and torch.equal(part[1], s[r])
        assert torch.equal(part[2], qt[:, r]) and torch.equal(part[3], st[:, i // 128:i // 128 + 1])
        assert torch.equal(part[4], hq[r]) and torch.equal(part[5], hs[r])
        dpart = lib.fp8_act_quantize_bwd(da[r], part[4], part[5])
        assert torch.equal(dpart[0], out[0][r]) and torch.equal(dpart[2], out[2][:, r])
        assert torch.equal(dpart[3], out[3][:, i // 128:i // 128 + 1])
    assert (q[128:256] == 0).all() and (out[0][256:512] == 0).all()


@pytest.mark.parametrize("rows", [300, 384])
def test_many_tiles_are_their_columns_calls(lib, rows):
    """Tiles are independent: 210 of them in one call, and in calls of a few columns each."""
    note(f"act_quantize {rows} rows of 70 tiles")
    g = torch.Generator("cuda").manual_seed(rows)
    cols, part, train = 70 * 128, 5 * 128, rows % 128 == 0
    h = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    da = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16)
    whole = lib.fp8_act_quantize(h, "gelu", False, want_q_t=train, want_checkpoint=True)
    back = lib.fp8_act_quantize_bwd(da, whole[4], whole[5], "gelu", False, want_q=True,
                                    want_q_t=train, want_dh=True)
    for c in range(0, cols, part):
        s, st = slice(c, c + part), slice(c // 128, (c + part) // 128)
        few = lib.fp8_act_quantize(h[:, s], "gelu", False, want_q_t=train, want_checkpoint=True)
        fewb = lib.fp8_act_quantize_bwd(da[:, s], few[4], few[5], "gelu", False, want_q=True,
                                        want_q_t=train, want_dh=True)
        for got, at in ((whole, few), (back, fewb)):
            assert torch.equal(got[0][:, s], at[0]) and torch.equal(got[1][:, st], at[1])
            if train:
                assert torch.equal(got[2][s], at[2]) and torch.equal(got[3][s], at[3])
        assert torch.equal(whole[4][:, s], few[4]) and torch.equal(whole[5][:, st], few[5])
        assert torch.equal(back[4][:, s], fewb[4])
