"""Outputs of the router, activation and grouped products that share memory with an input or with each
other are refused by the C entry points. Made-up addresses; every call here is refused."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

import scaled_fp8_linear_amd as m  # noqa: E402

LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "scaled_fp8_linear_amd", "libfp8lin.so")
pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="passes made-up addresses")
FAR = 1 << 30                   # apart from each other


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        pytest.skip("libfp8lin.so not built (python -m scaled_fp8_linear_amd.build)")
    return m.load()


def refusals(fn, names, sizes, outs, ins, order, **fixed):
    """Call ``fn`` with each output moved onto each other tensor: onto its start, its last bytes, and so
    that the output's own last bytes are on its start. ``sizes``: bytes by name."""
    places = {n: (i + 1) * FAR for i, n in enumerate(names)}

    def call(**moved):
        at = {**places, **moved}
        return fn(*[ctypes.c_void_p(at[a]) if a in at else fixed[a] for a in order])

    for o in outs:
        for other in [n for n in names if n != o and (n in ins or n in outs)]:
            at = places[other]
            for where in (at, at + sizes[other] - 16, at - sizes[o] + 16):
                where -= where % 16
                if where <= at - sizes[o] or where >= at + sizes[other]:
                    continue                     # an alignment of 16 leaves no shared byte
                assert call(**{o: where}) == 4, (o, other, where - at)
                message = m.fp8_last_error()
                assert "shares memory with" in message, (o, other, message)


@pytest.mark.parametrize("gated", [0, 1])
def test_act(lib, gated):
    rows, cols, ld = 256, 128, 1024
    w = 2 * cols if gated else cols
    sizes = {"h": ((rows - 1) * ld + w) * 2, "q": rows * cols, "scale": rows * cols // 32,
             "q_t": rows * cols, "scale_t": rows * cols // 32, "hq": rows * w, "hscale": rows * w // 32}
    outs = ["q", "scale", "q_t", "scale_t", "hq", "hscale"]
    refusals(lib.fp8_act_quantize, ["h"] + outs, sizes, outs, ["h"],
             ["h", "ld", "rows", "valid", "cols", "act", "gated", "dt", *outs, "stream"], ld=ld,
             rows=rows, valid=rows, cols=cols, act=1, gated=gated, dt=0, stream=None)
    sizes = {"da": ((rows - 1) * ld + cols) * 2, "hq": rows * w, "hscale": rows * w // 32,
             "q": rows * w, "scale": rows * w // 32, "q_t": rows * w, "scale_t": rows * w // 32,
             "dh": rows * w * 2}
    outs = ["q", "scale", "q_t", "scale_t", "dh"]
    refusals(lib.fp8_act_quantize_bwd, ["da", "hq", "hscale"] + outs, sizes, outs,
             ["da", "hq", "hscale"],
             ["da", "ld", "hq", "hscale", "rows", "valid", "cols", "act", "gated", "dt", *outs,
              "stream"], ld=ld, rows=rows, valid=rows, cols=cols, act=1, gated=gated, dt=0, stream=None)


def test_route(lib):
    tokens, experts, k, ld = 5000, 24, 3, 40
    ws = lib_workspace(lib, tokens, experts)
    sizes = {"logits": ((tokens - 1) * ld + experts) * 2, "idx": 4 * tokens * k, "w": 4 * tokens * k,
             "lse": 4 * tokens, "counts": 4 * experts, "losses": 8, "ws": ws}
    outs = ["idx", "w", "lse", "counts", "losses", "ws"]
    fixed = dict(ld=ld, tokens=tokens, valid=tokens, experts=experts, k=k, dt=0, norm=1, stream=None)
    refusals(lib.fp8_moe_route, ["logits"] + outs, sizes, outs, ["logits"],
             ["logits", "ld", "tokens", "valid", "experts", "k", "dt", "norm", *outs, "bytes", "stream"],
             bytes=ws, **fixed)
    ins = ["logits", "lse", "idx", "w", "counts", "dw", "dl"]
    sizes.update(dw=4 * tokens * k, dl=8, d=tokens * experts * 2)
    refusals(lib.fp8_moe_route_bwd, ins + ["d"], sizes, ["d"], ins,
             ["logits", "ld", "lse", "idx", "w", "counts", "dw", "dl", "tokens", "valid", "experts", "k",
              "dt", "norm", "d", "stream"], **fixed)


def lib_workspace(lib, tokens, experts):
    out = ctypes.c_int64(0)
    assert lib.fp8_moe_route_workspace(tokens, experts, ctypes.byref(out)) == 0 and out.value > 0
    return out.value


@pytest.mark.parametrize("transposed", [False, True])
def test_grouped(lib, transposed):
    e, rows, n, k = 3, 384, 256, 128
    ldw, sew = (e * k, k) if transposed else (k, n * k)         # experts' rows alternate
    ldsw, ses = (e * k // 128, k // 128) if transposed else (k // 128, n // 128 * (k // 128))
    sizes = {"x": rows * k, "w": e * n * k, "sx": rows * k // 32, "sw": e * n * k // 128 // 32,
             "off": 4 * (e + 1), "cnt": 4 * e, "y": 2 * rows * n}
    ins = ["x", "w", "sx", "sw", "off", "cnt"]
    refusals(lib.fp8_grouped_linear_fwd, ins + ["y"], sizes, ["y"], ins,
             ["x", "w", "ldw", "sew", "sx", "sw", "ldsw", "ses", "off", "cnt", "e", "rows", "n", "k",
              "most", "y", "stream"], ldw=ldw, sew=sew, ldsw=ldsw, ses=ses, e=e, rows=rows, n=n, k=k,
             most=rows, stream=None)
    sizes = {"g": n * rows, "x": k * rows, "sg": n * rows // 32, "sx": k * rows // 32,
             "off": 4 * (e + 1), "cnt": 4 * e, "dw": 2 * e * n * k}
    ins = ["g", "x", "sg", "sx", "off", "cnt"]
    refusals(lib.fp8_grouped_linear_wgrad, ins + ["dw"], sizes, ["dw"], ins,
             ["g", "x", "sg", "sx", "off", "cnt", "e", "rows", "n", "k", "dw", "stream"], e=e, rows=rows,
             n=n, k=k, stream=None)
