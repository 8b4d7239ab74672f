"""ctypes binding of ``libfp8lin.so``: argument marshalling only.

Each function here has the name of the C entry point it calls and passes
device pointers, sizes and the current HIP stream through. Every step of the
computation runs in the library's kernels; PyTorch only provides device
memory (outputs the caller did not pass are allocated with ``torch.empty``)
and the stream. If the library is missing this module raises: there is no
fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8lin.so")

FP8_OK, FP8_ERR_NULL, FP8_ERR_SHAPE, FP8_ERR_ALIGN, FP8_ERR_UNSUPPORTED, FP8_ERR_HIP = range(6)
FP8_TENSORWISE, FP8_BLOCK_1x128, FP8_BLOCK_128x128 = 0, 1, 2
FP8_SCALE_FROM_AMAX, FP8_SCALE_RECORD, FP8_SCALE_REFRESH = 0, 1, 2
FP8_AMAX_ACCUMULATE = 0x100     # flag for fp8_quantize_amax (tensorwise)
FP8_SCALE_CLEAR_AMAX = 0x100    # flag for fp8_scale_update (FROM_AMAX, RECORD)
FP8_E5M2 = 0x200                # flag: E5M2 codes (quantize), 57344 as format max (scale update)
FP8_A_E5M2 = 0x200              # flag for the GEMMs: the first operand holds E5M2 codes

EXPORTS = ("fp8_quantize_amax", "fp8_scale_update", "fp8_linear_fwd", "fp8_linear_dgrad",
           "fp8_linear_wgrad", "fp8_pad_tokens", "fp8_last_error", "fp8_version",
           "fp8_linear_fwd_bias", "fp8_bias_grad", "fp8_align_multiple", "fp8_pad_varlen",
           "fp8_unpad_varlen", "fp8_linear_fwd_current",
           "fp8_layernorm_fwd", "fp8_layernorm_bwd_workspace", "fp8_layernorm_bwd",
           "fp8_moe_rows", "fp8_moe_sort_workspace", "fp8_moe_sort", "fp8_moe_dispatch",
           "fp8_moe_dispatch_bwd", "fp8_moe_combine", "fp8_moe_combine_bwd")
FP8_DT_BF16, FP8_DT_F16, FP8_DT_F32 = 0, 1, 2
FP8_LAYOUT_THD, FP8_LAYOUT_BSHD = 0, 1


class Fp8Error(RuntimeError):
    """An fp8lin entry point returned an error status."""

    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed (status {status}): {msg}")
        self.status = status


_lib = None

_i64, _i32, _int, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_void_p


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library once; raise if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m scaled_fp8_linear_amd.build` "
                           "(the HIP library is required; there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    lib.fp8_quantize_amax.argtypes = [_vp, _i64, _i64, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    lib.fp8_scale_update.argtypes = [_int, _vp, _vp, _i32, _i32, _vp, _vp, _vp]
    lib.fp8_linear_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _vp]
    lib.fp8_linear_fwd_bias.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                        _int, _vp]
    lib.fp8_bias_grad.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp]
    lib.fp8_linear_fwd_current.argtypes = [_vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]
    lib.fp8_linear_dgrad.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _vp]
    lib.fp8_linear_wgrad.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp]
    lib.fp8_pad_tokens.argtypes = [_vp, _i64, _i64, _i32, _vp, ctypes.POINTER(_i64), _vp]
    _p64, _p32 = ctypes.POINTER(_i64), ctypes.POINTER(_i32)
    lib.fp8_align_multiple.argtypes = [_int, _i64, _i32, _i32, _i32, _p32, _p32]
    lib.fp8_pad_varlen.argtypes = [_vp, _p64, _i32, _i64, _i32, _i32, _vp, _p64, _p64, _vp]
    lib.fp8_unpad_varlen.argtypes = [_vp, _p64, _p64, _i32, _i64, _vp, _vp]
    lib.fp8_layernorm_fwd.argtypes = [_vp, _i64, _vp, _vp, _i64, _i64, _int, _int,
                                      ctypes.c_float, _vp, _vp, _vp, _vp]
    lib.fp8_layernorm_bwd_workspace.argtypes = [_i64, _i64, _p64]
    lib.fp8_layernorm_bwd.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _int, _int,
                                      _vp, _vp, _vp, _vp, _i64, _vp]
    lib.fp8_moe_rows.argtypes = [_i64, _i32, _i32, _i32, _p64]
    lib.fp8_moe_sort_workspace.argtypes = [_i64, _i32, _i32, _p64]
    lib.fp8_moe_sort.argtypes = [_vp, _int, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _i64,
                                 _vp]
    lib.fp8_moe_dispatch.argtypes = [_vp, _i64, _vp, _vp, _i64, _i32, _i64, _i64, _int, _vp, _vp]
    lib.fp8_moe_dispatch_bwd.argtypes = [_vp, _i64, _vp, _i64, _i32, _i64, _i64, _int, _vp, _vp]
    lib.fp8_moe_combine.argtypes = [_vp, _i64, _vp, _vp, _i64, _i32, _i64, _i64, _int, _vp, _vp]
    lib.fp8_moe_combine_bwd.argtypes = [_vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _i32, _i64,
                                        _i64, _int, _vp, _vp, _vp]
    for name in EXPORTS:
        if name not in ("fp8_last_error", "fp8_version"):
            getattr(lib, name).restype = _int
    lib.fp8_last_error.restype = ctypes.c_char_p
    lib.fp8_last_error.argtypes = []
    lib.fp8_version.restype = ctypes.c_char_p
    lib.fp8_version.argtypes = []
    _lib = lib
    return lib


def _check(fn: str, status: int) -> None:
    if status != FP8_OK:
        raise Fp8Error(fn, status, load().fp8_last_error().decode())


def _ptr(t, offset_elems: int = 0):
    """Device address of a tensor (plus an element offset), or None."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("fp8lin takes device tensors")
    if not t.is_contiguous():
        raise ValueError("fp8lin takes contiguous row-major tensors")
    p = t.data_ptr()
    return p + offset_elems * t.element_size() if offset_elems else p


# The current stream's raw handle. torch.cuda.current_stream() builds a Stream object on
# every call, about 3 us of host time, more than this library's own launch; torch's raw
# accessor returns the same handle without it. Where a torch build lacks it, the public
# call serves.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _cur_device is not None:
        return _raw_stream(_cur_device())
    return torch.cuda.current_stream().cuda_stream


_CODE_DTYPES = (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)
_BF16_DTYPES = (torch.bfloat16, torch.int16, torch.uint16)


def _codes(t):
    """uint8 view of an fp8 code tensor (uint8, float8_e4m3fn or float8_e5m2 storage)."""
    if t is None:
        return None
    if t.dtype in (torch.float8_e4m3fn, torch.float8_e5m2):
        return t.view(torch.uint8)
    if t.dtype != torch.uint8:
        raise ValueError(f"fp8 codes must be uint8 or float8 storage, got {t.dtype}")
    return t


def _bf16(t):
    if t.dtype not in _BF16_DTYPES:
        raise ValueError(f"expected a bf16 tensor, got {t.dtype}")
    return t


def _f32(t, name):
    if t is not None and t.dtype != torch.float32:
        raise ValueError(f"{name} must be float32")
    return t


class Slot:
    """A float32 element inside a device tensor (a scale slot), passed by address."""

    def __init__(self, tensor, index: int = 0):
        _f32(tensor, "slot")
        if not 0 <= int(index) < tensor.numel():
            raise ValueError(f"slot {index} is outside a tensor of {tensor.numel()} elements")
        self.tensor, self.index = tensor, int(index)

    def ptr(self):
        return _ptr(self.tensor, self.index)


def _fptr(v, name):
    if v is None:
        return None
    if isinstance(v, Slot):
        return v.ptr()
    return _ptr(_f32(v, name))


def _need(t, name, shape, dtypes, dev=None):
    """Check a buffer before its address goes to the library: dtype, exact shape,
    contiguity and device (``dev``: the device of the call's first operand). Raises
    ValueError; nothing has been enqueued at that point."""
    if t is None:
        return
    # one combined test on the common path (every attribute read costs), the reason after
    if (t.dtype in dtypes and t.shape == tuple(shape) and t.is_contiguous()
            and (dev is None or t.device == dev)):
        return
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if tuple(t.shape) != tuple(int(v) for v in shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    raise ValueError(f"{name} is on {t.device}, the operands on {dev}")


def _need_scalar(v, name, dev=None, count=1):
    """A float32 scale or amax: a Slot, or a tensor of at least ``count`` elements."""
    if v is None:
        return
    t = v.tensor if isinstance(v, Slot) else v
    _f32(t, name)
    if not isinstance(v, Slot) and t.numel() < count:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {count}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the operands on {dev}")


def _need_scales(v, name, gran, grid, dev):
    """Tensorwise: one float32 scale; block recipe: the scale grid of that exact shape."""
    if gran & 0xFF == FP8_TENSORWISE:
        _need_scalar(v, name, dev)
    else:
        if isinstance(v, Slot):
            raise ValueError(f"{name}: the block recipe takes a scale grid, not a slot")
        _need(v, name, grid, (torch.float32,), dev)


def _grids(gran, rows, cols):
    """Shapes of (amax, scale, scale_t) for a block-recipe quantize of [rows, cols]."""
    if gran == FP8_BLOCK_1x128:
        return (rows, cols // 128), (rows, cols // 128), (cols, rows // 128)
    return (rows // 128, cols // 128), (rows // 128, cols // 128), (cols // 128, rows // 128)


def fp8_quantize_amax(x, rows_valid=None, gran=FP8_TENSORWISE, scale_inv=None, q=None, q_t=None,
                      amax=None, scale=None, scale_t=None, want_q=True, want_q_t=True,
                      want_amax=True, amax_accumulate=False, e5m2=False, stream=None):
    """Quantize a bf16 [rows, cols] tensor. Returns (q, q_t, amax, scale, scale_t).

    Outputs that are not passed in are allocated here (``want_*`` False skips them).
    ``amax_accumulate`` (tensorwise): fold max|x| into the given ``amax`` instead of
    overwriting it. ``e5m2`` (tensorwise): E5M2 codes instead of E4M3.
    """
    if amax_accumulate and amax is None:
        raise ValueError("amax_accumulate needs the amax tensor to fold into")
    _bf16(x)
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [rows, cols], got shape {tuple(x.shape)}")
    rows, cols = x.shape
    rv = rows if rows_valid is None else int(rows_valid)
    dev = x.device
    q, q_t = _codes(q), _codes(q_t)
    _need(q, "q", (rows, cols), _CODE_DTYPES, dev)
    _need(q_t, "q_t", (cols, rows), _CODE_DTYPES, dev)
    if gran == FP8_TENSORWISE:
        _need_scalar(scale_inv, "scale_inv", dev)
        _need_scalar(amax, "amax", dev)
        if scale is not None or scale_t is not None:
            raise ValueError("tensorwise quantize takes no scale grids")
    elif gran in (FP8_BLOCK_1x128, FP8_BLOCK_128x128):
        ga, gs, gst = _grids(gran, rows, cols)
        _need(amax, "amax", ga, (torch.float32,), dev)
        _need(scale, "scale", gs, (torch.float32,), dev)
        _need(scale_t, "scale_t", gst, (torch.float32,), dev)
    if want_q and q is None:
        q = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    if want_q_t and q_t is None:
        q_t = torch.empty((cols, rows), dtype=torch.uint8, device=dev)
    if gran == FP8_TENSORWISE:
        if want_amax and amax is None:
            amax = torch.empty(1, dtype=torch.float32, device=dev)
    elif gran in (FP8_BLOCK_1x128, FP8_BLOCK_128x128):
        ga, gs, gst = _grids(gran, rows, cols)
        if want_amax and amax is None:
            amax = torch.empty(ga, dtype=torch.float32, device=dev)
        if q is not None and scale is None:
            scale = torch.empty(gs, dtype=torch.float32, device=dev)
        if q_t is not None and scale_t is None:
            scale_t = torch.empty(gst, dtype=torch.float32, device=dev)
    _check("fp8_quantize_amax", load().fp8_quantize_amax(
        _ptr(x), rows, cols, rv,
        gran | (FP8_AMAX_ACCUMULATE if amax_accumulate else 0) | (FP8_E5M2 if e5m2 else 0),
        _fptr(scale_inv, "scale_inv"), _ptr(q), _ptr(q_t),
        _fptr(amax, "amax"), _fptr(scale, "scale"), _fptr(scale_t, "scale_t"), _stream(stream)))
    return q, q_t, amax, scale, scale_t


def fp8_scale_update(mode, amax=None, hist=None, pos=0, scale=None, scale_inv=None,
                     clear_amax=False, e5m2=False, stream=None):
    """One scale bookkeeping op on the device (see fp8lin.h for the modes).
    ``clear_amax``: set amax to +0 after reading it (FROM_AMAX, RECORD).
    ``e5m2``: scales for E5M2 codes (57344 in place of 448; FROM_AMAX, REFRESH)."""
    if hist is not None:
        _f32(hist, "hist")
        if hist.dim() != 1 or not hist.is_contiguous():
            raise ValueError("hist must be a contiguous 1-D float32 tensor")
    length = 0 if hist is None else hist.numel()
    for v, name in ((amax, "amax"), (scale, "scale"), (scale_inv, "scale_inv")):
        _need_scalar(v, name)
    flags = (FP8_SCALE_CLEAR_AMAX if clear_amax else 0) | (FP8_E5M2 if e5m2 else 0)
    _check("fp8_scale_update", load().fp8_scale_update(
        int(mode) | flags, _fptr(amax, "amax"), _fptr(hist, "hist"), length, int(pos),
        _fptr(scale, "scale"), _fptr(scale_inv, "scale_inv"), _stream(stream)))


def _operands(a, b, an, bn):
    """Two code operands with the contraction index last; returns (a, b) as uint8 views."""
    a, b = _codes(a), _codes(b)
    for t, name in ((a, an), (b, bn)):
        if t.dim() != 2 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 2-D code tensor")
    if b.device != a.device:
        raise ValueError(f"{bn} is on {b.device}, {an} on {a.device}")
    if a.shape[1] != b.shape[1]:
        raise ValueError(f"{an} {tuple(a.shape)} and {bn} {tuple(b.shape)}: contraction sizes "
                         "differ")
    return a, b


def _m_valid(M_valid, M):
    mv = M if M_valid is None else int(M_valid)
    if not 0 <= mv <= M:
        raise ValueError(f"M_valid={mv} outside [0, {M}]")
    return mv


def fp8_linear_fwd(qx, qw, sx, sw, y=None, M_valid=None, gran=FP8_TENSORWISE, stream=None,
                   bias=None, a_e5m2=False):
    """y [M, N] bf16 = sx * sw * qx [M, K] . qw [N, K]^T (+ bias [N], bf16, in the epilogue).
    ``a_e5m2``: qx holds E5M2 codes."""
    qx, qw = _operands(qx, qw, "qx", "qw")
    M, K = qx.shape
    N = qw.shape[0]
    dev = qx.device
    _need_scales(sx, "sx", gran, (M, K // 128), dev)
    _need_scales(sw, "sw", gran, (N // 128, K // 128), dev)
    _need(y, "y", (M, N), _BF16_DTYPES, dev)
    if bias is not None:
        _need(_bf16(bias), "bias", (N,), _BF16_DTYPES, dev)
    mv = _m_valid(M_valid, M)
    gran = gran | (FP8_A_E5M2 if a_e5m2 else 0)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if bias is not None:
        _check("fp8_linear_fwd_bias", load().fp8_linear_fwd_bias(
            _ptr(qx), _ptr(qw), _fptr(sx, "sx"), _fptr(sw, "sw"), _ptr(bias), _ptr(y), M, N, K,
            mv, gran, _stream(stream)))
        return y
    _check("fp8_linear_fwd", load().fp8_linear_fwd(
        _ptr(qx), _ptr(qw), _fptr(sx, "sx"), _fptr(sw, "sw"), _ptr(y), M, N, K, mv, gran,
        _stream(stream)))
    return y


def fp8_linear_fwd_current(x, w, y=None, scales=None, qx=None, qw=None, want_codes=False,
                           stream=None):
    """One current-scaling forward of a small linear in one launch: amax of x [M, K] and of
    w [N, K] (bf16), their scales, the casts, y [M, N] bf16. Returns (y, scales, qx, qw):
    scales float32 [4] = {sx, sw, sx_inv, sw_inv}; qx, qw the e4m3 codes when passed or
    ``want_codes``, else None."""
    x, w = _bf16(x), _bf16(w)
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError(f"x {tuple(x.shape)} and w {tuple(w.shape)} must be [M, K] and [N, K]")
    M, K = x.shape
    N = w.shape[0]
    dev = x.device
    _need(x, "x", (M, K), _BF16_DTYPES, dev)
    _need(w, "w", (N, K), _BF16_DTYPES, dev)
    _need(y, "y", (M, N), _BF16_DTYPES, dev)
    _need(scales, "scales", (4,), (torch.float32,), dev)
    _need(qx, "qx", (M, K), (torch.uint8,), dev)
    _need(qw, "qw", (N, K), (torch.uint8,), dev)
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    if scales is None:
        scales = torch.empty(4, dtype=torch.float32, device=dev)
    if want_codes and qx is None:
        qx = torch.empty((M, K), dtype=torch.uint8, device=dev)
    if want_codes and qw is None:
        qw = torch.empty((N, K), dtype=torch.uint8, device=dev)
    _check("fp8_linear_fwd_current", load().fp8_linear_fwd_current(
        _ptr(x), _ptr(w), M, N, K, _ptr(y), _ptr(scales), _ptr(qx), _ptr(qw), _stream(stream)))
    return y, scales, qx, qw


def fp8_bias_grad(g, rows_valid=None, db=None, stream=None):
    """db [cols] bf16 = column sums of g [rows, cols] over the valid rows (float32 sums)."""
    _bf16(g)
    if g.dim() != 2:
        raise ValueError(f"g must be 2-D [rows, cols], got shape {tuple(g.shape)}")
    rows, cols = g.shape
    rv = _m_valid(rows_valid, rows)
    _need(db, "db", (cols,), _BF16_DTYPES, g.device)
    if db is None:
        db = torch.empty(cols, dtype=torch.bfloat16, device=g.device)
    _check("fp8_bias_grad", load().fp8_bias_grad(_ptr(g), rows, cols, rv, _ptr(db),
                                                 _stream(stream)))
    return db


def fp8_linear_dgrad(qg, qw_t, sg, sw, dx=None, M_valid=None, gran=FP8_TENSORWISE, stream=None,
                     a_e5m2=False):
    """dx [M, K] bf16 = sg * sw * qg [M, N] . qw_t [K, N]^T. ``a_e5m2``: qg holds E5M2 codes.
    Block recipe: sg [M, N/128], sw is W's transposed scale grid [K/128, N/128]."""
    qg, qw_t = _operands(qg, qw_t, "qg", "qw_t")
    M, N = qg.shape
    K = qw_t.shape[0]
    dev = qg.device
    _need_scales(sg, "sg", gran, (M, N // 128), dev)
    _need_scales(sw, "sw", gran, (K // 128, N // 128), dev)
    _need(dx, "dx", (M, K), _BF16_DTYPES, dev)
    mv = _m_valid(M_valid, M)
    gran = gran | (FP8_A_E5M2 if a_e5m2 else 0)
    if dx is None:
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dev)
    _check("fp8_linear_dgrad", load().fp8_linear_dgrad(
        _ptr(qg), _ptr(qw_t), _fptr(sg, "sg"), _fptr(sw, "sw"), _ptr(dx), M, N, K, mv, gran,
        _stream(stream)))
    return dx


def fp8_linear_wgrad(qg_t, qx_t, sg, sx, dw=None, gran=FP8_TENSORWISE, stream=None,
                     a_e5m2=False):
    """dw [N, K] bf16 = sg * sx * qg_t [N, M] . qx_t [K, M]^T. ``a_e5m2``: qg_t holds E5M2
    codes. Block recipe: sg [N, M/128], sx [K, M/128] (the transposed copies' grids)."""
    qg_t, qx_t = _operands(qg_t, qx_t, "qg_t", "qx_t")
    N, M = qg_t.shape
    K = qx_t.shape[0]
    dev = qg_t.device
    _need_scales(sg, "sg", gran, (N, M // 128), dev)
    _need_scales(sx, "sx", gran, (K, M // 128), dev)
    _need(dw, "dw", (N, K), _BF16_DTYPES, dev)
    gran = gran | (FP8_A_E5M2 if a_e5m2 else 0)
    if dw is None:
        dw = torch.empty((N, K), dtype=torch.bfloat16, device=dev)
    _check("fp8_linear_wgrad", load().fp8_linear_wgrad(
        _ptr(qg_t), _ptr(qx_t), _fptr(sg, "sg"), _fptr(sx, "sx"), _ptr(dw), M, N, K, gran,
        _stream(stream)))
    return dw


def fp8_pad_tokens(x, T=None, multiple=16, x_pad=None, query_only=False, stream=None):
    """Pad a bf16 [T, cols] batch to a multiple of ``multiple`` rows.

    Returns ``(x_pad, T_pad)``. With ``query_only`` only T_pad is computed. If
    ``x_pad is x`` the tail of x's own buffer (which must hold T_pad rows) is
    zeroed in place, with T given explicitly.
    """
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [rows, cols], got shape {tuple(x.shape)}")
    cols = x.shape[1]
    T = x.shape[0] if T is None else int(T)
    out = ctypes.c_int64(0)
    lib = load()
    _check("fp8_pad_tokens", lib.fp8_pad_tokens(None, T, cols, int(multiple), None,
                                                ctypes.byref(out), None))
    T_pad = out.value
    if query_only:
        return None, T_pad
    _bf16(x)
    if x_pad is x:
        if x.shape[0] < T_pad:
            raise ValueError(f"in place: the buffer holds {x.shape[0]} rows, needs {T_pad}")
    elif x.shape[0] < T:
        raise ValueError(f"x holds {x.shape[0]} rows, T={T}")
    if x_pad is None:
        x_pad = torch.empty((T_pad, cols), dtype=x.dtype, device=x.device)
    _bf16(x_pad)
    if x_pad.dim() != 2 or x_pad.shape[0] < T_pad or x_pad.shape[1] != cols:
        raise ValueError(f"x_pad has shape {tuple(x_pad.shape)}, needs at least [{T_pad}, {cols}]")
    if x_pad.device != x.device:
        raise ValueError("x_pad and x are on different devices")
    _check("fp8_pad_tokens", lib.fp8_pad_tokens(_ptr(x), T, cols, int(multiple),
                                                _ptr(x_pad), ctypes.byref(out), _stream(stream)))
    return x_pad, T_pad


def fp8_align_multiple(layout, batch=1, tp=1, cp=1, base=16):
    """(per-sequence multiple, total multiple) of a token layout (FP8_LAYOUT_THD or
    FP8_LAYOUT_BSHD) under tensor/sequence (tp) and context (cp) parallelism."""
    seq, tot = ctypes.c_int32(0), ctypes.c_int32(0)
    _check("fp8_align_multiple", load().fp8_align_multiple(
        int(layout), int(batch), int(tp), int(cp), int(base), ctypes.byref(seq),
        ctypes.byref(tot)))
    return seq.value, tot.value


def _offsets(cu):
    arr = (_i64 * len(cu))(*[int(v) for v in cu])
    return arr


def fp8_pad_varlen(x, cu_seqlens, seq_multiple=1, total_multiple=16, x_pad=None,
                   query_only=False, stream=None):
    """Pad every sequence of a packed bf16 [T, cols] batch to a multiple of ``seq_multiple``
    rows and the batch to a multiple of ``total_multiple``. ``cu_seqlens``: host offsets
    [nseq + 1] (a list, or a CPU tensor). Returns ``(x_pad, cu_seqlens_pad, T_pad)``;
    ``query_only`` computes the offsets only (x_pad is None)."""
    cu = _offsets([int(v) for v in cu_seqlens])
    nseq = len(cu) - 1
    if x.dim() != 2:
        raise ValueError(f"x must be 2-D [rows, cols], got shape {tuple(x.shape)}")
    cols = x.shape[1]
    cu_pad = (_i64 * (nseq + 1))()
    T_pad = ctypes.c_int64(0)
    lib = load()
    _check("fp8_pad_varlen", lib.fp8_pad_varlen(None, cu, nseq, cols, int(seq_multiple),
                                                int(total_multiple), None, cu_pad,
                                                ctypes.byref(T_pad), None))
    if query_only:
        return None, list(cu_pad), T_pad.value
    _bf16(x)
    if x.shape[0] < cu[nseq]:
        raise ValueError(f"x holds {x.shape[0]} rows, the offsets reach {cu[nseq]}")
    if x_pad is None:
        x_pad = torch.empty((T_pad.value, cols), dtype=x.dtype, device=x.device)
    _bf16(x_pad)
    if x_pad.dim() != 2 or x_pad.shape[0] < T_pad.value or x_pad.shape[1] != cols:
        raise ValueError(f"x_pad has shape {tuple(x_pad.shape)}, needs at least "
                         f"[{T_pad.value}, {cols}]")
    if x_pad.device != x.device:
        raise ValueError("x_pad and x are on different devices")
    _check("fp8_pad_varlen", lib.fp8_pad_varlen(_ptr(x), cu, nseq, cols,
                                                int(seq_multiple), int(total_multiple),
                                                _ptr(x_pad), cu_pad, ctypes.byref(T_pad),
                                                _stream(stream)))
    return x_pad, list(cu_pad), T_pad.value


def fp8_unpad_varlen(x_pad, cu_seqlens, cu_seqlens_pad, x=None, stream=None):
    """The inverse gather of fp8_pad_varlen: the sequences' rows of x_pad, packed."""
    cu = _offsets([int(v) for v in cu_seqlens])
    cu_pad = _offsets([int(v) for v in cu_seqlens_pad])
    nseq = len(cu) - 1
    if len(cu_pad) != nseq + 1:
        raise ValueError("cu_seqlens and cu_seqlens_pad differ in length")
    _bf16(x_pad)
    if x_pad.dim() != 2:
        raise ValueError(f"x_pad must be 2-D [rows, cols], got shape {tuple(x_pad.shape)}")
    cols = x_pad.shape[1]
    if x_pad.shape[0] < cu_pad[nseq]:
        raise ValueError(f"x_pad holds {x_pad.shape[0]} rows, the padded offsets reach "
                         f"{cu_pad[nseq]}")
    if x is None:
        x = torch.empty((int(cu[nseq]), cols), dtype=x_pad.dtype, device=x_pad.device)
    _bf16(x)
    if x.dim() != 2 or x.shape[0] < cu[nseq] or x.shape[1] != cols:
        raise ValueError(f"x has shape {tuple(x.shape)}, needs at least [{cu[nseq]}, {cols}]")
    if x.device != x_pad.device:
        raise ValueError("x and x_pad are on different devices")
    _check("fp8_unpad_varlen", load().fp8_unpad_varlen(_ptr(x_pad), cu, cu_pad, nseq,
                                                      cols, _ptr(x), _stream(stream)))
    return x


# ------------------------------------------------------- layer norm, expert dispatch
_DT = {torch.bfloat16: FP8_DT_BF16, torch.float16: FP8_DT_F16, torch.float32: FP8_DT_F32}
_I32 = (torch.int32,)
_F32 = (torch.float32,)


def _rows2d(t, name, dev=None, dtype=None, cols=None, rows=None):
    """Check a [rows, cols] input whose rows may be a cut out of a wider tensor; returns its
    row stride in elements (at least the width; 0- and 1-row tensors may have any)."""
    if t.dtype not in _DT:
        raise ValueError(f"{name} has dtype {t.dtype}, expected bfloat16, float16 or float32")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D [rows, cols], got shape {tuple(t.shape)}")
    r, c = t.shape
    if (cols is not None and c != cols) or (rows is not None and r != rows):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected "
                         f"({'any' if rows is None else rows}, {'any' if cols is None else cols})")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the operands on {dev}")
    ld, inner = t.stride()
    if c > 1 and inner != 1:
        raise ValueError(f"{name}: the columns of a row must be contiguous, stride {inner}")
    if r <= 1:
        return max(ld, c)
    if ld < c:
        raise ValueError(f"{name}: rows overlap (stride {ld}, {c} columns)")
    return ld


def _dptr(t):
    """Address of a device tensor whose layout was checked (any row stride)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("fp8lin takes device tensors")
    return t.data_ptr()


def _launch_on(x, stream):
    """Checks before the call's own allocations: a device tensor, on the current device
    (kernels go to the current device's stream)."""
    if not x.is_cuda:
        raise ValueError("fp8lin takes device tensors")
    cur = _cur_device() if _cur_device is not None else torch.cuda.current_device()
    if x.device.index != cur:
        raise ValueError(f"the operands are on {x.device}, the current device is cuda:{cur}")
    if stream is not None and stream.device.index != cur:
        raise ValueError(f"the stream is on {stream.device}, the current device is cuda:{cur}")


def _new(shape, dtype, dev, stream):
    """An output or workspace in the memory pool of the stream that will write it, so that a
    call on a stream other than the current one never reuses memory in use on the latter."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _params(dtype, cols, dev, *named):
    """The common dtype of the given parameter tensors [cols]: the rows' dtype or float32."""
    pdt = None
    for t, name in named:
        if t is None:
            continue
        if pdt is None:
            if t.dtype != dtype and t.dtype != torch.float32:
                raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype} or float32")
            pdt = t.dtype
        _need(t, name, (cols,), (pdt,), dev)
    return pdt


def fp8_layernorm_fwd(x, gamma=None, beta=None, eps=1e-5, y=None, mean=None, rstd=None,
                      want_stats=True, stream=None):
    """Layer norm of each row of x [rows, cols] (bf16, f16 or f32; rows may be strided).
    gamma, beta [cols] in x's dtype or float32, or None. Returns (y, mean, rstd): y in x's
    dtype, the statistics float32 [rows] (None without ``want_stats`` unless passed)."""
    ldx = _rows2d(x, "x")
    rows, cols = x.shape
    dev = x.device
    pdt = _params(x.dtype, cols, dev, (gamma, "gamma"), (beta, "beta")) or x.dtype
    _need(y, "y", (rows, cols), (x.dtype,), dev)
    _need(mean, "mean", (rows,), _F32, dev)
    _need(rstd, "rstd", (rows,), _F32, dev)
    _launch_on(x, stream)
    if y is None:
        y = _new((rows, cols), x.dtype, dev, stream)
    if want_stats:
        if mean is None:
            mean = _new((rows,), torch.float32, dev, stream)
        if rstd is None:
            rstd = _new((rows,), torch.float32, dev, stream)
    _check("fp8_layernorm_fwd", load().fp8_layernorm_fwd(
        x.data_ptr(), ldx, _dptr(gamma), _dptr(beta), rows, cols, _DT[x.dtype], _DT[pdt],
        float(eps), y.data_ptr(), _dptr(mean), _dptr(rstd), _stream(stream)))
    return y, mean, rstd


def fp8_layernorm_bwd(dy, x, mean, rstd, gamma=None, dx=None, dgamma=None, dbeta=None,
                      want_dx=True, want_dgamma=True, want_dbeta=True, param_dtype=None,
                      workspace=None, stream=None):
    """The gradient of fp8_layernorm_fwd from dy and what the forward kept. Returns
    (dx, dgamma, dbeta), None for those not wanted and not passed. dgamma and dbeta have
    gamma's dtype (``param_dtype``, else x's dtype, without gamma). ``workspace``: a uint8
    tensor of at least fp8_layernorm_bwd_workspace(rows, cols) bytes, else allocated."""
    ldx = _rows2d(x, "x")
    rows, cols = x.shape
    dev = x.device
    lddy = _rows2d(dy, "dy", dev, x.dtype, cols, rows)
    _need(mean, "mean", (rows,), _F32, dev)
    _need(rstd, "rstd", (rows,), _F32, dev)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd of the forward are needed")
    pdt = _params(x.dtype, cols, dev, (gamma, "gamma"), (dgamma, "dgamma"), (dbeta, "dbeta"))
    if pdt is None:
        pdt = x.dtype if param_dtype is None else param_dtype
        if pdt not in (x.dtype, torch.float32):
            raise ValueError(f"param_dtype {pdt}, expected {x.dtype} or float32")
    _need(dx, "dx", (rows, cols), (x.dtype,), dev)
    _launch_on(x, stream)
    if want_dx and dx is None:
        dx = _new((rows, cols), x.dtype, dev, stream)
    if want_dgamma and dgamma is None:
        dgamma = _new((cols,), pdt, dev, stream)
    if want_dbeta and dbeta is None:
        dbeta = _new((cols,), pdt, dev, stream)
    need = 0
    if dgamma is not None or dbeta is not None:
        need = fp8_layernorm_bwd_workspace(rows, cols)
        workspace = _workspace(workspace, need, dev, stream)
    _check("fp8_layernorm_bwd", load().fp8_layernorm_bwd(
        dy.data_ptr(), lddy, x.data_ptr(), ldx, mean.data_ptr(), rstd.data_ptr(), _dptr(gamma),
        rows, cols, _DT[x.dtype], _DT[pdt], _dptr(dx), _dptr(dgamma), _dptr(dbeta),
        _dptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream)))
    return dx, dgamma, dbeta


def _workspace(t, need, dev, stream):
    if t is None:
        return _new((need,), torch.uint8, dev, stream) if need else None
    if t.dtype != torch.uint8 or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    if t.numel() < need:
        raise ValueError(f"workspace holds {t.numel()} bytes, needs {need}")
    return t


def fp8_layernorm_bwd_workspace(rows, cols):
    """Bytes of workspace of fp8_layernorm_bwd."""
    out = _i64(0)
    _check("fp8_layernorm_bwd_workspace",
           load().fp8_layernorm_bwd_workspace(int(rows), int(cols), ctypes.byref(out)))
    return out.value


def fp8_moe_rows(tokens, topk, experts, multiple=16):
    """Rows of the sorted buffer for any routing of ``tokens`` tokens to ``topk`` of
    ``experts`` experts, each expert's rows padded to a multiple of ``multiple``."""
    out = _i64(0)
    _check("fp8_moe_rows", load().fp8_moe_rows(int(tokens), int(topk), int(experts),
                                               int(multiple), ctypes.byref(out)))
    return out.value


def fp8_moe_sort_workspace(tokens, topk, experts):
    """Bytes of workspace of fp8_moe_sort."""
    out = _i64(0)
    _check("fp8_moe_sort_workspace", load().fp8_moe_sort_workspace(
        int(tokens), int(topk), int(experts), ctypes.byref(out)))
    return out.value


def fp8_moe_sort(expert_idx, experts, multiple=16, slot=None, source=None, counts=None,
                 offsets=None, workspace=None, stream=None):
    """Sort the (token, choice) pairs of expert_idx [tokens, topk] (int32 or int64; an index
    outside [0, experts) drops its pair) by expert, stably, every expert's rows padded to a
    multiple of ``multiple``. Returns int32 (slot [tokens, topk], source [rows], counts
    [experts], offsets [experts + 1]); see fp8lin.h. Nothing reaches the host."""
    if expert_idx.dim() != 2:
        raise ValueError(f"expert_idx must be 2-D [tokens, topk], got {tuple(expert_idx.shape)}")
    tokens, topk = expert_idx.shape
    dev = expert_idx.device
    _need(expert_idx, "expert_idx", (tokens, topk), (torch.int32, torch.int64))
    rows = fp8_moe_rows(tokens, topk, experts, multiple)
    _need(slot, "slot", (tokens, topk), _I32, dev)
    _need(source, "source", (rows,), _I32, dev)
    _need(counts, "counts", (experts,), _I32, dev)
    _need(offsets, "offsets", (experts + 1,), _I32, dev)
    _launch_on(expert_idx, stream)
    if slot is None:
        slot = _new((tokens, topk), torch.int32, dev, stream)
    if source is None:
        source = _new((rows,), torch.int32, dev, stream)
    if counts is None:
        counts = _new((experts,), torch.int32, dev, stream)
    if offsets is None:
        offsets = _new((experts + 1,), torch.int32, dev, stream)
    workspace = _workspace(workspace, fp8_moe_sort_workspace(tokens, topk, experts), dev, stream)
    _check("fp8_moe_sort", load().fp8_moe_sort(
        expert_idx.data_ptr(), expert_idx.element_size(), tokens, topk, int(experts),
        int(multiple), slot.data_ptr(), source.data_ptr(), counts.data_ptr(), offsets.data_ptr(),
        _dptr(workspace), 0 if workspace is None else workspace.numel(), _stream(stream)))
    return slot, source, counts, offsets


def _plan(slot, source, dev):
    """(tokens, topk, rows) of a sort's index tensors."""
    if slot.dim() != 2:
        raise ValueError(f"slot must be 2-D [tokens, topk], got {tuple(slot.shape)}")
    _need(slot, "slot", slot.shape, _I32, dev)
    if source is not None:
        if source.dim() != 1:
            raise ValueError(f"source must be 1-D [rows], got {tuple(source.shape)}")
        _need(source, "source", source.shape, _I32, dev)
    return slot.shape[0], slot.shape[1], 0 if source is None else source.shape[0]


def fp8_moe_dispatch(x, slot, source, xs=None, stream=None):
    """xs [rows, cols]: the tokens' rows of x [tokens, cols] (rows may be strided) in the order
    of the sort, 0 in the padding rows."""
    ldx = _rows2d(x, "x")
    dev, cols = x.device, x.shape[1]
    tokens, topk, rows = _plan(slot, source, dev)
    if x.shape[0] != tokens:
        raise ValueError(f"x has {x.shape[0]} rows, slot is for {tokens} tokens")
    _need(xs, "xs", (rows, cols), (x.dtype,), dev)
    _launch_on(x, stream)
    if xs is None:
        xs = _new((rows, cols), x.dtype, dev, stream)
    _check("fp8_moe_dispatch", load().fp8_moe_dispatch(
        x.data_ptr(), ldx, slot.data_ptr(), source.data_ptr(), tokens, topk, rows, cols,
        _DT[x.dtype], xs.data_ptr(), _stream(stream)))
    return xs


def fp8_moe_dispatch_bwd(dxs, slot, dx=None, stream=None):
    """dx [tokens, cols]: the dispatch's gradient, each token's rows of dxs [rows, cols] (may be
    strided) added up."""
    ld = _rows2d(dxs, "dxs")
    dev, (rows, cols) = dxs.device, dxs.shape
    tokens, topk, _ = _plan(slot, None, dev)
    _need(dx, "dx", (tokens, cols), (dxs.dtype,), dev)
    _launch_on(dxs, stream)
    if dx is None:
        dx = _new((tokens, cols), dxs.dtype, dev, stream)
    _check("fp8_moe_dispatch_bwd", load().fp8_moe_dispatch_bwd(
        dxs.data_ptr(), ld, slot.data_ptr(), tokens, topk, rows, cols, _DT[dxs.dtype],
        dx.data_ptr(), _stream(stream)))
    return dx


def fp8_moe_combine(ys, slot, weights, y=None, stream=None):
    """y [tokens, cols]: each token's rows of ys [rows, cols] (may be strided) added with the
    router's weights, float32 [tokens, topk]; dropped pairs add nothing."""
    ld = _rows2d(ys, "ys")
    dev, (rows, cols) = ys.device, ys.shape
    tokens, topk, _ = _plan(slot, None, dev)
    _need(weights, "weights", (tokens, topk), _F32, dev)
    _need(y, "y", (tokens, cols), (ys.dtype,), dev)
    _launch_on(ys, stream)
    if y is None:
        y = _new((tokens, cols), ys.dtype, dev, stream)
    _check("fp8_moe_combine", load().fp8_moe_combine(
        ys.data_ptr(), ld, slot.data_ptr(), weights.data_ptr(), tokens, topk, rows, cols,
        _DT[ys.dtype], y.data_ptr(), _stream(stream)))
    return y


def fp8_moe_combine_bwd(dy, ys, slot, source, weights, dys=None, dw=None, stream=None):
    """The combine's gradients (dys [rows, cols], dw float32 [tokens, topk]) from dy
    [tokens, cols] and ys; padding rows of dys and dropped pairs of dw are 0."""
    ldys = _rows2d(ys, "ys")
    dev, cols = ys.device, ys.shape[1]
    tokens, topk, rows = _plan(slot, source, dev)
    if ys.shape[0] != rows:
        raise ValueError(f"ys has {ys.shape[0]} rows, source {rows}")
    lddy = _rows2d(dy, "dy", dev, ys.dtype, cols, tokens)
    _need(weights, "weights", (tokens, topk), _F32, dev)
    _need(dys, "dys", (rows, cols), (ys.dtype,), dev)
    _need(dw, "dw", (tokens, topk), _F32, dev)
    _launch_on(ys, stream)
    if dys is None:
        dys = _new((rows, cols), ys.dtype, dev, stream)
    if dw is None:
        dw = _new((tokens, topk), torch.float32, dev, stream)
    _check("fp8_moe_combine_bwd", load().fp8_moe_combine_bwd(
        dy.data_ptr(), lddy, ys.data_ptr(), ldys, slot.data_ptr(), source.data_ptr(),
        weights.data_ptr(), tokens, topk, rows, cols, _DT[ys.dtype], dys.data_ptr(),
        dw.data_ptr(), _stream(stream)))
    return dys, dw


def fp8_last_error() -> str:
    return load().fp8_last_error().decode()


def fp8_version() -> str:
    return load().fp8_version().decode()
