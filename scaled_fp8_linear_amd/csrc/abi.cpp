// C ABI of the scaled FP8 linear layer: argument checking and dispatch.
// The declarations, with the meaning of every argument, are in include/fp8lin.h.
#include "../../include/fp8lin.h"

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include <initializer_list>

#include "launch.h"

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return code;
}

int ok() {
  g_err[0] = '\0';
  return FP8_OK;
}

int hip_status(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(FP8_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
  return ok();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

constexpr int64_t kMaxOperandBytes = (int64_t)1 << 31;
constexpr int64_t kMaxContraction = (int64_t)1 << 17;

// Checks shared by the three GEMM entry points. A is [rows_a, kc], B is [rows_b, kc].
int check_gemm(const char* fn, const void* a, const void* b, const float* s1, const float* s2,
               const void* d, int64_t rows_a, int64_t rows_b, int64_t kc, int64_t m_valid,
               int gran, bool a_e5m2) {
  if (rows_a < 0 || rows_b < 0 || kc < 0)
    return fail(FP8_ERR_SHAPE, "%s: negative size", fn);
  if (rows_a % 16 || rows_b % 16 || kc % 16)
    return fail(FP8_ERR_SHAPE,
                "%s: sizes must be multiples of 16 (got %lld x %lld x %lld); FP8 GEMMs need the "
                "token count and every dimension divisible by 16",
                fn, (long long)rows_a, (long long)rows_b, (long long)kc);
  if (m_valid < 0 || m_valid > rows_a)
    return fail(FP8_ERR_SHAPE, "%s: M_valid=%lld outside [0, %lld]", fn, (long long)m_valid,
                (long long)rows_a);
  if (gran != FP8_TENSORWISE && gran != FP8_BLOCK_1x128)
    return fail(FP8_ERR_UNSUPPORTED, "%s: granularity %d (use FP8_TENSORWISE or FP8_BLOCK_1x128)",
                fn, gran);
  if (a_e5m2 && gran != FP8_TENSORWISE)
    return fail(FP8_ERR_UNSUPPORTED, "%s: e5m2 operands (FP8_A_E5M2) are for FP8_TENSORWISE", fn);
  if (gran == FP8_BLOCK_1x128 && kc % 128)
    return fail(FP8_ERR_SHAPE, "%s: block recipe needs the contraction size %% 128 == 0 (got %lld)",
                fn, (long long)kc);
  if (rows_a * kc >= kMaxOperandBytes || rows_b * kc >= kMaxOperandBytes ||
      rows_a * rows_b * 2 >= kMaxOperandBytes)
    return fail(FP8_ERR_UNSUPPORTED, "%s: an operand or the output holds 2^31 bytes or more", fn);
  if (kc >= kMaxContraction)
    return fail(FP8_ERR_UNSUPPORTED, "%s: contraction size %lld >= 2^17", fn, (long long)kc);
  if (rows_a * rows_b > 0) {
    if (!d) return fail(FP8_ERR_NULL, "%s: NULL output", fn);
    // an empty contraction reads neither operands nor scales (the output is all zeros)
    if (kc > 0 && (!a || !b || !s1 || !s2))
      return fail(FP8_ERR_NULL, "%s: NULL operand or scale pointer", fn);
    if (!aligned16(a) || !aligned16(b) || !aligned16(d))
      return fail(FP8_ERR_ALIGN, "%s: operands and output must be 16-byte aligned", fn);
  }
  return FP8_OK;
}

}  // namespace

extern "C" {

const char* fp8_last_error(void) { return g_err; }

const char* fp8_version(void) { return "fp8lin 0.1 gfx950"; }

int fp8_quantize_amax(const void* x, int64_t rows, int64_t cols, int64_t rows_valid, int gran,
                      const float* scale_inv, void* q, void* q_t, float* amax, float* scale,
                      float* scale_t, void* stream) {
  const char* fn = "fp8_quantize_amax";
  const bool accumulate = (gran & FP8_AMAX_ACCUMULATE) != 0;
  const bool e5m2 = (gran & FP8_E5M2) != 0;
  gran &= ~(FP8_AMAX_ACCUMULATE | FP8_E5M2);
  if (accumulate && gran != FP8_TENSORWISE)
    return fail(FP8_ERR_UNSUPPORTED, "%s: FP8_AMAX_ACCUMULATE is for FP8_TENSORWISE", fn);
  if (e5m2 && gran != FP8_TENSORWISE)
    return fail(FP8_ERR_UNSUPPORTED, "%s: FP8_E5M2 codes are for FP8_TENSORWISE", fn);
  if (rows < 0 || cols < 0) return fail(FP8_ERR_SHAPE, "%s: negative size", fn);
  if (rows_valid < 0 || rows_valid > rows)
    return fail(FP8_ERR_SHAPE, "%s: rows_valid=%lld outside [0, %lld]", fn, (long long)rows_valid,
                (long long)rows);
  const int64_t mult = (gran == FP8_TENSORWISE) ? 16 : 128;
  if (rows % mult || cols % mult)
    return fail(FP8_ERR_SHAPE, "%s: rows and cols must be multiples of %lld (got %lld x %lld)", fn,
                (long long)mult, (long long)rows, (long long)cols);
  if (rows * cols > 0 && !x) return fail(FP8_ERR_NULL, "%s: x is NULL", fn);
  if (!aligned16(x) || !aligned16(q) || !aligned16(q_t))
    return fail(FP8_ERR_ALIGN, "%s: x, q and q_t must be 16-byte aligned", fn);
  const hipStream_t s = as_stream(stream);
  auto* xb = static_cast<const uint16_t*>(x);
  auto* qb = static_cast<uint8_t*>(q);
  auto* qtb = static_cast<uint8_t*>(q_t);
  switch (gran) {
    case FP8_TENSORWISE:
      if ((q || q_t) && !scale_inv) return fail(FP8_ERR_NULL, "%s: scale_inv is NULL", fn);
      if (scale || scale_t)
        return fail(FP8_ERR_UNSUPPORTED, "%s: scale/scale_t are outputs of the block modes only", fn);
      return hip_status(
          fp8lin::launch_quantize_tensorwise(xb, rows, cols, rows_valid, scale_inv, qb, qtb, amax,
                                             accumulate, e5m2, s),
          fn);
    case FP8_BLOCK_1x128:
    case FP8_BLOCK_128x128:
      if (scale_inv)
        return fail(FP8_ERR_UNSUPPORTED, "%s: block modes compute their own multipliers; pass NULL", fn);
      if ((q == nullptr) != (scale == nullptr))
        return fail(FP8_ERR_NULL, "%s: q and scale must both be given or both be NULL", fn);
      if ((q_t == nullptr) != (scale_t == nullptr))
        return fail(FP8_ERR_NULL, "%s: q_t and scale_t must both be given or both be NULL", fn);
      if (gran == FP8_BLOCK_128x128) {
        if (rows_valid != rows)
          return fail(FP8_ERR_SHAPE, "%s: 128x128 tiles (weights) take no padding rows", fn);
        return hip_status(fp8lin::launch_quantize_block_128x128(xb, rows, cols, qb, qtb, amax,
                                                                scale, scale_t, s),
                          fn);
      }
      return hip_status(fp8lin::launch_quantize_block_1x128(xb, rows, cols, rows_valid, qb, qtb,
                                                            amax, scale, scale_t, s),
                        fn);
    default:
      return fail(FP8_ERR_UNSUPPORTED, "%s: unknown granularity %d", fn, gran);
  }
}

int fp8_scale_update(int mode, float* amax, float* hist, int32_t len, int32_t pos,
                     float* scale, float* scale_inv, void* stream) {
  const char* fn = "fp8_scale_update";
  const bool clear = (mode & FP8_SCALE_CLEAR_AMAX) != 0;
  const bool e5m2 = (mode & FP8_E5M2) != 0;
  mode &= ~(FP8_SCALE_CLEAR_AMAX | FP8_E5M2);
  if (clear && mode != FP8_SCALE_FROM_AMAX && mode != FP8_SCALE_RECORD)
    return fail(FP8_ERR_UNSUPPORTED, "%s: FP8_SCALE_CLEAR_AMAX needs a mode that reads amax", fn);
  if (e5m2 && mode != FP8_SCALE_FROM_AMAX && mode != FP8_SCALE_REFRESH)
    return fail(FP8_ERR_UNSUPPORTED, "%s: FP8_E5M2 goes with a mode that writes scales", fn);
  switch (mode) {
    case FP8_SCALE_FROM_AMAX:
      if (!amax || !scale || !scale_inv) return fail(FP8_ERR_NULL, "%s: NULL pointer", fn);
      break;
    case FP8_SCALE_RECORD:
      if (!amax || !hist) return fail(FP8_ERR_NULL, "%s: NULL pointer", fn);
      if (len < 1 || pos < 0 || pos >= len)
        return fail(FP8_ERR_SHAPE, "%s: pos=%d outside a ring of %d", fn, pos, len);
      break;
    case FP8_SCALE_REFRESH:
      if (!hist || !scale || !scale_inv) return fail(FP8_ERR_NULL, "%s: NULL pointer", fn);
      if (len < 1) return fail(FP8_ERR_SHAPE, "%s: empty history", fn);
      break;
    default:
      return fail(FP8_ERR_UNSUPPORTED, "%s: unknown mode %d", fn, mode);
  }
  return hip_status(fp8lin::launch_scale_update(mode, amax, clear, hist, len, pos, scale,
                                                scale_inv, e5m2, as_stream(stream)),
                    fn);
}

int fp8_linear_fwd(const void* qx, const void* qw, const float* sx, const float* sw, void* y,
                   int64_t M, int64_t N, int64_t K, int64_t M_valid, int gran, void* stream) {
  const bool a5 = (gran & FP8_A_E5M2) != 0;
  gran &= ~FP8_A_E5M2;
  int e = check_gemm("fp8_linear_fwd", qx, qw, sx, sw, y, M, N, K, M_valid, gran, a5);
  if (e) return e;
  if (gran == FP8_BLOCK_1x128 && N % 128)
    return fail(FP8_ERR_SHAPE, "fp8_linear_fwd: block recipe needs N %% 128 == 0");
  return hip_status(fp8lin::launch_gemm_fp8(static_cast<const uint8_t*>(qx),
                                            static_cast<const uint8_t*>(qw), sx, sw, nullptr,
                                            static_cast<uint16_t*>(y), M, N, K, M_valid,
                                            gran == FP8_BLOCK_1x128, 128, a5, as_stream(stream)),
                    "fp8_linear_fwd");
}

int fp8_linear_fwd_current(const void* x, const void* w, int64_t M, int64_t N, int64_t K,
                           void* y, float* scales, void* qx, void* qw, void* stream) {
  const char* fn = "fp8_linear_fwd_current";
  if (M < 16 || N < 16 || K < 128 || M % 16 || N % 16 || K % 128)
    return fail(FP8_ERR_SHAPE,
                "%s: M and N must be positive multiples of 16 and K a positive multiple of 128 "
                "(got %lld x %lld x %lld)",
                fn, (long long)M, (long long)N, (long long)K);
  if ((M + N) * K > fp8lin::kSmallLinearCodes)
    return fail(FP8_ERR_UNSUPPORTED,
                "%s: (M + N) K = %lld bytes of codes exceed the small-linear limit of %d; use "
                "fp8_quantize_amax, fp8_scale_update and fp8_linear_fwd",
                fn, (long long)((M + N) * K), fp8lin::kSmallLinearCodes);
  if (!x || !w || !y || !scales) return fail(FP8_ERR_NULL, "%s: NULL x, w, y or scales", fn);
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned16(qx) || !aligned16(qw))
    return fail(FP8_ERR_ALIGN, "%s: x, w, y, qx and qw must be 16-byte aligned", fn);
  return hip_status(fp8lin::launch_linear_current_small(
                        static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), (int)M,
                        (int)N, (int)K, static_cast<uint16_t*>(y), scales,
                        static_cast<uint8_t*>(qx), static_cast<uint8_t*>(qw), as_stream(stream)),
                    fn);
}

int fp8_linear_fwd_bias(const void* qx, const void* qw, const float* sx, const float* sw,
                        const void* bias, void* y, int64_t M, int64_t N, int64_t K,
                        int64_t M_valid, int gran, void* stream) {
  const char* fn = "fp8_linear_fwd_bias";
  if (bias == nullptr)
    return fp8_linear_fwd(qx, qw, sx, sw, y, M, N, K, M_valid, gran, stream);
  if (gran & FP8_A_E5M2)
    return fail(FP8_ERR_UNSUPPORTED, "%s: the bias epilogue takes e4m3 operands", fn);
  int e = check_gemm(fn, qx, qw, sx, sw, y, M, N, K, M_valid, gran, false);
  if (e) return e;
  if (gran != FP8_TENSORWISE)
    return fail(FP8_ERR_UNSUPPORTED, "%s: the bias epilogue is for FP8_TENSORWISE", fn);
  if (!aligned16(bias)) return fail(FP8_ERR_ALIGN, "%s: bias must be 16-byte aligned", fn);
  return hip_status(fp8lin::launch_gemm_fp8(static_cast<const uint8_t*>(qx),
                                            static_cast<const uint8_t*>(qw), sx, sw,
                                            static_cast<const uint16_t*>(bias),
                                            static_cast<uint16_t*>(y), M, N, K, M_valid, false,
                                            128, false, as_stream(stream)),
                    fn);
}

int fp8_bias_grad(const void* g, int64_t rows, int64_t cols, int64_t rows_valid, void* db,
                  void* stream) {
  const char* fn = "fp8_bias_grad";
  if (rows < 0 || cols < 0) return fail(FP8_ERR_SHAPE, "%s: negative size", fn);
  if (cols % 16) return fail(FP8_ERR_SHAPE, "%s: cols=%lld not a multiple of 16", fn,
                             (long long)cols);
  if (rows_valid < 0 || rows_valid > rows)
    return fail(FP8_ERR_SHAPE, "%s: rows_valid=%lld outside [0, %lld]", fn,
                (long long)rows_valid, (long long)rows);
  if (cols > 0 && !db) return fail(FP8_ERR_NULL, "%s: db is NULL", fn);
  if (rows_valid > 0 && cols > 0 && !g) return fail(FP8_ERR_NULL, "%s: g is NULL", fn);
  if (!aligned16(g)) return fail(FP8_ERR_ALIGN, "%s: g must be 16-byte aligned", fn);
  if (rows * cols * 2 >= kMaxOperandBytes)
    return fail(FP8_ERR_UNSUPPORTED, "%s: g holds 2^31 bytes or more", fn);
  return hip_status(fp8lin::launch_bias_grad(static_cast<const uint16_t*>(g), rows, cols,
                                             rows_valid, static_cast<uint16_t*>(db),
                                             as_stream(stream)),
                    fn);
}

int fp8_linear_dgrad(const void* qg, const void* qw_t, const float* sg, const float* sw, void* dx,
                     int64_t M, int64_t N, int64_t K, int64_t M_valid, int gran, void* stream) {
  const bool a5 = (gran & FP8_A_E5M2) != 0;
  gran &= ~FP8_A_E5M2;
  int e = check_gemm("fp8_linear_dgrad", qg, qw_t, sg, sw, dx, M, K, N, M_valid, gran, a5);
  if (e) return e;
  if (gran == FP8_BLOCK_1x128 && K % 128)
    return fail(FP8_ERR_SHAPE, "fp8_linear_dgrad: block recipe needs K %% 128 == 0");
  return hip_status(fp8lin::launch_gemm_fp8(static_cast<const uint8_t*>(qg),
                                            static_cast<const uint8_t*>(qw_t), sg, sw, nullptr,
                                            static_cast<uint16_t*>(dx), M, K, N, M_valid,
                                            gran == FP8_BLOCK_1x128, 128, a5, as_stream(stream)),
                    "fp8_linear_dgrad");
}

int fp8_linear_wgrad(const void* qg_t, const void* qx_t, const float* sg, const float* sx, void* dw,
                     int64_t M, int64_t N, int64_t K, int gran, void* stream) {
  const bool a5 = (gran & FP8_A_E5M2) != 0;
  gran &= ~FP8_A_E5M2;
  int e = check_gemm("fp8_linear_wgrad", qg_t, qx_t, sg, sx, dw, N, K, M, N, gran, a5);
  if (e) return e;
  return hip_status(fp8lin::launch_gemm_fp8(static_cast<const uint8_t*>(qg_t),
                                            static_cast<const uint8_t*>(qx_t), sg, sx, nullptr,
                                            static_cast<uint16_t*>(dw), N, K, M, N,
                                            gran == FP8_BLOCK_1x128, 1, a5, as_stream(stream)),
                    "fp8_linear_wgrad");
}

int fp8_pad_tokens(const void* x, int64_t T, int64_t cols, int32_t multiple, void* x_pad,
                   int64_t* T_pad, void* stream) {
  const char* fn = "fp8_pad_tokens";
  if (!T_pad) return fail(FP8_ERR_NULL, "%s: T_pad is NULL", fn);
  if (T < 0 || cols < 0) return fail(FP8_ERR_SHAPE, "%s: negative size", fn);
  if (multiple < 1) return fail(FP8_ERR_SHAPE, "%s: multiple=%d must be >= 1", fn, multiple);
  const int64_t pad = ((-T) % multiple + multiple) % multiple;
  *T_pad = T + pad;
  if (!x_pad) return ok();
  if (T * cols > 0 && !x) return fail(FP8_ERR_NULL, "%s: x is NULL", fn);
  return hip_status(fp8lin::launch_pad_tokens(static_cast<const uint16_t*>(x), T, cols, *T_pad,
                                              static_cast<uint16_t*>(x_pad), as_stream(stream)),
                    fn);
}

int fp8_align_multiple(int layout, int64_t batch, int32_t tp, int32_t cp, int32_t base,
                       int32_t* seq_multiple, int32_t* total_multiple) {
  const char* fn = "fp8_align_multiple";
  if (!seq_multiple || !total_multiple) return fail(FP8_ERR_NULL, "%s: NULL output", fn);
  if (batch < 1 || tp < 1 || cp < 1 || base < 1)
    return fail(FP8_ERR_SHAPE, "%s: batch, tp, cp and base must be positive", fn);
  auto gcd = [](int64_t a, int64_t b) {
    while (b) { const int64_t t = a % b; a = b; b = t; }
    return a;
  };
  int64_t seq = 1, total = 1;
  if (layout == FP8_LAYOUT_THD) {
    seq = cp > 1 ? 2 * (int64_t)cp : 1;
    total = (int64_t)base * cp * tp;
  } else if (layout == FP8_LAYOUT_BSHD) {
    if (cp != 1)
      return fail(FP8_ERR_UNSUPPORTED, "%s: BSHD alignment covers tensor/sequence parallelism only",
                  fn);
    const int64_t bt = (int64_t)base * tp;
    const int64_t need = bt / gcd(batch, bt);
    seq = tp / gcd(tp, need) * need;                  // lcm(tp, need)
  } else {
    return fail(FP8_ERR_UNSUPPORTED, "%s: unknown layout %d", fn, layout);
  }
  if (seq > 0x7FFFFFFF || total > 0x7FFFFFFF)
    return fail(FP8_ERR_SHAPE, "%s: multiple does not fit 32 bits", fn);
  *seq_multiple = (int32_t)seq;
  *total_multiple = (int32_t)total;
  return ok();
}

namespace {

// cu: nseq + 1 non-decreasing host offsets starting at 0.
int check_offsets(const char* fn, const int64_t* cu, int32_t nseq, const char* what) {
  if (!cu) return fail(FP8_ERR_NULL, "%s: %s is NULL", fn, what);
  if (cu[0] != 0) return fail(FP8_ERR_SHAPE, "%s: %s[0] must be 0", fn, what);
  for (int32_t i = 0; i < nseq; ++i)
    if (cu[i + 1] < cu[i])
      return fail(FP8_ERR_SHAPE, "%s: %s decreases at %d", fn, what, i);
  return FP8_OK;
}

}  // namespace

int fp8_pad_varlen(const void* x, const int64_t* cu_seqlens, int32_t nseq, int64_t cols,
                   int32_t seq_multiple, int32_t total_multiple, void* x_pad,
                   int64_t* cu_seqlens_pad, int64_t* T_pad, void* stream) {
  const char* fn = "fp8_pad_varlen";
  if (!T_pad) return fail(FP8_ERR_NULL, "%s: T_pad is NULL", fn);
  if (nseq < 0 || cols < 0) return fail(FP8_ERR_SHAPE, "%s: negative size", fn);
  if (seq_multiple < 1 || total_multiple < 1)
    return fail(FP8_ERR_SHAPE, "%s: multiples must be >= 1", fn);
  if (cols % 16) return fail(FP8_ERR_SHAPE, "%s: cols=%lld not a multiple of 16", fn, (long long)cols);
  int e = check_offsets(fn, cu_seqlens, nseq, "cu_seqlens");
  if (e) return e;
  // padded offsets on the host
  int64_t end = 0;
  int64_t* pad_off = cu_seqlens_pad;
  for (int32_t i = 0; i <= nseq; ++i) {
    if (i > 0) {
      const int64_t len = cu_seqlens[i] - cu_seqlens[i - 1];
      end += len + ((-len) % seq_multiple + seq_multiple) % seq_multiple;
    }
    if (pad_off) pad_off[i] = end;
  }
  *T_pad = end + ((-end) % total_multiple + total_multiple) % total_multiple;
  if (!x_pad) return ok();
  if (!pad_off) return fail(FP8_ERR_NULL, "%s: cu_seqlens_pad is needed with x_pad", fn);
  if (*T_pad == 0 || cols == 0) return ok();                 // nothing to write
  if (x == x_pad) return fail(FP8_ERR_UNSUPPORTED, "%s: x_pad must not be x", fn);
  if (cu_seqlens[nseq] * cols > 0 && !x) return fail(FP8_ERR_NULL, "%s: x is NULL", fn);
  if (!aligned16(x) || !aligned16(x_pad))
    return fail(FP8_ERR_ALIGN, "%s: x and x_pad must be 16-byte aligned", fn);
  return hip_status(fp8lin::launch_pad_varlen(true, static_cast<const uint16_t*>(x),
                                              static_cast<uint16_t*>(x_pad), cols, cu_seqlens,
                                              pad_off, nseq, *T_pad, as_stream(stream)),
                    fn);
}

int fp8_unpad_varlen(const void* x_pad, const int64_t* cu_seqlens, const int64_t* cu_seqlens_pad,
                     int32_t nseq, int64_t cols, void* x, void* stream) {
  const char* fn = "fp8_unpad_varlen";
  if (nseq < 0 || cols < 0) return fail(FP8_ERR_SHAPE, "%s: negative size", fn);
  if (cols % 16) return fail(FP8_ERR_SHAPE, "%s: cols=%lld not a multiple of 16", fn, (long long)cols);
  int e = check_offsets(fn, cu_seqlens, nseq, "cu_seqlens");
  if (e) return e;
  e = check_offsets(fn, cu_seqlens_pad, nseq, "cu_seqlens_pad");
  if (e) return e;
  for (int32_t i = 0; i < nseq; ++i)
    if (cu_seqlens_pad[i + 1] - cu_seqlens_pad[i] < cu_seqlens[i + 1] - cu_seqlens[i])
      return fail(FP8_ERR_SHAPE, "%s: padded sequence %d is shorter than the sequence", fn, i);
  if (cu_seqlens[nseq] * cols == 0) return ok();
  if (!x || !x_pad) return fail(FP8_ERR_NULL, "%s: NULL tensor", fn);
  if (x == x_pad) return fail(FP8_ERR_UNSUPPORTED, "%s: x must not be x_pad", fn);
  if (!aligned16(x) || !aligned16(x_pad))
    return fail(FP8_ERR_ALIGN, "%s: x and x_pad must be 16-byte aligned", fn);
  return hip_status(fp8lin::launch_pad_varlen(false, static_cast<const uint16_t*>(x_pad),
                                              static_cast<uint16_t*>(x), cols, cu_seqlens,
                                              cu_seqlens_pad, nseq, cu_seqlens_pad[nseq],
                                              as_stream(stream)),
                    fn);
}

namespace {

int64_t elem_bytes(int dtype) { return dtype == FP8_DT_F32 ? 4 : 2; }

bool aligned_to(const void* p, int64_t n) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(n - 1)) == 0;
}

int check_dtype(const char* fn, int dtype) {
  if (dtype != FP8_DT_BF16 && dtype != FP8_DT_F16 && dtype != FP8_DT_F32)
    return fail(FP8_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  return FP8_OK;
}

// A [rows, cols] input with row stride ld.
int check_rows(const char* fn, const char* what, const void* p, int64_t ld, int64_t rows,
               int64_t cols, int dtype) {
  if (ld < cols)
    return fail(FP8_ERR_SHAPE, "%s: row stride %lld of %s is below its %lld columns", fn,
                (long long)ld, what, (long long)cols);
  if (rows > 1 && ld > (INT64_MAX >> 3) / rows)
    return fail(FP8_ERR_SHAPE, "%s: %s does not fit 64-bit addresses", fn, what);
  if (rows * cols > 0 && !p) return fail(FP8_ERR_NULL, "%s: %s is NULL", fn, what);
  if (!aligned_to(p, elem_bytes(dtype)))
    return fail(FP8_ERR_ALIGN, "%s: %s is not aligned to its elements", fn, what);
  return FP8_OK;
}

int check_layernorm(const char* fn, int64_t rows, int64_t cols, int dtype, int param_dtype) {
  if (rows < 0 || cols < 1)
    return fail(FP8_ERR_SHAPE, "%s: needs rows >= 0 and cols >= 1 (got %lld x %lld)", fn,
                (long long)rows, (long long)cols);
  if (cols > fp8lin::kLayerNormMaxCols)
    return fail(FP8_ERR_UNSUPPORTED, "%s: %lld columns, the limit is %lld", fn, (long long)cols,
                (long long)fp8lin::kLayerNormMaxCols);
  if (rows >= ((int64_t)1 << 31))
    return fail(FP8_ERR_UNSUPPORTED, "%s: 2^31 rows or more", fn);
  if (int e = check_dtype(fn, dtype)) return e;
  if (param_dtype != dtype && param_dtype != FP8_DT_F32)
    return fail(FP8_ERR_UNSUPPORTED, "%s: parameters must have the rows' dtype or be f32", fn);
  return FP8_OK;
}

int check_moe_sizes(const char* fn, int64_t tokens, int32_t topk) {
  if (tokens < 0) return fail(FP8_ERR_SHAPE, "%s: negative token count", fn);
  if (topk < 1 || topk > fp8lin::kMoeMaxTopk)
    return fail(FP8_ERR_SHAPE, "%s: topk=%d outside [1, %d]", fn, topk, fp8lin::kMoeMaxTopk);
  if (tokens >= ((int64_t)1 << 31) || tokens * topk >= ((int64_t)1 << 31))
    return fail(FP8_ERR_UNSUPPORTED, "%s: 2^31 token-expert pairs or more", fn);
  return FP8_OK;
}

int check_experts(const char* fn, int32_t experts) {
  if (experts < 1 || experts > fp8lin::kMoeMaxExperts)
    return fail(FP8_ERR_SHAPE, "%s: experts=%d outside [1, %d]", fn, experts,
                fp8lin::kMoeMaxExperts);
  return FP8_OK;
}

int moe_rows(const char* fn, int64_t tokens, int32_t topk, int32_t experts, int32_t multiple,
             int64_t* rows) {
  if (int e = check_moe_sizes(fn, tokens, topk)) return e;
  if (int e = check_experts(fn, experts)) return e;
  if (multiple < 1) return fail(FP8_ERR_SHAPE, "%s: multiple=%d", fn, multiple);
  const int64_t pairs = tokens * topk;
  const int64_t used = pairs < experts ? pairs : experts;
  const int64_t r = (pairs + used * (multiple - 1)) / multiple * multiple;
  if (r >= ((int64_t)1 << 31)) return fail(FP8_ERR_UNSUPPORTED, "%s: 2^31 sorted rows or more", fn);
  *rows = r;
  return FP8_OK;
}

// Sizes and index tensors of the row exchanges.
int check_exchange(const char* fn, int64_t tokens, int32_t topk, int64_t rows, int64_t cols,
                   int dtype, const int32_t* slot, const int32_t* source, bool need_source) {
  if (int e = check_moe_sizes(fn, tokens, topk)) return e;
  if (rows < 0 || cols < 0) return fail(FP8_ERR_SHAPE, "%s: negative size", fn);
  if (int e = check_dtype(fn, dtype)) return e;
  const int64_t limit = (int64_t)1 << 24;
  if (rows >= ((int64_t)1 << 31) || cols >= ((int64_t)1 << 30) ||
      (tokens + rows) * ((cols * elem_bytes(dtype) + 2047) / 2048) >= limit ||
      tokens + rows >= limit)
    return fail(FP8_ERR_UNSUPPORTED,
                "%s: (tokens + rows) * ceil(row bytes / 2048) must be below 2^24", fn);
  if (tokens > 0 && !slot) return fail(FP8_ERR_NULL, "%s: slot is NULL", fn);
  if (need_source && rows > 0 && !source) return fail(FP8_ERR_NULL, "%s: source is NULL", fn);
  if (!aligned_to(slot, 4) || !aligned_to(source, 4))
    return fail(FP8_ERR_ALIGN, "%s: slot and source must be 4-byte aligned", fn);
  return FP8_OK;
}

int check_out(const char* fn, const char* what, const void* p, int64_t n, int64_t align) {
  if (n > 0 && !p) return fail(FP8_ERR_NULL, "%s: %s is NULL", fn, what);
  if (!aligned_to(p, align))
    return fail(FP8_ERR_ALIGN, "%s: %s is not aligned to its elements", fn, what);
  return FP8_OK;
}

int check_workspace(const char* fn, const void* p, int64_t have, int64_t need) {
  if (need == 0) return FP8_OK;
  if (!p) return fail(FP8_ERR_NULL, "%s: workspace is NULL, needs %lld bytes", fn, (long long)need);
  if (have < need)
    return fail(FP8_ERR_SHAPE, "%s: workspace of %lld bytes, needs %lld", fn, (long long)have,
                (long long)need);
  if (!aligned_to(p, 4)) return fail(FP8_ERR_ALIGN, "%s: workspace must be 4-byte aligned", fn);
  return FP8_OK;
}

}  // namespace

int fp8_layernorm_fwd(const void* x, int64_t ldx, const void* gamma, const void* beta,
                      int64_t rows, int64_t cols, int dtype, int param_dtype, float eps, void* y,
                      float* mean, float* rstd, void* stream) {
  const char* fn = "fp8_layernorm_fwd";
  if (int e = check_layernorm(fn, rows, cols, dtype, param_dtype)) return e;
  if (!(eps >= 0.f) || eps > 3.402823466e38f)
    return fail(FP8_ERR_SHAPE, "%s: eps must be finite and not negative", fn);
  if (int e = check_rows(fn, "x", x, ldx, rows, cols, dtype)) return e;
  if (int e = check_out(fn, "y", y, rows, elem_bytes(dtype))) return e;
  if (x && x == y) return fail(FP8_ERR_UNSUPPORTED, "%s: y must not be x", fn);
  if (!aligned_to(gamma, elem_bytes(param_dtype)) || !aligned_to(beta, elem_bytes(param_dtype)) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return fail(FP8_ERR_ALIGN, "%s: a parameter or statistic is not aligned to its elements", fn);
  if (rows == 0) return ok();
  fp8lin::LayerNormArgs a{};
  a.x = x, a.ldx = ldx, a.gamma = gamma, a.beta = beta, a.rows = rows, a.cols = cols;
  a.dtype = dtype, a.param_dtype = param_dtype, a.eps = eps, a.y = y, a.mean = mean, a.rstd = rstd;
  return hip_status(fp8lin::launch_layernorm(a, false, as_stream(stream)), fn);
}

int fp8_layernorm_bwd_workspace(int64_t rows, int64_t cols, int64_t* bytes) {
  const char* fn = "fp8_layernorm_bwd_workspace";
  if (!bytes) return fail(FP8_ERR_NULL, "%s: bytes is NULL", fn);
  if (int e = check_layernorm(fn, rows, cols, FP8_DT_F32, FP8_DT_F32)) return e;
  *bytes = fp8lin::layernorm_bwd_workspace(rows, cols);
  return ok();
}

int fp8_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx, const float* mean,
                      const float* rstd, const void* gamma, int64_t rows, int64_t cols, int dtype,
                      int param_dtype, void* dx, void* dgamma, void* dbeta, void* workspace,
                      int64_t workspace_bytes, void* stream) {
  const char* fn = "fp8_layernorm_bwd";
  if (int e = check_layernorm(fn, rows, cols, dtype, param_dtype)) return e;
  if (int e = check_rows(fn, "dy", dy, lddy, rows, cols, dtype)) return e;
  if (int e = check_rows(fn, "x", x, ldx, rows, cols, dtype)) return e;
  if (rows > 0 && (!mean || !rstd)) return fail(FP8_ERR_NULL, "%s: mean or rstd is NULL", fn);
  if (!aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dx, elem_bytes(dtype)) ||
      !aligned_to(gamma, elem_bytes(param_dtype)) || !aligned_to(dgamma, elem_bytes(param_dtype)) ||
      !aligned_to(dbeta, elem_bytes(param_dtype)))
    return fail(FP8_ERR_ALIGN, "%s: a tensor is not aligned to its elements", fn);
  if (dx && (dx == x || dx == dy))
    return fail(FP8_ERR_UNSUPPORTED, "%s: dx must not be an input", fn);
  if (!dx && !dgamma && !dbeta) return ok();
  if (rows == 0 && !dgamma && !dbeta) return ok();
  const int64_t need = (dgamma || dbeta) ? fp8lin::layernorm_bwd_workspace(rows, cols) : 0;
  if (int e = check_workspace(fn, workspace, workspace_bytes, need)) return e;
  fp8lin::LayerNormArgs a{};
  a.x = x, a.ldx = ldx, a.dy = dy, a.lddy = lddy, a.gamma = gamma, a.rows = rows, a.cols = cols;
  a.dtype = dtype, a.param_dtype = param_dtype, a.y = dx, a.dgamma = dgamma, a.dbeta = dbeta;
  a.mean = const_cast<float*>(mean), a.rstd = const_cast<float*>(rstd);
  a.workspace = need ? static_cast<float*>(workspace) : nullptr;
  return hip_status(fp8lin::launch_layernorm(a, true, as_stream(stream)), fn);
}

int fp8_moe_rows(int64_t tokens, int32_t topk, int32_t experts, int32_t multiple, int64_t* rows) {
  const char* fn = "fp8_moe_rows";
  if (!rows) return fail(FP8_ERR_NULL, "%s: rows is NULL", fn);
  if (int e = moe_rows(fn, tokens, topk, experts, multiple, rows)) return e;
  return ok();
}

int fp8_moe_sort_workspace(int64_t tokens, int32_t topk, int32_t experts, int64_t* bytes) {
  const char* fn = "fp8_moe_sort_workspace";
  if (!bytes) return fail(FP8_ERR_NULL, "%s: bytes is NULL", fn);
  if (int e = check_moe_sizes(fn, tokens, topk)) return e;
  if (int e = check_experts(fn, experts)) return e;
  *bytes = fp8lin::moe_sort_workspace(tokens * topk, experts);
  return ok();
}

int fp8_moe_sort(const void* expert_idx, int idx_bytes, int64_t tokens, int32_t topk,
                 int32_t experts, int32_t multiple, int32_t* slot, int32_t* source,
                 int32_t* counts, int32_t* offsets, void* workspace, int64_t workspace_bytes,
                 void* stream) {
  const char* fn = "fp8_moe_sort";
  int64_t rows = 0;
  if (int e = moe_rows(fn, tokens, topk, experts, multiple, &rows)) return e;
  if (idx_bytes != 4 && idx_bytes != 8)
    return fail(FP8_ERR_UNSUPPORTED, "%s: expert indices of %d bytes (4 or 8)", fn, idx_bytes);
  const int64_t pairs = tokens * topk;
  if (int e = check_out(fn, "expert_idx", expert_idx, pairs, idx_bytes)) return e;
  if (int e = check_out(fn, "slot", slot, pairs, 4)) return e;
  if (int e = check_out(fn, "source", source, rows, 4)) return e;
  if (int e = check_out(fn, "counts", counts, experts, 4)) return e;
  if (int e = check_out(fn, "offsets", offsets, experts + 1, 4)) return e;
  const int64_t need = fp8lin::moe_sort_workspace(pairs, experts);
  if (int e = check_workspace(fn, workspace, workspace_bytes, need)) return e;
  fp8lin::MoeSortArgs a{};
  a.idx = expert_idx, a.idx_bytes = idx_bytes, a.pairs = pairs, a.rows = rows;
  a.experts = experts, a.multiple = multiple, a.slot = slot, a.source = source;
  a.counts = counts, a.offsets = offsets, a.workspace = static_cast<int32_t*>(workspace);
  return hip_status(fp8lin::launch_moe_sort(a, as_stream(stream)), fn);
}

int fp8_moe_dispatch(const void* x, int64_t ldx, const int32_t* slot, const int32_t* source,
                     int64_t tokens, int32_t topk, int64_t rows, int64_t cols, int dtype, void* xs,
                     void* stream) {
  const char* fn = "fp8_moe_dispatch";
  if (int e = check_exchange(fn, tokens, topk, rows, cols, dtype, slot, source, true)) return e;
  if (int e = check_rows(fn, "x", x, ldx, tokens, cols, dtype)) return e;
  if (int e = check_out(fn, "xs", xs, rows * cols, elem_bytes(dtype))) return e;
  if (rows * cols == 0) return ok();
  if (x == xs) return fail(FP8_ERR_UNSUPPORTED, "%s: xs must not be x", fn);
  fp8lin::MoeArgs a{};
  a.x = x, a.ldx = ldx, a.slot = slot, a.source = source, a.tokens = tokens, a.topk = topk;
  a.rows = rows, a.cols = cols, a.dtype = dtype, a.out = xs;
  return hip_status(fp8lin::launch_moe_dispatch(a, as_stream(stream)), fn);
}

namespace {

int combine(const char* fn, const char* in, const char* out, const void* ys, int64_t ldys,
            const int32_t* slot, const float* weights, int64_t tokens, int32_t topk, int64_t rows,
            int64_t cols, int dtype, void* y, void* stream) {
  if (int e = check_exchange(fn, tokens, topk, rows, cols, dtype, slot, nullptr, false)) return e;
  if (int e = check_rows(fn, in, ys, ldys, rows, cols, dtype)) return e;
  if (int e = check_out(fn, out, y, tokens * cols, elem_bytes(dtype))) return e;
  if (tokens * cols == 0) return ok();
  if (ys == y) return fail(FP8_ERR_UNSUPPORTED, "%s: %s must not be %s", fn, out, in);
  fp8lin::MoeArgs a{};
  a.ys = ys, a.ldys = ldys, a.slot = slot, a.weights = weights, a.tokens = tokens, a.topk = topk;
  a.rows = rows, a.cols = cols, a.dtype = dtype, a.out = y;
  return hip_status(fp8lin::launch_moe_combine(a, as_stream(stream)), fn);
}

}  // namespace

int fp8_moe_dispatch_bwd(const void* dxs, int64_t lddxs, const int32_t* slot, int64_t tokens,
                         int32_t topk, int64_t rows, int64_t cols, int dtype, void* dx,
                         void* stream) {
  return combine("fp8_moe_dispatch_bwd", "dxs", "dx", dxs, lddxs, slot, nullptr, tokens, topk,
                 rows, cols, dtype, dx, stream);
}

int fp8_moe_combine(const void* ys, int64_t ldys, const int32_t* slot, const float* weights,
                    int64_t tokens, int32_t topk, int64_t rows, int64_t cols, int dtype, void* y,
                    void* stream) {
  const char* fn = "fp8_moe_combine";
  if (tokens > 0 && !weights) return fail(FP8_ERR_NULL, "%s: weights is NULL", fn);
  if (!aligned_to(weights, 4)) return fail(FP8_ERR_ALIGN, "%s: weights must be 4-byte aligned", fn);
  return combine(fn, "ys", "y", ys, ldys, slot, weights, tokens, topk, rows, cols, dtype, y, stream);
}

int fp8_moe_combine_bwd(const void* dy, int64_t lddy, const void* ys, int64_t ldys,
                        const int32_t* slot, const int32_t* source, const float* weights,
                        int64_t tokens, int32_t topk, int64_t rows, int64_t cols, int dtype,
                        void* dys, float* dw, void* stream) {
  const char* fn = "fp8_moe_combine_bwd";
  if (int e = check_exchange(fn, tokens, topk, rows, cols, dtype, slot, source, true)) return e;
  if (tokens > 0 && !weights) return fail(FP8_ERR_NULL, "%s: weights is NULL", fn);
  if (!aligned_to(weights, 4)) return fail(FP8_ERR_ALIGN, "%s: weights must be 4-byte aligned", fn);
  if (int e = check_rows(fn, "dy", dy, lddy, tokens, cols, dtype)) return e;
  if (int e = check_rows(fn, "ys", ys, ldys, rows, cols, dtype)) return e;
  if (int e = check_out(fn, "dys", dys, rows * cols, elem_bytes(dtype))) return e;
  if (int e = check_out(fn, "dw", dw, tokens * topk, 4)) return e;
  if (tokens == 0 && rows * cols == 0) return ok();
  if (dys && (dys == dy || dys == ys))
    return fail(FP8_ERR_UNSUPPORTED, "%s: dys must not be an input", fn);
  fp8lin::MoeArgs a{};
  a.x = dy, a.ldx = lddy, a.ys = ys, a.ldys = ldys, a.slot = slot, a.source = source;
  a.weights = weights, a.tokens = tokens, a.topk = topk, a.rows = rows, a.cols = cols;
  a.dtype = dtype, a.out = dys, a.dw = dw;
  return hip_status(fp8lin::launch_moe_combine_bwd(a, as_stream(stream)), fn);
}

namespace {

int check_route(const char* fn, const void* logits, int64_t ldl, int64_t tokens, int64_t valid,
                int32_t experts, int32_t topk, int dtype) {
  if (int e = check_moe_sizes(fn, tokens, topk)) return e;
  if (int e = check_experts(fn, experts)) return e;
  if (topk > experts)
    return fail(FP8_ERR_SHAPE, "%s: topk=%d of %d experts", fn, topk, experts);
  if (valid < 0 || valid > tokens)
    return fail(FP8_ERR_SHAPE, "%s: tokens_valid=%lld outside [0, %lld]", fn, (long long)valid,
                (long long)tokens);
  if (int e = check_dtype(fn, dtype)) return e;
  return check_rows(fn, "logits", logits, ldl, tokens, experts, dtype);
}

// A pair of outputs (or inputs) of which both or none are given.
int check_pair(const char* fn, const char* what, const void* codes, const float* scale,
               int64_t n) {
  if (n > 0 && (codes == nullptr) != (scale == nullptr))
    return fail(FP8_ERR_NULL, "%s: %s and its scales must both be given or both be NULL", fn, what);
  if (!aligned16(codes) || !aligned_to(scale, 4))
    return fail(FP8_ERR_ALIGN, "%s: %s must be 16-byte aligned and its scales 4-byte", fn, what);
  return FP8_OK;
}

// Memory of a tensor: rows of `bytes` each, `pitch` apart (one row: dense).
struct Region {
  const char* what;
  const void* p;
  int64_t bytes, rows = 1, pitch = 0;
};

// Whether the dense region d shares a byte with one of the rows of s.
bool meet(const Region& d, const Region& s) {
  if (!d.p || !s.p || d.bytes <= 0 || s.bytes <= 0 || s.rows <= 0) return false;
  const int64_t at = static_cast<int64_t>(reinterpret_cast<uintptr_t>(d.p)) -
                     static_cast<int64_t>(reinterpret_cast<uintptr_t>(s.p));
  // the first row of s that ends behind d's start
  const int64_t r = at < s.bytes ? 0 : s.rows > 1 ? (at - s.bytes) / s.pitch + 1 : 1;
  return r < s.rows && r * s.pitch < at + d.bytes;
}

// Outputs are written by workgroups while others still read the inputs, so none of them (all dense)
// may share memory with an input or another output.
int check_apart(const char* fn, std::initializer_list<Region> outs,
                std::initializer_list<Region> ins) {
  for (const Region* o = outs.begin(); o != outs.end(); ++o) {
    for (const Region& i : ins)
      if (meet(*o, i))
        return fail(FP8_ERR_UNSUPPORTED, "%s: %s shares memory with %s", fn, o->what, i.what);
    for (const Region* q = outs.begin(); q != o; ++q)
      if (meet(*o, *q))
        return fail(FP8_ERR_UNSUPPORTED, "%s: %s shares memory with %s", fn, o->what, q->what);
  }
  return FP8_OK;
}

constexpr int64_t kMaxGroupedRows = (int64_t)1 << 23;

int check_act(const char* fn, int64_t rows, int64_t valid, int64_t cols, int act, int dtype) {
  if (rows < 0 || cols < 1 || cols % 128)
    return fail(FP8_ERR_SHAPE, "%s: needs rows >= 0 and cols a positive multiple of 128 (got %lld x "
                "%lld)", fn, (long long)rows, (long long)cols);
  if (rows >= kMaxGroupedRows || cols >= kMaxContraction)
    return fail(FP8_ERR_UNSUPPORTED, "%s: 2^23 rows or 2^17 columns or more", fn);
  // a workgroup of 512 threads a tile, in sixty-fours, and fewer than 2^32 threads in a launch
  if ((rows + 127) / 128 * (cols / 128) > ((int64_t)1 << 23) - 64)
    return fail(FP8_ERR_UNSUPPORTED, "%s: more than 2^23 - 64 tiles of 128 x 128", fn);
  if (valid < 0 || valid > rows)
    return fail(FP8_ERR_SHAPE, "%s: rows_valid=%lld outside [0, %lld]", fn, (long long)valid,
                (long long)rows);
  if (act != FP8_ACT_RELU && act != FP8_ACT_SILU && act != FP8_ACT_GELU)
    return fail(FP8_ERR_UNSUPPORTED, "%s: unknown activation %d", fn, act);
  return check_dtype(fn, dtype);
}

int check_grouped(const char* fn, const int32_t* offsets, const int32_t* counts, int32_t experts,
                  int64_t rows, int64_t N, int64_t K) {
  if (int e = check_experts(fn, experts)) return e;
  if (rows < 0 || N < 1 || K < 1 || N % 128 || K % 128)
    return fail(FP8_ERR_SHAPE, "%s: needs rows >= 0 and N, K positive multiples of 128 (got %lld x "
                "%lld x %lld)", fn, (long long)rows, (long long)N, (long long)K);
  if (rows >= kMaxGroupedRows || N >= kMaxContraction || K >= kMaxContraction)
    return fail(FP8_ERR_UNSUPPORTED, "%s: 2^23 rows, or N or K of 2^17, or more", fn);
  if (!offsets || !counts) return fail(FP8_ERR_NULL, "%s: offsets or counts is NULL", fn);
  if (!aligned_to(offsets, 4) || !aligned_to(counts, 4))
    return fail(FP8_ERR_ALIGN, "%s: offsets and counts must be 4-byte aligned", fn);
  return FP8_OK;
}

// y [rows, N] over contraction length K.
int grouped(const char* fn, const void* x, const void* w, int64_t ldw, int64_t stride_w,
            const float* sx, const float* sw, int64_t ldsw, int64_t stride_sw,
            const int32_t* offsets, const int32_t* counts, int32_t experts, int64_t rows,
            int64_t N, int64_t K, int64_t max_rows, void* y, void* stream) {
  if (int e = check_grouped(fn, offsets, counts, experts, rows, N, K)) return e;
  if (ldw < K || ldw % 16 || stride_w < 0 || stride_w % 16)
    return fail(FP8_ERR_SHAPE, "%s: weight strides %lld and %lld (rows of %lld codes, multiples of "
                "16)", fn, (long long)stride_w, (long long)ldw, (long long)K);
  if (ldsw < K / 128 || stride_sw < 0)
    return fail(FP8_ERR_SHAPE, "%s: scale strides %lld and %lld (rows of %lld scales)", fn,
                (long long)stride_sw, (long long)ldsw, (long long)(K / 128));
  if (ldw >= kMaxGroupedRows || ldsw >= kMaxGroupedRows ||
      stride_w > (INT64_MAX >> 10) || stride_sw > (INT64_MAX >> 12))
    return fail(FP8_ERR_UNSUPPORTED, "%s: a row stride of 2^23 or more, or experts too far apart",
                fn);
  if (max_rows < 0) return fail(FP8_ERR_SHAPE, "%s: max_rows=%lld", fn, (long long)max_rows);
  if (rows == 0) return ok();
  if (!x || !w || !sx || !sw || !y) return fail(FP8_ERR_NULL, "%s: NULL operand or scale pointer", fn);
  if (!aligned16(x) || !aligned16(w) || !aligned16(y) || !aligned_to(sx, 4) || !aligned_to(sw, 4))
    return fail(FP8_ERR_ALIGN, "%s: operands and output must be 16-byte aligned, scales 4-byte", fn);
  if (int e = check_apart(fn, {{"the output", y, 2 * rows * N}},
                          {{"the codes", x, rows * K}, {"their scales", sx, rows * K / 32},
                           {"offsets", offsets, 4 * ((int64_t)experts + 1)},
                           {"counts", counts, 4 * (int64_t)experts}}))
    return e;
  // the experts' rows may alternate in memory (ldw above stride_w): one by one if y is among them
  const Region out = {"", y, 2 * rows * N};
  const int64_t far = experts - 1;
  if (meet(out, {"", w, far * stride_w + (N - 1) * ldw + K}) ||
      meet(out, {"", sw, 4 * (far * stride_sw + (N / 128 - 1) * ldsw + K / 128)}))
    for (int64_t i = 0; i < experts; ++i)
      if (int e = check_apart(fn, {{"the output", y, 2 * rows * N}},
                              {{"the weights", static_cast<const uint8_t*>(w) + i * stride_w, K, N, ldw},
                               {"their scales", sw + i * stride_sw, K / 32, N / 128, 4 * ldsw}}))
        return e;
  fp8lin::GroupedArgs a{};
  a.x = static_cast<const uint8_t*>(x), a.w = static_cast<const uint8_t*>(w), a.sx = sx, a.sw = sw;
  a.ldw = ldw, a.stride_w = stride_w, a.ldsw = ldsw, a.stride_sw = stride_sw;
  a.offsets = offsets, a.counts = counts, a.experts = experts, a.rows = rows, a.N = N, a.K = K;
  a.max_rows = max_rows < rows ? max_rows : rows;
  a.y = static_cast<uint16_t*>(y);
  return hip_status(fp8lin::launch_grouped_gemm(a, as_stream(stream)), fn);
}

}  // namespace

int fp8_moe_route_workspace(int64_t tokens, int32_t experts, int64_t* bytes) {
  const char* fn = "fp8_moe_route_workspace";
  if (!bytes) return fail(FP8_ERR_NULL, "%s: bytes is NULL", fn);
  if (int e = check_moe_sizes(fn, tokens, 1)) return e;
  if (int e = check_experts(fn, experts)) return e;
  *bytes = fp8lin::moe_route_workspace(tokens, experts);
  return ok();
}

int fp8_moe_route(const void* logits, int64_t ldl, int64_t tokens, int64_t tokens_valid,
                  int32_t experts, int32_t topk, int dtype, int normalize, int32_t* expert_idx,
                  float* weights, float* lse, int32_t* counts, float* losses, void* workspace,
                  int64_t workspace_bytes, void* stream) {
  const char* fn = "fp8_moe_route";
  if (int e = check_route(fn, logits, ldl, tokens, tokens_valid, experts, topk, dtype)) return e;
  if (int e = check_out(fn, "expert_idx", expert_idx, tokens, 4)) return e;
  if (int e = check_out(fn, "weights", weights, tokens, 4)) return e;
  if (int e = check_out(fn, "lse", lse, tokens, 4)) return e;
  if (int e = check_out(fn, "counts", counts, 1, 4)) return e;
  if (int e = check_out(fn, "losses", losses, 1, 4)) return e;
  const int64_t need = fp8lin::moe_route_workspace(tokens, experts);
  if (int e = check_workspace(fn, workspace, workspace_bytes, need)) return e;
  const int64_t eb = elem_bytes(dtype), pairs = 4 * tokens * topk;
  if (int e = check_apart(fn, {{"expert_idx", expert_idx, pairs}, {"weights", weights, pairs},
                               {"lse", lse, 4 * tokens}, {"counts", counts, 4 * experts},
                               {"losses", losses, 8}, {"workspace", workspace, need}},
                          {{"logits", logits, experts * eb, tokens_valid, ldl * eb}}))
    return e;
  fp8lin::MoeRouteArgs a{};
  a.logits = logits, a.ldl = ldl, a.tokens = tokens, a.valid = tokens_valid, a.experts = experts;
  a.topk = topk, a.dtype = dtype, a.normalize = normalize != 0, a.idx = expert_idx;
  a.weights = weights, a.lse = lse, a.counts = counts, a.losses = losses;
  a.workspace = need ? static_cast<float*>(workspace) : nullptr;
  return hip_status(fp8lin::launch_moe_route(a, as_stream(stream)), fn);
}

int fp8_moe_route_bwd(const void* logits, int64_t ldl, const float* lse, const int32_t* expert_idx,
                      const float* weights, const int32_t* counts, const float* dweights,
                      const float* dlosses, int64_t tokens, int64_t tokens_valid, int32_t experts,
                      int32_t topk, int dtype, int normalize, void* dlogits, void* stream) {
  const char* fn = "fp8_moe_route_bwd";
  if (int e = check_route(fn, logits, ldl, tokens, tokens_valid, experts, topk, dtype)) return e;
  if (int e = check_out(fn, "lse", lse, tokens, 4)) return e;
  if (int e = check_out(fn, "expert_idx", expert_idx, tokens, 4)) return e;
  if (int e = check_out(fn, "weights", weights, tokens, 4)) return e;
  if (int e = check_out(fn, "counts", counts, 1, 4)) return e;
  if (!aligned_to(dweights, 4) || !aligned_to(dlosses, 4))
    return fail(FP8_ERR_ALIGN, "%s: dweights and dlosses must be 4-byte aligned", fn);
  if (int e = check_out(fn, "dlogits", dlogits, tokens, elem_bytes(dtype))) return e;
  if (tokens == 0) return ok();
  const int64_t eb = elem_bytes(dtype), pairs = 4 * tokens * topk;
  if (int e = check_apart(fn, {{"dlogits", dlogits, tokens * experts * eb}},
                          {{"logits", logits, experts * eb, tokens_valid, ldl * eb},
                           {"lse", lse, 4 * tokens}, {"expert_idx", expert_idx, pairs},
                           {"weights", weights, pairs}, {"counts", counts, 4 * experts},
                           {"dweights", dweights, pairs}, {"dlosses", dlosses, 8}}))
    return e;
  fp8lin::MoeRouteArgs a{};
  a.logits = logits, a.ldl = ldl, a.tokens = tokens, a.valid = tokens_valid, a.experts = experts;
  a.topk = topk, a.dtype = dtype, a.normalize = normalize != 0;
  a.idx = const_cast<int32_t*>(expert_idx), a.weights = const_cast<float*>(weights);
  a.lse = const_cast<float*>(lse), a.counts = const_cast<int32_t*>(counts);
  a.dweights = dweights, a.dlosses = dlosses, a.dlogits = dlogits;
  return hip_status(fp8lin::launch_moe_route_bwd(a, as_stream(stream)), fn);
}

int fp8_act_quantize(const void* h, int64_t ldh, int64_t rows, int64_t rows_valid, int64_t cols,
                     int act, int gated, int dtype, void* q, float* scale, void* q_t,
                     float* scale_t, void* hq, float* hscale, void* stream) {
  const char* fn = "fp8_act_quantize";
  if (int e = check_act(fn, rows, rows_valid, cols, act, dtype)) return e;
  if (int e = check_rows(fn, "h", h, ldh, rows_valid, gated ? 2 * cols : cols, dtype)) return e;
  if (int e = check_pair(fn, "q", q, scale, rows)) return e;
  if (int e = check_pair(fn, "q_t", q_t, scale_t, rows)) return e;
  if (int e = check_pair(fn, "hq", hq, hscale, rows)) return e;
  if (q_t && rows % 128)
    return fail(FP8_ERR_SHAPE, "%s: q_t needs rows %% 128 == 0 (got %lld)", fn, (long long)rows);
  if (rows == 0 || (!q && !q_t && !hq)) return ok();
  const int64_t width = gated ? 2 * cols : cols, eb = elem_bytes(dtype);
  if (int e = check_apart(fn, {{"q", q, rows * cols}, {"scale", scale, rows * cols / 32},
                               {"q_t", q_t, rows * cols}, {"scale_t", scale_t, rows * cols / 32},
                               {"hq", hq, rows * width}, {"hscale", hscale, rows * width / 32}},
                          {{"h", h, width * eb, rows_valid, ldh * eb}}))
    return e;
  fp8lin::ActArgs a{};
  a.x = h, a.ldx = ldh, a.rows = rows, a.valid = rows_valid, a.cols = cols, a.act = act;
  a.gated = gated != 0, a.dtype = dtype, a.q = static_cast<uint8_t*>(q), a.scale = scale;
  a.q_t = static_cast<uint8_t*>(q_t), a.scale_t = scale_t, a.hq = static_cast<uint8_t*>(hq);
  a.hscale = hscale;
  return hip_status(fp8lin::launch_act_quantize(a, as_stream(stream)), fn);
}

int fp8_act_quantize_bwd(const void* da, int64_t ldda, const void* hq, const float* hscale,
                         int64_t rows, int64_t rows_valid, int64_t cols, int act, int gated,
                         int dtype, void* q, float* scale, void* q_t, float* scale_t, void* dh,
                         void* stream) {
  const char* fn = "fp8_act_quantize_bwd";
  if (int e = check_act(fn, rows, rows_valid, cols, act, dtype)) return e;
  if (int e = check_rows(fn, "da", da, ldda, rows_valid, cols, dtype)) return e;
  if (rows_valid > 0 && (!hq || !hscale)) return fail(FP8_ERR_NULL, "%s: hq or hscale is NULL", fn);
  if (int e = check_pair(fn, "hq", hq, hscale, rows_valid)) return e;
  if (int e = check_pair(fn, "q", q, scale, rows)) return e;
  if (int e = check_pair(fn, "q_t", q_t, scale_t, rows)) return e;
  if (!aligned_to(dh, elem_bytes(dtype)))
    return fail(FP8_ERR_ALIGN, "%s: dh is not aligned to its elements", fn);
  if (q_t && rows % 128)
    return fail(FP8_ERR_SHAPE, "%s: q_t needs rows %% 128 == 0 (got %lld)", fn, (long long)rows);
  if (rows == 0 || (!q && !q_t && !dh)) return ok();
  const int64_t width = gated ? 2 * cols : cols, eb = elem_bytes(dtype);
  if (int e = check_apart(fn, {{"q", q, rows * width}, {"scale", scale, rows * width / 32},
                               {"q_t", q_t, rows * width}, {"scale_t", scale_t, rows * width / 32},
                               {"dh", dh, rows * width * eb}},
                          {{"da", da, cols * eb, rows_valid, ldda * eb},
                           {"hq", hq, rows_valid * width}, {"hscale", hscale, rows_valid * width / 32}}))
    return e;
  fp8lin::ActArgs a{};
  a.x = da, a.ldx = ldda, a.rows = rows, a.valid = rows_valid, a.cols = cols, a.act = act;
  a.gated = gated != 0, a.dtype = dtype, a.q = static_cast<uint8_t*>(q), a.scale = scale;
  a.q_t = static_cast<uint8_t*>(q_t), a.scale_t = scale_t;
  a.hq = static_cast<uint8_t*>(const_cast<void*>(hq)), a.hscale = const_cast<float*>(hscale);
  a.dh = dh;
  return hip_status(fp8lin::launch_act_quantize_bwd(a, as_stream(stream)), fn);
}

int fp8_grouped_linear_fwd(const void* qx, const void* qw, int64_t ldw, int64_t stride_w,
                           const float* sx, const float* sw, int64_t ldsw, int64_t stride_sw,
                           const int32_t* offsets, const int32_t* counts, int32_t experts,
                           int64_t rows, int64_t N, int64_t K, int64_t max_rows, void* y,
                           void* stream) {
  return grouped("fp8_grouped_linear_fwd", qx, qw, ldw, stride_w, sx, sw, ldsw, stride_sw, offsets,
                 counts, experts, rows, N, K, max_rows, y, stream);
}

int fp8_grouped_linear_dgrad(const void* qg, const void* qw_t, int64_t ldw, int64_t stride_w,
                             const float* sg, const float* sw_t, int64_t ldsw, int64_t stride_sw,
                             const int32_t* offsets, const int32_t* counts, int32_t experts,
                             int64_t rows, int64_t N, int64_t K, int64_t max_rows, void* dx,
                             void* stream) {
  return grouped("fp8_grouped_linear_dgrad", qg, qw_t, ldw, stride_w, sg, sw_t, ldsw, stride_sw,
                 offsets, counts, experts, rows, K, N, max_rows, dx, stream);
}

int fp8_grouped_linear_wgrad(const void* qg_t, const void* qx_t, const float* sg_t,
                             const float* sx_t, const int32_t* offsets, const int32_t* counts,
                             int32_t experts, int64_t rows, int64_t N, int64_t K, void* dw,
                             void* stream) {
  const char* fn = "fp8_grouped_linear_wgrad";
  if (int e = check_grouped(fn, offsets, counts, experts, rows, N, K)) return e;
  if (rows % 128)
    return fail(FP8_ERR_SHAPE, "%s: rows=%lld not a multiple of 128", fn, (long long)rows);
  if (!dw) return fail(FP8_ERR_NULL, "%s: dw is NULL", fn);
  if (rows > 0 && (!qg_t || !qx_t || !sg_t || !sx_t))
    return fail(FP8_ERR_NULL, "%s: NULL operand or scale pointer", fn);
  if (!aligned16(qg_t) || !aligned16(qx_t) || !aligned16(dw) || !aligned_to(sg_t, 4) ||
      !aligned_to(sx_t, 4))
    return fail(FP8_ERR_ALIGN, "%s: operands and output must be 16-byte aligned, scales 4-byte", fn);
  if (int e = check_apart(fn, {{"dw", dw, 2 * experts * N * K}},
                          {{"qg_t", qg_t, N * rows}, {"sg_t", sg_t, N * rows / 32},
                           {"qx_t", qx_t, K * rows}, {"sx_t", sx_t, K * rows / 32},
                           {"offsets", offsets, 4 * ((int64_t)experts + 1)},
                           {"counts", counts, 4 * (int64_t)experts}}))
    return e;
  fp8lin::GroupedArgs a{};
  a.w = static_cast<const uint8_t*>(qg_t), a.x = static_cast<const uint8_t*>(qx_t);
  a.sw = sg_t, a.sx = sx_t, a.offsets = offsets, a.counts = counts, a.experts = experts;
  a.rows = rows, a.N = N, a.K = K, a.y = static_cast<uint16_t*>(dw);
  return hip_status(fp8lin::launch_grouped_wgrad(a, as_stream(stream)), fn);
}

}  // extern "C"
