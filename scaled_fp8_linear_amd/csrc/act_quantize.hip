// The activation between two FP8 linears with its quantization, the 8-bit copy of its input that
// the backward reads, and that backward, by the block recipe's 1x128 tiles.
//
//   forward    h [rows, cols] or, gated, [g | u] of 2 cols columns;  a = act(h) or act(g) u
//              q, scale       a in tiles of 128 along a row (the next product's operand)
//              q_t, scale_t   a^T in tiles of 128 along the rows (its weight gradient's)
//              hq, hscale     h in tiles of 128 along a row (kept for the backward)
//   backward   from da and hq, hscale:  dh = da act'(h), or dg = da u act'(g), du = da act(g);
//              dh as it is and/or q, scale, q_t, scale_t of dh
//
//   act        relu(x) = max(x, 0);  silu(x) = x s(x), s the logistic function;
//              gelu(x) = x s(2 z), z = sqrt(2 / pi) (x + 0.044715 x^3), which is the form with
//              tanh: 0.5 (1 + tanh z) = s(2 z)
//
// A tile with largest magnitude m has the scale max(m, 1e-12) / 448 and its codes are
// e4m3(v / scale). All values are float32 until then. The scale is m times the rounded 1/448 and
// the multiplier the hardware's reciprocal of it: both within 2 units in the last place, against
// codes that keep 3 bits; two correctly rounded divisions a tile would be some 30 instructions in
// every lane. A product may so exceed 448 by 2^-21 of it, which still rounds to the code of 448. A
// NaN is coded as NaN and does not enter m; an infinity makes its tile's scale infinite.
//
// A workgroup owns 128 x 128 elements of a: 512 lanes of 4 rows x 8 columns. Row maxima are DPP
// steps over the 16 lanes of a row; column maxima go over the lanes and then through LDS, as do
// the transposed codes (4 rows in a dword).
//
// What bounds it: memory. 17408 x 14336 bf16 gated, calls over three sets of inputs: forward 393 us,
// 2.0 GB (5.1 TB/s), backward 430 us, 2.0 GB (4.7 TB/s). Either reads about as much as it writes, and
// writes 10 to 13 % more than that, since a tile's scales are 4 bytes of a line that other tiles write
// too. Why the backward is the slower one is not known. A token of 128 padding rows 5.5 us, most of it
// the call.
#include "common.h"
#include "launch.h"
#include "rows.h"

namespace fp8lin {

namespace {

constexpr int kAT = 128;                     // tile edge
constexpr int kAThreads = 512;
constexpr int kARows = 4;                    // rows of a lane
constexpr int kAWaves = kAThreads / 64;
constexpr int kAColDwords = kAT / 4;
constexpr float kInvE4M3Max = 1.0f / kE4M3Max;
constexpr float kLog2e = 1.4426950408889634f;

enum Act { kRelu = 0, kSilu = 1, kGelu = 2 };

// Maxima over lanes go by the bits of the magnitudes, which order as the numbers do (a lane's own
// maximum is never NaN): float maxima of values from other lanes would first be made quiet.
template <int CTRL> __device__ __forceinline__ uint32_t dpp_bits(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
// over 16 consecutive lanes, of several values step by step (a step has to wait for the last one)
template <int N> __device__ __forceinline__ void row16_max(uint32_t (&m)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = max(m[i], dpp_bits<0xB1>(m[i]));
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = max(m[i], dpp_bits<0x4E>(m[i]));
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = max(m[i], dpp_bits<0x141>(m[i]));
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = max(m[i], dpp_bits<0x140>(m[i]));
}
// over the 4 lanes that differ in bits 4 and 5
__device__ __forceinline__ uint32_t col4_max(uint32_t u) {
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t w = max((uint32_t)r[0], (uint32_t)r[1]);
  const auto s = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return max((uint32_t)s[0], (uint32_t)s[1]);
}

// s(x) = 1 / (1 + exp(-x)); 0 and 1 where the exponential leaves float32
__device__ __forceinline__ float logistic(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}
constexpr float kGeluA = 0.7978845608028654f;            // sqrt(2 / pi)
constexpr float kGeluB = 0.7978845608028654f * 0.044715f;

// act(x), and with D its derivative in `d`
template <int ACT, bool D>
__device__ __forceinline__ float activate(float x, float& d) {
  if constexpr (ACT == kRelu) {
    if (D) d = x > 0.f ? 1.f : 0.f;
    return x < 0.f ? 0.f : x;                            // a NaN stays
  } else if constexpr (ACT == kSilu) {
    const float s = logistic(x), y = x * s;
    if (D) d = fmaf(y, 1.f - s, s);
    return y;
  } else {
    const float x2 = __builtin_fminf(x * x, 1e30f);      // (1 - s) x2 is 0, not 0 times infinity
    const float s = logistic(2.f * x * fmaf(kGeluB, x2, kGeluA)), y = x * s;
    if (D) d = fmaf(y * (1.f - s), fmaf(6.f * kGeluB, x2, 2.f * kGeluA), s);
    return y;
  }
}

struct TileScale { float scale, mul; };
__device__ __forceinline__ TileScale tile_scale(float m) {
  const float a = __builtin_fmaxf(m, kAmaxFloor);
  const float s = a * kInvE4M3Max;
  return {s, __builtin_amdgcn_rcpf(s)};
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float ma, float mb,
                                           float mc, float md) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a * ma, b * mb, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * mc, d * md, lo, true);
}

// 4 rows x 4 codes (a dword each) -> 4 columns (rows 0 .. 3 in bytes 0 .. 3)
__device__ __forceinline__ void transpose4(const uint32_t (&w)[4], uint32_t (&c)[4]) {
  const uint32_t a01 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u);
  const uint32_t b01 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u);
  const uint32_t a23 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
  const uint32_t b23 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
  c[0] = __builtin_amdgcn_perm(a23, a01, 0x05040100u);
  c[1] = __builtin_amdgcn_perm(a23, a01, 0x07060302u);
  c[2] = __builtin_amdgcn_perm(b23, b01, 0x05040100u);
  c[3] = __builtin_amdgcn_perm(b23, b01, 0x07060302u);
}

// 8 elements at a row's column c
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    unpack(ld_piece<kStream>(p), f, T{});
  } else {
    float lo[4], hi[4];
    unpack(ld_piece<kStream>(p), lo, T{});
    unpack(ld_piece<kStream>(p + 4), hi, T{});
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = lo[j], f[4 + j] = hi[j];
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    st_piece<kStream>(p, pack(f, T{}));
  } else {
    st_piece<kStream>(p, pack({f[0], f[1], f[2], f[3]}, T{}));
    st_piece<kStream>(p + 4, pack({f[4], f[5], f[6], f[7]}, T{}));
  }
}

struct Lds {
  uint32_t tile[kAT * kAColDwords];          // transposed codes, 16 KiB
  uint32_t col[kAWaves][kAT];                // the waves' column maxima
  float mul[kAT];                            // the columns' multipliers
};

// dword i (rows 4 i .. 4 i + 3) of tile column c
__device__ __forceinline__ int tile_at(int c, int i) {
  return c * kAColDwords + (i ^ ((c >> 3) & (kAColDwords - 1)));
}

// Where a tile lies, and the lane's rows in it: 4 from `row` on, at columns 8 cc.
struct Place {
  int64_t rows, row0, row, tr;
  int t, rg, cc;
  bool whole;                                // all 128 rows are in the tensor
};

// One tile v (the lane's 4 x 8) quantized along its rows: codes q [rows, width], scales.
__device__ __forceinline__ void emit_rows(const float (&v)[kARows][8], const Place& at, int64_t tc,
                                          int64_t width, uint8_t* q, float* scale) {
  uint32_t m[kARows];
#pragma unroll
  for (int i = 0; i < kARows; ++i) {
    float f = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j += 2)
      f = __builtin_fmaxf(__builtin_fmaxf(f, __builtin_fabsf(v[i][j])), __builtin_fabsf(v[i][j + 1]));
    m[i] = __float_as_uint(f);
  }
  row16_max(m);
  uint8_t* p = q + at.row * width + tc * kAT + 8 * at.cc;
  const int64_t blocks = width / kAT;
  float* s = scale + at.row * blocks + tc;
#pragma unroll
  for (int i = 0; i < kARows; ++i, p += width, s += blocks) {
    const TileScale c = tile_scale(__uint_as_float(m[i]));
    if (!at.whole && at.row + i >= at.rows) continue;
    st_stream8(p, codes4(v[i][0], v[i][1], v[i][2], v[i][3], c.mul, c.mul, c.mul, c.mul),
               codes4(v[i][4], v[i][5], v[i][6], v[i][7], c.mul, c.mul, c.mul, c.mul));
    if (at.cc == 0) *s = c.scale;
  }
}

// The same tile quantized along its columns: q_t [width, rows], scales [width, rows / 128].
__device__ __forceinline__ void emit_cols(const float (&v)[kARows][8], const Place& at, int64_t tc,
                                          uint8_t* q_t, float* scale_t, Lds& lds) {
  static_assert(kARows == 4, "two steps of three");
  const int wave = at.t >> 6, lane = at.t & 63;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float f = 0.f;                           // NaN is no magnitude
#pragma unroll
    for (int i = 0; i < 4; i += 2)
      f = __builtin_fmaxf(__builtin_fmaxf(f, __builtin_fabsf(v[i][j])), __builtin_fabsf(v[i + 1][j]));
    const uint32_t m = col4_max(__float_as_uint(f));
    if (lane < 16) lds.col[wave][8 * at.cc + j] = m;
  }
  __syncthreads();
  if (at.t < kAT) {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < kAWaves; ++w) m = max(m, lds.col[w][at.t]);
    const TileScale s = tile_scale(__uint_as_float(m));
    lds.mul[at.t] = s.mul;
    scale_t[(tc * kAT + at.t) * (at.rows / kAT) + at.tr] = s.scale;
  }
  __syncthreads();
  float mul[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) mul[j] = lds.mul[8 * at.cc + j];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t w[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = codes4(v[i][4 * half], v[i][4 * half + 1], v[i][4 * half + 2], v[i][4 * half + 3],
                    mul[4 * half], mul[4 * half + 1], mul[4 * half + 2], mul[4 * half + 3]);
    transpose4(w, c);
#pragma unroll
    for (int j = 0; j < 4; ++j) lds.tile[tile_at(8 * at.cc + 4 * half + j, at.rg)] = c[j];
  }
  __syncthreads();
  constexpr int kItems = kAT * kAT / 16 / kAThreads;     // 16 rows of a column each
  const int c0 = at.t / 8, ch = at.t % 8;
  uint8_t* out = q_t + (tc * kAT + c0) * at.rows + at.row0 + 16 * ch;
#pragma unroll
  for (int n = 0; n < kItems; ++n, out += (int64_t)(kAThreads / 8) * at.rows) {
    const int c = n * (kAThreads / 8) + c0;
    uint4 o;
    o.x = lds.tile[tile_at(c, 4 * ch + 0)];
    o.y = lds.tile[tile_at(c, 4 * ch + 1)];
    o.z = lds.tile[tile_at(c, 4 * ch + 2)];
    o.w = lds.tile[tile_at(c, 4 * ch + 3)];
    *reinterpret_cast<uint4*>(out) = o;
  }
}

// Workgroups go round-robin over the 8 XCDs. An XCD takes runs of 8 tiles, so that the neighbours
// whose scales share 32 bytes write them in one L2 (17408 x 14336 gated, us: single tiles 410 forward
// and 472 backward, runs of 8 393 and 430, of 16 387 and 432, of 32 387 and 437; 80 tiles and 224 take
// the same either way).
constexpr int kRun = 8;
int64_t act_workgroups(int64_t tiles) { return (tiles + 8 * kRun - 1) / (8 * kRun) * (8 * kRun); }
__device__ __forceinline__ bool place(Place& at, int64_t rows, int tiles_c, int64_t& tc) {
  const int total = (int)((rows + kAT - 1) / kAT) * tiles_c, b = (int)blockIdx.x;
  const int id = b / (8 * kRun) * (8 * kRun) + (b & 7) * kRun + (b >> 3) % kRun;
  if (id >= total) return false;
  const int tr = id / tiles_c;
  at.rows = rows;
  at.tr = tr;
  tc = id - tr * tiles_c;
  at.row0 = (int64_t)tr * kAT;
  at.t = threadIdx.x, at.rg = at.t >> 4, at.cc = at.t & 15;
  at.row = at.row0 + kARows * at.rg;
  at.whole = at.row0 + kAT <= rows;
  return true;
}

template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(kAThreads)
act_quantize_kernel(const T* __restrict__ h, int64_t ldh, int64_t rows, int64_t valid,
                    int64_t cols, uint8_t* __restrict__ q, float* __restrict__ scale,
                    uint8_t* __restrict__ q_t, float* __restrict__ scale_t,
                    uint8_t* __restrict__ hq, float* __restrict__ hscale, int tiles_c) {
  __shared__ __attribute__((aligned(16))) Lds lds;
  int64_t tc;
  Place at;
  if (!place(at, rows, tiles_c, tc)) return;
  float v[kARows][8], u[kARows][8];
  const T* p = h + at.row * ldh + tc * kAT + 8 * at.cc;
  if (at.row0 + kAT <= valid) {
#pragma unroll
    for (int i = 0; i < kARows; ++i, p += ldh) {
      load8(p, v[i]);
      if constexpr (GATED) load8(p + cols, u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kARows; ++i, p += ldh) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.f, u[i][j] = 0.f;
      if (at.row + i >= valid) continue;
      load8(p, v[i]);
      if constexpr (GATED) load8(p + cols, u[i]);
    }
  }
  if (hq) {
    const int64_t width = GATED ? 2 * cols : cols;
    emit_rows(v, at, tc, width, hq, hscale);
    if constexpr (GATED) emit_rows(u, at, tc + tiles_c, width, hq, hscale);
  }
#pragma unroll
  for (int i = 0; i < kARows; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float d;
      v[i][j] = activate<ACT, false>(v[i][j], d);
      if constexpr (GATED) v[i][j] *= u[i][j];
    }
  if (q) emit_rows(v, at, tc, cols, q, scale);
  if (q_t) emit_cols(v, at, tc, q_t, scale_t, lds);
}

typedef float act_f32x2 __attribute__((ext_vector_type(2)));

// The 8 values of a row's codes (two dwords).
__device__ __forceinline__ void decode8(fp8lin_u32x2 w, float scale, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const act_f32x2 p = (i & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i / 2], true)
                                : __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i / 2], false);
    f[2 * i] = p[0] * scale, f[2 * i + 1] = p[1] * scale;
  }
}

template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(kAThreads)
act_quantize_bwd_kernel(const T* __restrict__ da, int64_t ldda, int64_t rows, int64_t valid,
                        int64_t cols, const uint8_t* __restrict__ hq,
                        const float* __restrict__ hscale, uint8_t* __restrict__ q,
                        float* __restrict__ scale, uint8_t* __restrict__ q_t,
                        float* __restrict__ scale_t, T* __restrict__ dh, int tiles_c) {
  __shared__ __attribute__((aligned(16))) Lds lds;
  int64_t tc;
  Place at;
  if (!place(at, rows, tiles_c, tc)) return;
  const int64_t col = tc * kAT + 8 * at.cc;
  const int64_t width = GATED ? 2 * cols : cols, blocks = width / kAT;
  float v[kARows][8], u[kARows][8];            // first da and the values of u, then dg and du
  fp8lin_u32x2 gq[kARows], uq[kARows];
  float gs[kARows], us[kARows];
  {
    const T* p = da + at.row * ldda + col;
    const uint8_t* ph = hq + at.row * width + col;
    const float* ps = hscale + at.row * blocks + tc;
    auto load = [&](int i) __attribute__((always_inline)) {
      load8(p, v[i]);
      gq[i] = __builtin_nontemporal_load(reinterpret_cast<const fp8lin_u32x2*>(ph));
      gs[i] = *ps;
      if constexpr (GATED) {
        uq[i] = __builtin_nontemporal_load(reinterpret_cast<const fp8lin_u32x2*>(ph + cols));
        us[i] = ps[tiles_c];
      }
    };
    if (at.row0 + kAT <= valid) {
#pragma unroll
      for (int i = 0; i < kARows; ++i, p += ldda, ph += width, ps += blocks) load(i);
    } else {
#pragma unroll
      for (int i = 0; i < kARows; ++i, p += ldda, ph += width, ps += blocks) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        gq[i] = uq[i] = fp8lin_u32x2{0u, 0u};
        gs[i] = us[i] = 0.f;
        if (at.row + i < valid) load(i);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kARows; ++i) {
    float g[8];
    decode8(gq[i], gs[i], g);
    if constexpr (GATED) decode8(uq[i], us[i], u[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float d;
      const float y = activate<ACT, true>(g[j], d);
      if constexpr (GATED) {
        const float da_j = v[i][j];
        v[i][j] = da_j * u[i][j] * d;
        u[i][j] = da_j * y;
      } else {
        v[i][j] *= d;
      }
    }
  }
  if (dh) {
    T* p = dh + at.row * width + col;
#pragma unroll
    for (int i = 0; i < kARows; ++i, p += width) {
      if (!at.whole && at.row + i >= rows) continue;
      store8(p, v[i]);
      if constexpr (GATED) store8(p + cols, u[i]);
    }
  }
  if (q) {
    emit_rows(v, at, tc, width, q, scale);
    if constexpr (GATED) emit_rows(u, at, tc + tiles_c, width, q, scale);
  }
  if (q_t) {
    emit_cols(v, at, tc, q_t, scale_t, lds);
    if constexpr (GATED) {
      __syncthreads();                         // the first tile's codes have been read
      emit_cols(u, at, tc + tiles_c, q_t, scale_t, lds);
    }
  }
}

template <typename F> hipError_t by_act(const ActArgs& a, F f) {
  using std::integral_constant;
  auto gated = [&](auto tag, auto act) {
    return a.gated ? f(tag, act, std::true_type{}) : f(tag, act, std::false_type{});
  };
  auto kind = [&](auto tag) {
    if (a.act == kRelu) return gated(tag, integral_constant<int, kRelu>{});
    if (a.act == kSilu) return gated(tag, integral_constant<int, kSilu>{});
    return gated(tag, integral_constant<int, kGelu>{});
  };
  if (a.dtype == kBF16) return kind(BF16{});
  if (a.dtype == kF16) return kind(F16{});
  return kind(0.0f);
}

}  // namespace

hipError_t launch_act_quantize(const ActArgs& a, hipStream_t s) {
  const int64_t tiles_c = a.cols / kAT, tiles = (a.rows + kAT - 1) / kAT * tiles_c;
  return by_act(a, [&](auto tag, auto act, auto gated) {
    using T = decltype(tag);
    hipLaunchKernelGGL((act_quantize_kernel<T, decltype(act)::value, decltype(gated)::value>),
                       dim3((unsigned)act_workgroups(tiles)), dim3(kAThreads), 0, s,
                       static_cast<const T*>(a.x), a.ldx, a.rows, a.valid, a.cols, a.q, a.scale,
                       a.q_t, a.scale_t, a.hq, a.hscale, (int)tiles_c);
    return hipGetLastError();
  });
}

hipError_t launch_act_quantize_bwd(const ActArgs& a, hipStream_t s) {
  const int64_t tiles_c = a.cols / kAT, tiles = (a.rows + kAT - 1) / kAT * tiles_c;
  return by_act(a, [&](auto tag, auto act, auto gated) {
    using T = decltype(tag);
    hipLaunchKernelGGL((act_quantize_bwd_kernel<T, decltype(act)::value, decltype(gated)::value>),
                       dim3((unsigned)act_workgroups(tiles)), dim3(kAThreads), 0, s,
                       static_cast<const T*>(a.x), a.ldx, a.rows, a.valid, a.cols, a.hq, a.hscale,
                       a.q, a.scale, a.q_t, a.scale_t, static_cast<T*>(a.dh), (int)tiles_c);
    return hipGetLastError();
  });
}

}  // namespace fp8lin
