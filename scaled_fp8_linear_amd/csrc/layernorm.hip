// Layer norm over the rows of a [rows, cols] tensor, and its gradient.
//
//   mean = sum_c x / cols,  rstd = 1 / sqrt(sum_c (x - mean)^2 / cols + eps)
//   y = (x - mean) rstd gamma + beta
//   with xh = (x - mean) rstd and g = dy gamma:
//   dx = rstd (g - sum_c(g) / cols - xh sum_c(g xh) / cols)
//   dgamma = sum_r dy xh,  dbeta = sum_r dy
//
// All sums are float32; y, dx, dgamma and dbeta are rounded once, on the store. The row
// stays in registers between the sums, so the variance is the sum of the squared distances
// from the mean (not a difference of two large sums) and x is read from memory once.
// Everything here is bound by memory: 2 (forward) or 3 (backward) tensor reads and writes
// against about 8 and 14 flops an element.
#include <algorithm>

#include "launch.h"
#include "rows.h"

namespace fp8lin {

namespace {

// The N elements at column c of a parameter row as floats (`fill` without a tensor). Read once
// a workgroup, so the parameters' type (the rows' or float32) is a value, not another kernel.
template <typename T, int N>
__device__ __forceinline__ void ld_params(const void* p, bool f32, int c, int cols, float fill,
                                          float (&f)[N]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = fill;
  } else if (f32) {
#pragma unroll
    for (int h = 0; h < N; h += 4) {
      float t[4];
      unpack(ld_row(static_cast<const float*>(p), c + h, cols), t, float{});
#pragma unroll
      for (int i = 0; i < 4; ++i) f[h + i] = t[i];
    }
  } else {
    unpack(ld_row(static_cast<const T*>(p), c, cols), f, T{});
  }
}
template <typename T>
__device__ __forceinline__ void st_param(void* p, bool f32, int c, float v) {
  if (f32) static_cast<float*>(p)[c] = v;
  else static_cast<T*>(p)[c] = from_f32<T>(v);
}

// Four partial sums; a workspace is aligned to its floats only.
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float sums_t __attribute__((ext_vector_type(4), aligned(4)));

// The lane group (row of a turn) of this thread; the same for a whole wave where a row takes
// one or more, so that row addresses are scalar.
template <int LPR>
__device__ __forceinline__ int row_group() {
  const int g = threadIdx.x / LPR;
  return LPR >= 64 ? __builtin_amdgcn_readfirstlane(g) : g;
}

// The row of a group in the turn that starts at r0. A group past the last row works on that
// row and stores nothing, so that every group takes the same number of turns and the barriers
// in a row's sums always meet.
__device__ __forceinline__ int64_t turn_row(int64_t r0, int group, int64_t rows) {
  return r0 + group < rows ? r0 + group : rows - 1;
}

// This lane's pieces of a row, not yet cut at its end.
template <Cache C, int LPR, typename T, int NV>
__device__ __forceinline__ void ld_rows(const T* row, int lane, int cols, piece_t (&p)[NV]) {
#pragma unroll
  for (int v = 0; v < NV; ++v)
    p[v] = ld_raw<C, LPR == 16>(row, (v * LPR + lane) * Piece<T>::N, cols);
}

// Sum over the LPR lanes of a row. Rows of several waves meet in LDS (`part`, one float per
// wave of the workgroup); the caller alternates buffers so that one barrier per sum is
// enough.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = lanes_sum<(LPR < 64 ? LPR : 64)>(v);
  if constexpr (LPR > 64) {
    constexpr int W = LPR / 64;
    const int wave = row_group<64>();
    if (threadIdx.x % 64 == 0) part[wave] = v;
    __syncthreads();
    v = lanes_sum<W>(part[wave / W * W + threadIdx.x % W]);
  }
  return v;
}

// The forward's workgroups are short (eight to a compute unit), the backward's hold one unit
// each: 16 waves of 128 registers, and as few rows of partial sums as that allows. Backward of
// 8192x4096 bf16: 45.0 us so, 45.3 us with twice as many workgroups of 512, 48.1 us with four
// times as many of 256; of 1021x5003 f16 21.4, 22.5 and 22.6 us, and with half the workgroups
// 24.6 us. The forward of 8192x4096 does not depend on its grid (23.0 to 23.7 us).
constexpr int kFwdBlock = 256, kBwdBlock = 1024;
constexpr int64_t kFwdGrid = 256 * 8, kBwdGrid = 256;

constexpr int fwd_block(int lpr) { return lpr > kFwdBlock ? lpr : kFwdBlock; }

// LPR lanes own a row; lane l holds the pieces l, l + LPR, ... (EPT elements). A workgroup
// walks the rows with the grid's stride and loads the next row while it works on this one.
template <typename T, int LPR, int EPT, int BLOCK, Cache LOAD>
__global__ void __launch_bounds__(BLOCK)
layernorm_fwd_kernel(const T* __restrict__ x, int64_t ldx, const void* __restrict__ gamma,
                     const void* __restrict__ beta, bool params_f32, int64_t rows, int cols, float eps,
                     T* __restrict__ y, float* __restrict__ mean_out,
                     float* __restrict__ rstd_out) {
  constexpr int N = Piece<T>::N, NV = EPT / N, ROWS = BLOCK / LPR;
  // gamma, beta and the next row stay in registers beside the row up to 16 elements a lane
  constexpr bool kAhead = EPT <= 16;
  __shared__ float part[2][BLOCK / 64];
  const int lane = threadIdx.x % LPR, group = row_group<LPR>();
  const float fcols = (float)cols;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  piece_t cur[NV], next[NV];
  if (kAhead)
    ld_rows<LOAD, LPR>(x + turn_row((int64_t)blockIdx.x * ROWS, group, rows) * ldx, lane, cols,
                        cur);
  float gm[NV][N], bt[NV][N];
  if constexpr (kAhead) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      ld_params<T>(gamma, params_f32, (v * LPR + lane) * N, cols, 1.f, gm[v]);
      ld_params<T>(beta, params_f32, (v * LPR + lane) * N, cols, 0.f, bt[v]);
    }
  }
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < rows; r0 += step) {
    if (!kAhead)
      ld_rows<LOAD, LPR>(x + turn_row(r0, group, rows) * ldx, lane, cols, cur);
    else if (r0 + step < rows)
      ld_rows<LOAD, LPR>(x + turn_row(r0 + step, group, rows) * ldx, lane, cols, next);
    const int64_t r = r0 + group;
    float f[NV][N];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      unpack(cut<T>(cur[v], (v * LPR + lane) * N, cols), f[v], T{});
#pragma unroll
      for (int i = 0; i < N; ++i) s += f[v][i];
    }
    const float mean = row_sum<LPR>(s, part[0]) / fcols;
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[v][i] -= mean;
        const float d = c + i < cols ? f[v][i] : 0.f;
        q = __builtin_fmaf(d, d, q);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<LPR>(q, part[1]) / fcols + eps);
    if (kAhead) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        arrived(next[v]);
        cur[v] = next[v];
      }
    }
    if (r < rows) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float o[N];
        if constexpr (!kAhead) {
          __builtin_amdgcn_sched_barrier(0);
          ld_params<T>(gamma, params_f32, (v * LPR + lane) * N, cols, 1.f, gm[v]);
          ld_params<T>(beta, params_f32, (v * LPR + lane) * N, cols, 0.f, bt[v]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = __builtin_fmaf(f[v][i] * rstd, gm[v][i], bt[v][i]);
        st_row<kStream>(y + r * cols, (v * LPR + lane) * N, cols, pack(o, T{}));
      }
      if (lane == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
      }
    }
  }
}

// The gradient in one pass over dy and x, the next row loaded while this one is worked on.
// Lanes own columns as in the forward, so each also sums dy xh and dy of its columns over the
// workgroup's rows, in registers; at the end the workgroup's row groups are added in LDS in
// group order and written as one row of partial sums, part[which][block][part_ld], which
// layernorm_bwd_params_kernel adds in a fixed order. A single workgroup writes dgamma and
// dbeta itself. Every order is fixed, so results repeat.
//
// A wave has 128 registers (16 waves a compute unit). What does not fit beside the two sums:
// gamma (then in LDS), the next row (then not loaded ahead), and for the widest float32 rows
// this row itself (then read again, from the cache, for dx).
template <typename T, int EPT> struct BwdFit {
  static constexpr int kRow = 2 * EPT * (int)sizeof(T) / 4, kSums = 2 * EPT;
  static constexpr bool kHold = kRow + kSums < 96;
  static constexpr bool kAhead = 2 * kRow + kSums <= 96;
  static constexpr bool kGammaLds = (kAhead ? 2 : 1) * kRow + kSums + EPT > 96;
};

template <typename T, int LPR, int EPT, Cache LOAD, Cache STORE>
__global__ void __launch_bounds__(kBwdBlock)
layernorm_bwd_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx,
                     const float* __restrict__ mean, const float* __restrict__ rstd,
                     const void* __restrict__ gamma, bool params_f32, int64_t rows, int cols,
                     T* __restrict__ dx, void* __restrict__ dgamma, void* __restrict__ dbeta,
                     float* __restrict__ part, int part_ld) {
  using Fit = BwdFit<T, EPT>;
  constexpr int BLOCK = kBwdBlock, WAVES = BLOCK / 64;
  constexpr int N = Piece<T>::N, NV = EPT / N, ROWS = BLOCK / LPR;
  constexpr bool kGammaLds = Fit::kGammaLds, kHold = Fit::kHold, kAhead = Fit::kAhead;
  __shared__ float red[2][2][WAVES];
  constexpr int kFold = ROWS > 1 ? BLOCK * EPT : 1;
  __shared__ __attribute__((aligned(16))) float fold[kGammaLds && kFold < LPR * EPT ? LPR * EPT : kFold];
  const int lane = threadIdx.x % LPR, group = row_group<LPR>();
  const float fcols = (float)cols;
  const int64_t step = (int64_t)gridDim.x * ROWS;
  const bool ragged = cols % N != 0;
  piece_t cx[NV], cd[NV], nx[NV], nd[NV];      // this row of x and dy, and the next
  float mu = 0.f, rs = 0.f, nmu = 0.f, nrs = 0.f;
  if (kAhead && (int64_t)blockIdx.x * ROWS < rows) {
    const int64_t r = turn_row((int64_t)blockIdx.x * ROWS, group, rows);
    ld_rows<LOAD, LPR>(x + r * ldx, lane, cols, cx);
    ld_rows<LOAD, LPR>(dy + r * lddy, lane, cols, cd);
    mu = mean[r], rs = rstd[r];
  }
  float gm[kGammaLds ? 1 : NV][N], ag[NV][N], ab[NV][N];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (kGammaLds) {
      float g[N];
      ld_params<T>(gamma, params_f32, (v * LPR + lane) * N, cols, 1.f, g);
      if (group == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) fold[(v * LPR + lane) * N + i] = g[i];
    } else {
      ld_params<T>(gamma, params_f32, (v * LPR + lane) * N, cols, 1.f, gm[v]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) ag[v][i] = ab[v][i] = 0.f;
  }
  if (kGammaLds && ROWS > 1) __syncthreads();     // one row group's lanes read their own
  auto gamma_of = [&](int v, int i) {
    if constexpr (kGammaLds) return fold[(v * LPR + lane) * N + i];
    else return gm[v][i];
  };
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < rows; r0 += step, turn ^= 1) {
    const int64_t r = r0 + group;
    const bool live = r < rows;
    const int64_t q = turn_row(kAhead ? r0 + step : r0, group, rows);
    if (!kAhead) {
      if constexpr (kHold) {
        ld_rows<LOAD, LPR>(x + q * ldx, lane, cols, cx);
        ld_rows<LOAD, LPR>(dy + q * lddy, lane, cols, cd);
      }
      mu = mean[q], rs = rstd[q];
    } else if (r0 + step < rows) {
      ld_rows<LOAD, LPR>(x + q * ldx, lane, cols, nx);
      ld_rows<LOAD, LPR>(dy + q * lddy, lane, cols, nd);
      nmu = mean[q], nrs = rstd[q];
    }
    // a group past the last row takes its turn (the barriers must meet) with dy = 0
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * N;
      float fx[N], fd[N];
      if constexpr (!kHold) {
        cx[v] = ld_raw<LOAD, false>(x + q * ldx, c, cols);
        cd[v] = ld_raw<LOAD, false>(dy + q * lddy, c, cols);
      }
      if (ragged) {
        cx[v] = cut<T>(cx[v], c, cols);
        cd[v] = cut<T>(cd[v], c, cols);
      }
      // past the row dy is 0 and x is some of the row's own values: nothing is added, and a
      // NaN there is one that the row has anyway
      if (!live || c >= cols) cd[v] = piece_t{0, 0, 0, 0};
      unpack(cx[v], fx, T{});
      unpack(cd[v], fd, T{});
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = (fx[i] - mu) * rs;
        const float g = fd[i] * gamma_of(v, i);
        s1 += g;
        s2 = __builtin_fmaf(g, xh, s2);
      }
      if constexpr (!kHold || kGammaLds) __builtin_amdgcn_sched_barrier(0);
    }
    s1 = lanes_sum<(LPR < 64 ? LPR : 64)>(s1);
    s2 = lanes_sum<(LPR < 64 ? LPR : 64)>(s2);
    if constexpr (LPR > 64) {
      constexpr int W = LPR / 64;
      const int wave = row_group<64>(), w = wave / W * W + threadIdx.x % W;
      if (threadIdx.x % 64 == 0) { red[turn][0][wave] = s1; red[turn][1][wave] = s2; }
      __syncthreads();
      s1 = lanes_sum<W>(red[turn][0][w]);
      s2 = lanes_sum<W>(red[turn][1][w]);
    }
    if (kAhead) {
#pragma unroll
      for (int v = 0; v < NV; ++v) { arrived(nx[v]); arrived(nd[v]); }
    }
    const float m1 = s1 / fcols, m2 = s2 / fcols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * N;
      float fx[N], fd[N], o[N];
      if constexpr (kHold) {
        // from the 16 bytes again: the floats of the first sums would not fit
        arrived(cx[v]);
        arrived(cd[v]);
      } else {
        cx[v] = cut<T>(ld_raw<LOAD, false>(x + q * ldx, c, cols), c, cols);
        cd[v] = cut<T>(ld_raw<LOAD, false>(dy + q * lddy, c, cols), c, cols);
        if (!live) cd[v] = piece_t{0, 0, 0, 0};
      }
      unpack(cx[v], fx, T{});
      unpack(cd[v], fd, T{});
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = (fx[i] - mu) * rs;
        o[i] = rs * __builtin_fmaf(-xh, m2, __builtin_fmaf(fd[i], gamma_of(v, i), -m1));
        ag[v][i] = __builtin_fmaf(fd[i], xh, ag[v][i]);
        ab[v][i] += fd[i];
      }
      if (live && dx) st_row<STORE>(dx + r * cols, c, cols, pack(o, T{}));
      if constexpr (!kHold || kGammaLds) __builtin_amdgcn_sched_barrier(0);
    }
    if (kAhead) {
#pragma unroll
      for (int v = 0; v < NV; ++v) cx[v] = nx[v], cd[v] = nd[v];
      mu = nmu, rs = nrs;
    }
  }
  if (!dgamma && !dbeta) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    void* out = which == 0 ? dgamma : dbeta;
    if (!out) continue;
    float (&acc)[NV][N] = which == 0 ? ag : ab;
    float* dst = part ? part + ((int64_t)which * gridDim.x + blockIdx.x) * part_ld : nullptr;
    if constexpr (ROWS > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < N; i += 4)
          *reinterpret_cast<f32x4_t*>(&fold[(group * NV * LPR + v * LPR + lane) * N + i]) =
              f32x4_t{acc[v][i], acc[v][i + 1], acc[v][i + 2], acc[v][i + 3]};
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += BLOCK) {
        float s = fold[c];
#pragma unroll
        for (int k = 1; k < ROWS; ++k) s += fold[k * LPR * EPT + c];
        if (dst) dst[c] = s;
        else st_param<T>(out, params_f32, c, s);
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const int c = (v * LPR + lane) * N + i;
          if (dst) {                       // part_ld is cols rounded up to 4
            if (c < cols)
              *reinterpret_cast<sums_t*>(dst + c) =
                  sums_t{acc[v][i], acc[v][i + 1], acc[v][i + 2], acc[v][i + 3]};
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (c + k < cols) st_param<T>(out, params_f32, c + k, acc[v][i + k]);
          }
        }
    }
  }
}

// out[c] = sum over the blocks of part[which][block][c]. 16 lanes take 64 columns, 64 such
// lane groups the blocks k, k + 64, ...; their sums are then added in order.
constexpr int kParamsRows = 64;
template <typename P>
__global__ void __launch_bounds__(1024)
layernorm_bwd_params_kernel(const float* __restrict__ part, int blocks, int cols, int part_ld,
                            P* __restrict__ dgamma, P* __restrict__ dbeta) {
  __shared__ f32x4_t s[kParamsRows][16];
  P* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (!out) return;
  const int cl = threadIdx.x % 16, rl = threadIdx.x / 16;
  const int c = blockIdx.x * 64 + cl * 4;
  const float* p = part + (int64_t)blockIdx.y * blocks * part_ld;
  f32x4_t a = {0.f, 0.f, 0.f, 0.f};
  if (c < cols) {
#pragma unroll 4
    for (int b = rl; b < blocks; b += kParamsRows)
      a += *reinterpret_cast<const sums_t*>(p + (int64_t)b * part_ld + c);
  }
  s[rl][cl] = a;
  __syncthreads();
  if (threadIdx.x < 64 && blockIdx.x * 64 + (int)threadIdx.x < cols) {
    const float* col = reinterpret_cast<const float*>(s) + threadIdx.x;
    float t = 0.f;
#pragma unroll 16
    for (int i = 0; i < kParamsRows; ++i) t += col[i * 64];
    out[blockIdx.x * 64 + threadIdx.x] = from_f32<P>(t);
  }
}

// Lanes and elements per lane of a row of `cols` elements.
struct Shape { int lpr, ept; };
Shape row_shape(int64_t cols) {
  if (cols <= 128) return {16, 8};
  if (cols <= 512) return {64, 8};
  if (cols <= 1024) return {64, 16};
  if (cols <= 2048) return {128, 16};
  if (cols <= 4096) return {256, 16};
  if (cols <= 8192) return {512, 16};
  if (cols <= 16384) return {1024, 16};
  return {1024, 32};
}

int64_t bwd_blocks(int64_t rows, int64_t cols) {
  const int64_t per = kBwdBlock / row_shape(cols).lpr, want = (rows + per - 1) / per;
  return want <= 4 ? 1 : std::min(want, kBwdGrid);     // 4 turns cost less than another launch
}

template <typename T, int LPR, int EPT, Cache LOAD>
hipError_t fwd(const LayerNormArgs& a, hipStream_t s) {
  constexpr int B = fwd_block(LPR);
  const int64_t blocks = std::min<int64_t>((a.rows + B / LPR - 1) / (B / LPR), kFwdGrid);
  hipLaunchKernelGGL((layernorm_fwd_kernel<T, LPR, EPT, B, LOAD>), dim3((unsigned)blocks), dim3(B),
                     0, s, static_cast<const T*>(a.x), a.ldx, a.gamma, a.beta,
                     a.param_dtype == kF32, a.rows, (int)a.cols, a.eps, static_cast<T*>(a.y),
                     a.mean, a.rstd);
  return hipGetLastError();
}

template <typename T, int LPR, int EPT, Cache LOAD, Cache STORE>
hipError_t bwd(const LayerNormArgs& a, hipStream_t s) {
  const int64_t blocks = bwd_blocks(a.rows, a.cols);
  float* part = blocks > 1 ? a.workspace : nullptr;
  const int part_ld = (int)((a.cols + 3) / 4 * 4);
  hipLaunchKernelGGL((layernorm_bwd_kernel<T, LPR, EPT, LOAD, STORE>), dim3((unsigned)blocks),
                     dim3(kBwdBlock), 0, s, static_cast<const T*>(a.dy), a.lddy, static_cast<const T*>(a.x),
                     a.ldx, a.mean, a.rstd, a.gamma, a.param_dtype == kF32, a.rows, (int)a.cols,
                     static_cast<T*>(a.y), a.dgamma, a.dbeta, part, part_ld);
  return hipGetLastError();
}

template <typename P>
hipError_t bwd_params(const LayerNormArgs& a, hipStream_t s) {
  const int part_ld = (int)((a.cols + 3) / 4 * 4);
  hipLaunchKernelGGL((layernorm_bwd_params_kernel<P>), dim3((unsigned)((a.cols + 63) / 64), 2),
                     dim3(1024), 0, s, a.workspace, (int)bwd_blocks(a.rows, a.cols), (int)a.cols,
                     part_ld, static_cast<P*>(a.dgamma), static_cast<P*>(a.dbeta));
  return hipGetLastError();
}

// What streams, by the bytes of one tensor of rows (the caches by the memory hold 256 MiB).
// Measured over three sets of tensors in turn, so that small ones are found in the caches.
//   Forward, x kept up to kKeepRows: 8192x4096 bf16 24.2 us (streamed 30.7), above 2048x14336
//   f32 63.4 us streamed (kept 65.7), 32768x4096 f32 191 us (201). y streams: 24.2 us against
//   30.7 with 8192x4096 bf16, 9.8 against 10.8 with 2048x4096, 53.3 against 54.0 with 8192x4096
//   f32. The quantize pass that reads y next then runs longer: addition, norm and quantize
//   together take 82.5 us at 8192x4096 with y streamed and 79.5 us with y kept, 29.4 and 29.8
//   us at 2048x4096.
//   Backward, dy and x kept up to kKeepGrad: 2048x4096 bf16 19.8 us (streamed 22.7), 8192x4096
//   49.0 us (43.9). dx kept up to kKeepRows: 8192x4096 bf16 43.9 us (streamed 47.8), above
//   16384x4096 bf16 77.7 us streamed (kept 80.6), 32768x4096 f32 293 us (312).
constexpr int64_t kKeepGrad = 24 << 20, kKeepRows = 96 << 20;

template <typename T, int LPR, int EPT>
hipError_t by_size(const LayerNormArgs& a, bool backward, hipStream_t s) {
  const int64_t bytes = a.rows * a.cols * (int64_t)sizeof(T);
  if (!backward)
    return bytes <= kKeepRows ? fwd<T, LPR, EPT, kKeep>(a, s) : fwd<T, LPR, EPT, kStream>(a, s);
  if (bytes <= kKeepGrad) return bwd<T, LPR, EPT, kKeep, kKeep>(a, s);
  return bytes <= kKeepRows ? bwd<T, LPR, EPT, kStream, kKeep>(a, s)
                          : bwd<T, LPR, EPT, kStream, kStream>(a, s);
}

template <typename T>
hipError_t by_shape(const LayerNormArgs& a, bool backward, hipStream_t s) {
  const Shape k = row_shape(a.cols);
#define FP8LIN_LN(L, E) \
  if (k.lpr == L && k.ept == E) return by_size<T, L, E>(a, backward, s);
  FP8LIN_LN(16, 8)
  FP8LIN_LN(64, 8)
  FP8LIN_LN(64, 16)
  FP8LIN_LN(128, 16)
  FP8LIN_LN(256, 16)
  FP8LIN_LN(512, 16)
  FP8LIN_LN(1024, 16)
  FP8LIN_LN(1024, 32)
#undef FP8LIN_LN
  return hipErrorInvalidValue;
}

}  // namespace

int64_t layernorm_bwd_workspace(int64_t rows, int64_t cols) {
  const int64_t b = bwd_blocks(rows, cols);
  return b > 1 ? 2 * b * ((cols + 3) / 4 * 4) * (int64_t)sizeof(float) : 0;
}

hipError_t launch_layernorm(const LayerNormArgs& a, bool backward, hipStream_t s) {
  const hipError_t e = a.dtype == kBF16  ? by_shape<BF16>(a, backward, s)
                       : a.dtype == kF16 ? by_shape<F16>(a, backward, s)
                                         : by_shape<float>(a, backward, s);
  if (e != hipSuccess || !backward || !a.workspace) return e;
  if (a.param_dtype == kBF16) return bwd_params<BF16>(a, s);
  return a.param_dtype == kF16 ? bwd_params<F16>(a, s) : bwd_params<float>(a, s);
}

}  // namespace fp8lin
