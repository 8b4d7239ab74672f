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

// EPT consecutive-piece elements of a parameter row as floats (`fill` without a tensor).
template <typename P, int N>
__device__ __forceinline__ void ld_params(const P* p, int c, int cols, float fill, float (&f)[N]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = fill;
    return;
  }
  constexpr int PN = Piece<P>::N;
  if constexpr (PN <= N) {
#pragma unroll
    for (int h = 0; h < N / PN; ++h) {
      float t[PN];
      unpack(ld_row(p, c + h * PN, cols), t, P{});
#pragma unroll
      for (int i = 0; i < PN; ++i) f[h * PN + i] = t[i];
    }
  } else {
    static_assert(PN <= N, "a parameter piece is at most a data piece");
  }
}

template <int LPR, int BLOCK> struct Group {
  static constexpr int kRows = BLOCK / LPR;             // rows in flight per workgroup
  static constexpr int kWaves = LPR > 64 ? LPR / 64 : 1;  // waves of a row
};

// Sum over the LPR lanes of a row. Rows of several waves meet in LDS (`part`, one float per
// wave of the workgroup); the caller alternates buffers so that one barrier per sum is
// enough.
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = lanes_sum<(LPR < 64 ? LPR : 64)>(v);
  if constexpr (LPR > 64) {
    constexpr int W = LPR / 64;
    const int wave = threadIdx.x / 64;
    if (threadIdx.x % 64 == 0) part[wave] = v;
    __syncthreads();
    const int w0 = wave / W * W;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += part[w0 + i];
  }
  return v;
}

// LPR lanes own a row; lane l holds the pieces l, l + LPR, ... (EPT elements). A workgroup
// walks the rows with the grid's stride.
template <typename T, typename P, int LPR, int EPT, int BLOCK>
__global__ void __launch_bounds__(BLOCK)
layernorm_fwd_kernel(const T* __restrict__ x, int64_t ldx, const P* __restrict__ gamma,
                     const P* __restrict__ beta, int64_t rows, int cols, float eps,
                     T* __restrict__ y, float* __restrict__ mean_out,
                     float* __restrict__ rstd_out) {
  constexpr int N = Piece<T>::N, NV = EPT / N, ROWS = BLOCK / LPR;
  __shared__ float part[2][BLOCK / 64];
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const float inv_n = (float)cols;
  float gm[NV][N], bt[NV][N];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    ld_params(gamma, (v * LPR + lane) * N, cols, 1.f, gm[v]);
    ld_params(beta, (v * LPR + lane) * N, cols, 0.f, bt[v]);
  }
  const int64_t step = (int64_t)gridDim.x * ROWS;
  // every group takes the same number of turns, so the barriers in row_sum always meet
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < rows; r0 += step) {
    const int64_t r = r0 + group;
    const bool live = r < rows;
    float f[NV][N];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const piece_t p = live ? ld_row(x + r * ldx, (v * LPR + lane) * N, cols) : piece_t{0, 0, 0, 0};
      unpack(p, f[v], T{});
#pragma unroll
      for (int i = 0; i < N; ++i) s += f[v][i];
    }
    const float mean = row_sum<LPR>(s, part[0]) / inv_n;
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[v][i] -= mean;
        if (c + i < cols) q += f[v][i] * f[v][i];
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<LPR>(q, part[1]) / inv_n + eps);
    if (live) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = f[v][i] * rstd * gm[v][i] + bt[v][i];
        st_row(y + r * cols, (v * LPR + lane) * N, cols, pack(o, T{}));
      }
      if (lane == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
      }
    }
  }
}

// The gradient in one pass over dy and x. Lanes own columns as in the forward, so each also
// sums dy xh and dy of its columns over the workgroup's rows, in registers; at the end the
// workgroup's row groups are added in LDS in group order and written as one row of partial
// sums, part[which][block][cols], which layernorm_bwd_params_kernel adds in block order. A
// single workgroup writes dgamma and dbeta itself. Every order is fixed, so results repeat.
template <typename T, typename P, int LPR, int EPT, int BLOCK>
__global__ void __launch_bounds__(BLOCK)
layernorm_bwd_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx,
                     const float* __restrict__ mean, const float* __restrict__ rstd,
                     const P* __restrict__ gamma, int64_t rows, int cols, T* __restrict__ dx,
                     P* __restrict__ dgamma, P* __restrict__ dbeta, float* __restrict__ part) {
  constexpr int N = Piece<T>::N, NV = EPT / N, ROWS = BLOCK / LPR, WAVES = BLOCK / 64;
  __shared__ float red[2][2][WAVES];
  __shared__ float fold[ROWS > 1 ? BLOCK * EPT : 1];
  const int lane = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const float fcols = (float)cols;
  float gm[NV][N], ag[NV][N], ab[NV][N];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    ld_params(gamma, (v * LPR + lane) * N, cols, 1.f, gm[v]);
#pragma unroll
    for (int i = 0; i < N; ++i) ag[v][i] = ab[v][i] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * ROWS;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < rows; r0 += step, turn ^= 1) {
    const int64_t r = r0 + group;
    const bool live = r < rows;
    piece_t px[NV], pd[NV];
    float mu = 0.f, rs = 0.f;
    if (live) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        px[v] = ld_row(x + r * ldx, (v * LPR + lane) * N, cols);
        pd[v] = ld_row(dy + r * lddy, (v * LPR + lane) * N, cols);
      }
      mu = mean[r];
      rs = rstd[r];
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) px[v] = pd[v] = piece_t{0, 0, 0, 0};
    }
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float fx[N], fd[N];
      unpack(px[v], fx, T{});
      unpack(pd[v], fd, T{});
      const int c = (v * LPR + lane) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // columns past the row hold dy = 0 and x = 0; an infinite mean must not reach them
        const float xh = c + i < cols ? (fx[i] - mu) * rs : 0.f;
        const float g = fd[i] * gm[v][i];
        s1 += g;
        s2 += g * xh;
        ag[v][i] += fd[i] * xh;
        ab[v][i] += fd[i];
      }
    }
    s1 = lanes_sum<(LPR < 64 ? LPR : 64)>(s1);
    s2 = lanes_sum<(LPR < 64 ? LPR : 64)>(s2);
    if constexpr (LPR > 64) {
      constexpr int W = LPR / 64;
      const int wave = threadIdx.x / 64, w0 = wave / W * W;
      if (threadIdx.x % 64 == 0) { red[turn][0][wave] = s1; red[turn][1][wave] = s2; }
      __syncthreads();
      s1 = s2 = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) { s1 += red[turn][0][w0 + i]; s2 += red[turn][1][w0 + i]; }
    }
    if (live && dx) {
      const float m1 = s1 / fcols, m2 = s2 / fcols;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float fx[N], fd[N], o[N];
        unpack(px[v], fx, T{});
        unpack(pd[v], fd, T{});
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float xh = (fx[i] - mu) * rs;
          o[i] = rs * (fd[i] * gm[v][i] - m1 - xh * m2);
        }
        st_row(dx + r * cols, (v * LPR + lane) * N, cols, pack(o, T{}));
      }
    }
  }
  if (!dgamma && !dbeta) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    P* out = which == 0 ? dgamma : dbeta;
    if (!out) continue;
    float (&acc)[NV][N] = which == 0 ? ag : ab;
    if constexpr (ROWS > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) fold[(group * NV + v) * (LPR * N) + i * LPR + lane] = acc[v][i];
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < N; ++i) {
            float s = acc[v][i];
            for (int k = 1; k < ROWS; ++k) s += fold[(k * NV + v) * (LPR * N) + i * LPR + lane];
            acc[v][i] = s;
          }
      }
    }
    if (group == 0) {
      float* dst = part ? part + ((int64_t)which * gridDim.x + blockIdx.x) * cols : nullptr;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = (v * LPR + lane) * N + i;
          if (c < cols) {
            if (dst) dst[c] = acc[v][i];
            else out[c] = from_f32<P>(acc[v][i]);
          }
        }
    }
  }
}

// out[c] = sum over the blocks of part[which][block][c]: 64 columns a workgroup, 16 lanes of
// rows per column, each adding its blocks in order; the 16 sums are then added in order.
template <typename P>
__global__ void __launch_bounds__(1024)
layernorm_bwd_params_kernel(const float* __restrict__ part, int blocks, int cols,
                            P* __restrict__ dgamma, P* __restrict__ dbeta) {
  __shared__ float s[16][64];
  P* out = blockIdx.y == 0 ? dgamma : dbeta;
  if (!out) return;
  const int cl = threadIdx.x % 64, rl = threadIdx.x / 64;
  const int c = blockIdx.x * 64 + cl;
  const float* p = part + (int64_t)blockIdx.y * blocks * cols;
  float v = 0.f;
  if (c < cols)
    for (int b = rl; b < blocks; b += 16) v += p[(int64_t)b * cols + c];
  s[rl][cl] = v;
  __syncthreads();
  if (rl == 0 && c < cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][cl];
    out[c] = from_f32<P>(t);
  }
}

constexpr int kFwdBlock = 256, kBwdBlock = 512;
constexpr int64_t kFwdGrid = 256 * 8, kBwdGrid = 512;

constexpr int block_of(int lpr, int block) { return lpr > block ? lpr : block; }

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
  const int lpr = row_shape(cols).lpr;
  const int64_t per = block_of(lpr, kBwdBlock) / lpr;
  const int64_t want = (rows + per - 1) / per;
  if (want <= 4) return 1;
  return std::min(want, kBwdGrid);
}

template <typename T, typename P, int LPR, int EPT>
hipError_t fwd(const LayerNormArgs& a, hipStream_t s) {
  constexpr int B = block_of(LPR, kFwdBlock);
  const int64_t blocks = std::min<int64_t>((a.rows + B / LPR - 1) / (B / LPR), kFwdGrid);
  hipLaunchKernelGGL((layernorm_fwd_kernel<T, P, LPR, EPT, B>), dim3((unsigned)blocks), dim3(B), 0,
                     s, static_cast<const T*>(a.x), a.ldx, static_cast<const P*>(a.gamma),
                     static_cast<const P*>(a.beta), a.rows, (int)a.cols, a.eps,
                     static_cast<T*>(a.y), a.mean, a.rstd);
  return hipGetLastError();
}

template <typename T, typename P, int LPR, int EPT>
hipError_t bwd(const LayerNormArgs& a, hipStream_t s) {
  constexpr int B = block_of(LPR, kBwdBlock);
  const int64_t blocks = bwd_blocks(a.rows, a.cols);
  float* part = blocks > 1 ? a.workspace : nullptr;
  hipLaunchKernelGGL((layernorm_bwd_kernel<T, P, LPR, EPT, B>), dim3((unsigned)blocks), dim3(B), 0,
                     s, static_cast<const T*>(a.dy), a.lddy, static_cast<const T*>(a.x), a.ldx,
                     a.mean, a.rstd, static_cast<const P*>(a.gamma), a.rows, (int)a.cols,
                     static_cast<T*>(a.y), static_cast<P*>(a.dgamma), static_cast<P*>(a.dbeta),
                     part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !part || (!a.dgamma && !a.dbeta)) return e;
  hipLaunchKernelGGL((layernorm_bwd_params_kernel<P>), dim3((unsigned)((a.cols + 63) / 64), 2),
                     dim3(1024), 0, s, part, (int)blocks, (int)a.cols, static_cast<P*>(a.dgamma),
                     static_cast<P*>(a.dbeta));
  return hipGetLastError();
}

template <typename T, typename P>
hipError_t by_shape(const LayerNormArgs& a, bool backward, hipStream_t s) {
  const Shape k = row_shape(a.cols);
#define FP8LIN_LN(L, E) \
  if (k.lpr == L && k.ept == E) return backward ? bwd<T, P, L, E>(a, s) : fwd<T, P, L, E>(a, s);
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
  return b > 1 ? 2 * b * cols * (int64_t)sizeof(float) : 0;
}

hipError_t launch_layernorm(const LayerNormArgs& a, bool backward, hipStream_t s) {
  const bool same = a.param_dtype == a.dtype;
  if (a.dtype == kBF16)
    return same ? by_shape<BF16, BF16>(a, backward, s) : by_shape<BF16, float>(a, backward, s);
  if (a.dtype == kF16)
    return same ? by_shape<F16, F16>(a, backward, s) : by_shape<F16, float>(a, backward, s);
  return by_shape<float, float>(a, backward, s);
}

}  // namespace fp8lin
