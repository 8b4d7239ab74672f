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
// against about 8 and 14 flops an element. Measured on one MI355X, where a large copy reaches
// 5.2 TB/s: forward 8192x4096 bf16 24.2 us, 5.5 TB/s; backward 8192x4096 bf16 40.6 us for the
// rows, 4.9 TB/s, and 4.8 us for the partial sums; 4096x14336 f32 124 and 5.8 us, 5.7 TB/s.
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

// Which lanes own a row. Narrow rows take 16 or 64 lanes (LPR); wide ones (LPR = 0) as many
// whole waves as their pieces fill, a value of the launch, since rounding it up to a power of two
// would leave almost half the lanes without elements just above one (8000x4104 bf16 forward 31.5
// us, with five waves 27.1 us; 4000x9000 50.0 and 35.5 us; backward 8000x4104 56.5 and 51.5 us).
// For a whole wave or more the row is the same in all lanes of a wave, so that row addresses are
// scalar.
struct Lanes {
  int per_row, lane, group, groups;       // lanes of a row, this one; the row of a turn, rows of it
};
template <int LPR>
__device__ __forceinline__ Lanes lanes_of(int row_waves) {
  const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t / 64);
  if constexpr (LPR == 0) {
    const int g = wave / row_waves;
    return {row_waves * 64, (wave - g * row_waves) * 64 + t % 64, g,
            (int)(blockDim.x / 64) / row_waves};
  } else {
    return {LPR, t % LPR, LPR == 64 ? wave : t / LPR, (int)blockDim.x / LPR};
  }
}

// The row of a group in the turn that starts at r0. A group past the last row works on that
// row and stores nothing, so that every group takes the same number of turns and the barriers
// in a row's sums always meet.
__device__ __forceinline__ int64_t turn_row(int64_t r0, int group, int64_t rows) {
  return r0 + group < rows ? r0 + group : rows - 1;
}

// This lane's pieces of a row, not yet cut at its end.
template <Cache C, int LPR, Fill FILL = kZero, typename T, int NV>
__device__ __forceinline__ void ld_rows(const T* row, const Lanes& l, int cols,
                                        piece_t (&p)[NV]) {
#pragma unroll
  for (int v = 0; v < NV; ++v)
    p[v] = ld_raw<C, LPR == 16, FILL>(row, (v * l.per_row + l.lane) * Piece<T>::N, cols);
}

// Sum over the lanes of a row. Rows of several waves meet in LDS (`part`, one float per wave of
// the workgroup); the caller alternates buffers so that one barrier per sum is enough.
constexpr int kMaxWaves = 16;
__device__ __forceinline__ float waves_sum(const float* part, const Lanes& l) {
  const int i = threadIdx.x % kMaxWaves, w = l.per_row / 64;
  return lanes_sum<kMaxWaves>(i < w ? part[l.group * w + i] : 0.f);
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v, float* part, const Lanes& l) {
  v = lanes_sum<(LPR == 16 ? 16 : 64)>(v);
  if constexpr (LPR == 0) {
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = v;
    __syncthreads();
    v = waves_sum(part, l);
  }
  return v;
}

// The forward's workgroups are short (eight to a compute unit), the backward's hold one unit
// each: 16 waves of 128 registers, and as few rows of partial sums as that allows. Backward of
// 8192x4096 bf16: 45.0 us so, 45.3 us with twice as many workgroups of 512, 48.1 us with four
// times as many of 256; of 1021x5003 f16 21.4, 22.5 and 22.6 us, and with half the workgroups
// 24.6 us. The forward of 8192x4096 does not depend on its grid (23.0 to 23.7 us).
constexpr int kFwdBlock = 256, kBwdBlock = 1024, kMaxBlock = 64 * kMaxWaves;
constexpr int64_t kFwdGrid = 256 * 8, kBwdGrid = 256;

// Lane l of a row's n holds the pieces l, l + n, ... (EPT elements). A workgroup walks the rows
// with the grid's stride; the other workgroups of its compute unit cover its waits, which takes
// registers better than loading the next row ahead does (2000x16384 bf16 33.8 us, ahead 38.6 us;
// 2000x12000 f32 39.7 and 56.5 us; 8192x4096 bf16 23.7 us either way). Holding gamma and beta is
// worth theirs: read again for every row 8192x4096 bf16 takes 34.0 us.
template <typename T, int LPR, int EPT, Cache LOAD>
__global__ void __launch_bounds__(LPR ? kFwdBlock : kMaxBlock)
layernorm_fwd_kernel(const T* __restrict__ x, int64_t ldx, const void* __restrict__ gamma,
                     const void* __restrict__ beta, bool params_f32, int64_t rows, int cols,
                     int row_waves, float eps, T* __restrict__ y, float* __restrict__ mean_out,
                     float* __restrict__ rstd_out) {
  constexpr int N = Piece<T>::N, NV = EPT / N;
  // gamma and beta stay in registers beside the row up to 16 elements a lane
  constexpr bool kHeld = EPT <= 16;
  __shared__ float part[2][kMaxWaves];
  const Lanes l = lanes_of<LPR>(row_waves);
  const float fcols = (float)cols;
  const int64_t step = (int64_t)gridDim.x * l.groups;
  float gm[NV][N], bt[NV][N];
  if constexpr (kHeld) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      ld_params<T>(gamma, params_f32, (v * l.per_row + l.lane) * N, cols, 1.f, gm[v]);
      ld_params<T>(beta, params_f32, (v * l.per_row + l.lane) * N, cols, 0.f, bt[v]);
    }
  }
  for (int64_t r0 = (int64_t)blockIdx.x * l.groups; r0 < rows; r0 += step) {
    piece_t p[NV];
    ld_rows<LOAD, LPR>(x + turn_row(r0, l.group, rows) * ldx, l, cols, p);
    const int64_t r = r0 + l.group;
    float f[NV][N];
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      unpack(cut<T>(p[v], (v * l.per_row + l.lane) * N, cols), f[v], T{});
#pragma unroll
      for (int i = 0; i < N; ++i) s += f[v][i];
    }
    const float mean = row_sum<LPR>(s, part[0], l) / fcols;
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * l.per_row + l.lane) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[v][i] -= mean;
        const float d = c + i < cols ? f[v][i] : 0.f;
        q = __builtin_fmaf(d, d, q);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<LPR>(q, part[1], l) / fcols + eps);
    if (r < rows) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float o[N];
        if constexpr (!kHeld) {
          __builtin_amdgcn_sched_barrier(0);
          ld_params<T>(gamma, params_f32, (v * l.per_row + l.lane) * N, cols, 1.f, gm[v]);
          ld_params<T>(beta, params_f32, (v * l.per_row + l.lane) * N, cols, 0.f, bt[v]);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = __builtin_fmaf(f[v][i] * rstd, gm[v][i], bt[v][i]);
        st_row<kStream>(y + r * cols, (v * l.per_row + l.lane) * N, cols, pack(o, T{}));
      }
      if (l.lane == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
      }
    }
  }
}

// Columns c to c + 3 of the groups' sums, added in the order of the groups; their number is known
// to the loop, so that its reads are in flight together.
template <int G>
__device__ __forceinline__ f32x4_t sum_of(const float* fold, int width, int c) {
  f32x4_t s = *reinterpret_cast<const f32x4_t*>(fold + c);
#pragma unroll
  for (int k = 1; k < G; ++k) s += *reinterpret_cast<const f32x4_t*>(fold + k * width + c);
  return s;
}
template <int LPR>
__device__ __forceinline__ f32x4_t groups_sum(const float* fold, int width, int groups, int c) {
  if constexpr (LPR > 0) return sum_of<kMaxWaves>(fold, width, c);      // a wave's are one
  if (groups == 2) return sum_of<2>(fold, width, c);      // 16 waves by the waves of a row
  if (groups == 3) return sum_of<3>(fold, width, c);
  if (groups == 4) return sum_of<4>(fold, width, c);
  return groups == 5 ? sum_of<5>(fold, width, c) : sum_of<8>(fold, width, c);
}

// The gradient in one pass over dy and x, the next row loaded while this one is worked on.
// Lanes own columns as in the forward, so each also sums dy xh and dy of its columns over the
// workgroup's rows, in registers; at the end the workgroup's row groups are added in LDS in
// group order and written as one row of partial sums, part[which][block][part_ld], which
// layernorm_bwd_params_kernel adds in a fixed order. A single workgroup (one row of more than 16384
// columns, or none) writes dgamma and dbeta itself; two rows take another launch rather than
// another turn (2x16388 bf16 18.9 us, in turns 35.5 us; 4x32768 f32 38.3 and 90.4 us). Every
// order is fixed, so results repeat.
//
// Loading ahead took 8192x4096 bf16 from 57.6 to 44.2 us, 4096x14336 f32 from 177 to 143 us.
// A wave has 128 registers (16 waves a compute unit). What does not fit beside the two sums:
// gamma (then in LDS), the next row (then not loaded ahead), and above 16384 columns, for every
// type, this row itself (then read again, from the cache, for dx). The count leaves no room for
// addresses and for cutting a row off: the compiler spills 3 registers a lane of float32 rows of
// 513 to 1024 columns, 7 where they are cut off, 17 of cut-off float32 rows of 1025 to 16384
// columns (4000x5003 62.6 us, 4000x5004 51.5 us), and 48 to 196 of all rows above 16384
// (1000x20000 bf16 102 us for 120 MB).
template <typename T, int EPT> struct BwdFit {
  static constexpr int kRow = 2 * EPT * (int)sizeof(T) / 4, kSums = 2 * EPT;
  static constexpr bool kHold = kRow + kSums < 96;
  static constexpr bool kAhead = 2 * kRow + kSums <= 96;
  static constexpr bool kGammaLds = (kAhead ? 2 : 1) * kRow + kSums + EPT > 96;
};

template <typename T, int LPR, int EPT, Cache LOAD, Cache STORE, bool RAGGED>
__global__ void __launch_bounds__(kMaxBlock)
layernorm_bwd_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx,
                     const float* __restrict__ mean, const float* __restrict__ rstd,
                     const void* __restrict__ gamma, bool params_f32, int64_t rows, int cols,
                     int row_waves, T* __restrict__ dx, void* __restrict__ dgamma,
                     void* __restrict__ dbeta, float* __restrict__ part, int part_ld) {
  using Fit = BwdFit<T, EPT>;
  constexpr int N = Piece<T>::N, NV = EPT / N;
  constexpr bool kGammaLds = Fit::kGammaLds, kHold = Fit::kHold, kAhead = Fit::kAhead;
  __shared__ float red[2][2][kMaxWaves];
  // the groups' sums before they are added, or gamma of one row
  __shared__ __attribute__((aligned(16))) float fold[kMaxBlock * EPT];
  const Lanes l = lanes_of<LPR>(row_waves);
  const float fcols = (float)cols;
  const int64_t step = (int64_t)gridDim.x * l.groups;
  piece_t cx[NV], cd[NV], nx[NV], nd[NV];      // this row of x and dy, and the next
  float mu = 0.f, rs = 0.f, nmu = 0.f, nrs = 0.f;
  if (kAhead && (int64_t)blockIdx.x * l.groups < rows) {
    const int64_t r = turn_row((int64_t)blockIdx.x * l.groups, l.group, rows);
    ld_rows<LOAD, LPR, kOwn>(x + r * ldx, l, cols, cx);
    ld_rows<LOAD, LPR>(dy + r * lddy, l, cols, cd);
    mu = mean[r], rs = rstd[r];
  }
  float gm[kGammaLds ? 1 : NV][N], ag[NV][N], ab[NV][N];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if constexpr (kGammaLds) {
      float g[N];
      ld_params<T>(gamma, params_f32, (v * l.per_row + l.lane) * N, cols, 1.f, g);
      if (l.group == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) fold[(v * l.per_row + l.lane) * N + i] = g[i];
    } else {
      ld_params<T>(gamma, params_f32, (v * l.per_row + l.lane) * N, cols, 1.f, gm[v]);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) ag[v][i] = ab[v][i] = 0.f;
  }
  if (kGammaLds && l.groups > 1) __syncthreads();     // one row group's lanes read their own
  auto gamma_of = [&](int v, int i) {
    if constexpr (kGammaLds) return fold[(v * l.per_row + l.lane) * N + i];
    else return gm[v][i];
  };
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * l.groups; r0 < rows; r0 += step, turn ^= 1) {
    const int64_t r = r0 + l.group;
    const bool live = r < rows;
    const int64_t q = turn_row(kAhead ? r0 + step : r0, l.group, rows);
    if (!kAhead) {
      if constexpr (kHold) {
        ld_rows<LOAD, LPR, kOwn>(x + q * ldx, l, cols, cx);
        ld_rows<LOAD, LPR>(dy + q * lddy, l, cols, cd);
      }
      mu = mean[q], rs = rstd[q];
    } else if (r0 + step < rows) {
      ld_rows<LOAD, LPR, kOwn>(x + q * ldx, l, cols, nx);
      ld_rows<LOAD, LPR>(dy + q * lddy, l, cols, nd);
      nmu = mean[q], nrs = rstd[q];
    }
    // a group past the last row takes its turn (the barriers must meet) with dy = 0
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * l.per_row + l.lane) * N;
      float fx[N], fd[N];
      if constexpr (!kHold) {
        cx[v] = ld_raw<LOAD, false>(x + q * ldx, c, cols);
        cd[v] = ld_raw<LOAD, false>(dy + q * lddy, c, cols);
      }
      if constexpr (RAGGED) {
        cx[v] = cut<T, kHold ? kOwn : kZero>(cx[v], c, cols);
        cd[v] = cut<T>(cd[v], c, cols);
      }
      // past the row dy is 0 and x is some of the row's own values: nothing is added, and a NaN
      // there is one that the row has anyway (with x = 0 instead, -mean * rstd may leave float32
      // for a row of one large value). Rows that do not stay in registers are cut to 0 and xh
      // with them, which takes fewer (1000x20001 bf16 123.9 us, 129.6 us the other way)
      if (!live || c >= cols) cd[v] = piece_t{0, 0, 0, 0};
      unpack(cx[v], fx, T{});
      unpack(cd[v], fd, T{});
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float xh = (fx[i] - mu) * rs;
        if constexpr (RAGGED && !kHold) xh = c + i < cols ? xh : 0.f;
        const float g = fd[i] * gamma_of(v, i);
        s1 += g;
        s2 = __builtin_fmaf(g, xh, s2);
      }
      if constexpr (!kHold || kGammaLds) __builtin_amdgcn_sched_barrier(0);
    }
    s1 = lanes_sum<(LPR == 16 ? 16 : 64)>(s1);
    s2 = lanes_sum<(LPR == 16 ? 16 : 64)>(s2);
    if constexpr (LPR == 0) {
      const int wave = threadIdx.x / 64;
      if (threadIdx.x % 64 == 0) { red[turn][0][wave] = s1; red[turn][1][wave] = s2; }
      __syncthreads();
      s1 = waves_sum(red[turn][0], l);
      s2 = waves_sum(red[turn][1], l);
    }
    if (kAhead) {
#pragma unroll
      for (int v = 0; v < NV; ++v) { arrived(nx[v]); arrived(nd[v]); }
    }
    const float m1 = s1 / fcols, m2 = s2 / fcols;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * l.per_row + l.lane) * N;
      float fx[N], fd[N], o[N];
      if constexpr (kHold) {
        // from the 16 bytes again: the floats of the first sums would not fit
        arrived(cx[v]);
        arrived(cd[v]);
      } else {
        cx[v] = ld_raw<LOAD, false>(x + q * ldx, c, cols);
        cd[v] = ld_raw<LOAD, false>(dy + q * lddy, c, cols);
        if constexpr (RAGGED) {
          cx[v] = cut<T>(cx[v], c, cols);
          cd[v] = cut<T>(cd[v], c, cols);
        }
        if (!live || c >= cols) cd[v] = piece_t{0, 0, 0, 0};
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
      if (live && dx) {
        if constexpr (RAGGED) st_row<STORE>(dx + r * cols, c, cols, pack(o, T{}));
        else if (c < cols) st_piece<STORE>(elem_at(dx + r * cols, c), pack(o, T{}));
      }
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
    if (l.groups > 1) {
      __syncthreads();
      const int width = l.per_row * EPT;
      // the four groups of a wave of narrow rows are added among its lanes first
      const int at = (LPR == 16 ? (int)threadIdx.x / 64 : l.group) * width;
      const bool writes = LPR != 16 || threadIdx.x % 64 < 16;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if constexpr (LPR == 16)
#pragma unroll
          for (int i = 0; i < N; ++i) acc[v][i] = lanes_sum<64, 16>(acc[v][i]);
        if (!writes) continue;
#pragma unroll
        for (int i = 0; i < N; i += 4)
          *reinterpret_cast<f32x4_t*>(&fold[at + (v * l.per_row + l.lane) * N + i]) =
              f32x4_t{acc[v][i], acc[v][i + 1], acc[v][i + 2], acc[v][i + 3]};
      }
      __syncthreads();
      // rows of so few lanes that there are several groups never come to a single workgroup
      // (by_columns takes those), so dst is there; part_ld is cols rounded up to 4
      for (int c = threadIdx.x * 4; c < cols; c += blockDim.x * 4)
        *reinterpret_cast<sums_t*>(dst + c) = groups_sum<LPR>(fold, width, l.groups, c);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const int c = (v * l.per_row + l.lane) * N + i;
          if (dst) {
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

// The gradient of few rows: dx by rows, and dgamma and dbeta by columns, with dy and x read again
// from the caches. Workgroups of a row or two would write more partial sums than they read (8
// bytes a column each). Neither part needs the other, so one launch holds both kinds of
// workgroup.
template <typename T, int LPR, int EPT>
__device__ __forceinline__ void dx_rows(int block, int blocks, const T* __restrict__ dy,
                                        int64_t lddy, const T* __restrict__ x, int64_t ldx,
                                        const float* __restrict__ mean,
                                        const float* __restrict__ rstd,
                                        const void* __restrict__ gamma, bool params_f32,
                                        int64_t rows, int cols, int row_waves,
                                        T* __restrict__ dx) {
  constexpr int N = Piece<T>::N, NV = EPT / N;
  __shared__ float red[2][2][kMaxWaves];
  const Lanes l = lanes_of<LPR>(row_waves);
  const float fcols = (float)cols;
  const int64_t step = (int64_t)blocks * l.groups;
  float gm[NV][N];
#pragma unroll
  for (int v = 0; v < NV; ++v)
    ld_params<T>(gamma, params_f32, (v * l.per_row + l.lane) * N, cols, 1.f, gm[v]);
  int turn = 0;
  for (int64_t r0 = (int64_t)block * l.groups; r0 < rows; r0 += step, turn ^= 1) {
    const int64_t r = turn_row(r0, l.group, rows);
    piece_t cx[NV], cd[NV];
    ld_rows<kKeep, LPR, kOwn>(x + r * ldx, l, cols, cx);
    ld_rows<kKeep, LPR>(dy + r * lddy, l, cols, cd);
    const float mu = mean[r], rs = rstd[r];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * l.per_row + l.lane) * N;
      float fx[N], fd[N];
      cx[v] = cut<T, kOwn>(cx[v], c, cols);
      cd[v] = cut<T>(cd[v], c, cols);
      unpack(cx[v], fx, T{});
      unpack(cd[v], fd, T{});
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = (fx[i] - mu) * rs;
        const float g = fd[i] * gm[v][i];
        s1 += g;
        s2 = __builtin_fmaf(g, xh, s2);
      }
    }
    s1 = lanes_sum<(LPR == 16 ? 16 : 64)>(s1);
    s2 = lanes_sum<(LPR == 16 ? 16 : 64)>(s2);
    if constexpr (LPR == 0) {
      const int wave = threadIdx.x / 64;
      if (threadIdx.x % 64 == 0) { red[turn][0][wave] = s1; red[turn][1][wave] = s2; }
      __syncthreads();
      s1 = waves_sum(red[turn][0], l);
      s2 = waves_sum(red[turn][1], l);
    }
    const float m1 = s1 / fcols, m2 = s2 / fcols;
    if (r0 + l.group >= rows) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float fx[N], fd[N], o[N];
      unpack(cx[v], fx, T{});
      unpack(cd[v], fd, T{});
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = (fx[i] - mu) * rs;
        o[i] = rs * __builtin_fmaf(-xh, m2, __builtin_fmaf(fd[i], gm[v][i], -m1));
      }
      st_row<kKeep>(dx + r * cols, (v * l.per_row + l.lane) * N, cols, pack(o, T{}));
    }
  }
}

// A workgroup has 64 columns: the lanes of 128 bytes (256 of float32) a row, and as many rows at
// once as its lanes hold. A lane's rows are added in order, then the lanes, then the waves.
template <typename T>
__device__ __forceinline__ void sum_cols(int block, const T* __restrict__ dy, int64_t lddy,
                                         const T* __restrict__ x, int64_t ldx,
                                         const float* __restrict__ mean,
                                         const float* __restrict__ rstd, int64_t rows, int cols,
                                         bool params_f32, void* __restrict__ dgamma,
                                         void* __restrict__ dbeta) {
  constexpr int N = Piece<T>::N, LANES = 64 / N;
  __shared__ float sums[kMaxWaves][2][64];
  const int cl = threadIdx.x % LANES, c = block * 64 + cl * N;
  const int at_once = (int)blockDim.x / LANES;
  float ag[N], ab[N];
#pragma unroll
  for (int i = 0; i < N; ++i) ag[i] = ab[i] = 0.f;
  if (c < cols) {
    // bound by what one compute unit reads: more rows in flight change nothing
#pragma unroll 2
    for (int64_t r = threadIdx.x / LANES; r < rows; r += at_once) {
      const piece_t px = ld_raw<kKeep>(x + r * ldx, c, cols);
      const piece_t pd = ld_raw<kKeep>(dy + r * lddy, c, cols);
      const float mu = mean[r], rs = rstd[r];
      float fx[N], fd[N];
      unpack(cut<T>(px, c, cols), fx, T{});
      unpack(cut<T>(pd, c, cols), fd, T{});
#pragma unroll
      for (int i = 0; i < N; ++i) {
        ag[i] = __builtin_fmaf(fd[i], (fx[i] - mu) * rs, ag[i]);
        ab[i] += fd[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (LANES == 8) {                  // 8 lanes on, within 16
      ag[i] += dpp<0x128>(ag[i]);
      ab[i] += dpp<0x128>(ab[i]);
    }
    ag[i] = lanes_sum<64, 16>(ag[i]);
    ab[i] = lanes_sum<64, 16>(ab[i]);
  }
  if (threadIdx.x % 64 < LANES) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      sums[threadIdx.x / 64][0][cl * N + i] = ag[i];
      sums[threadIdx.x / 64][1][cl * N + i] = ab[i];
    }
  }
  __syncthreads();
  // 128 sums; a workgroup has 256 lanes at least
  const int which = threadIdx.x / 64, k = threadIdx.x % 64;
  void* out = which == 0 ? dgamma : dbeta;
  if (which < 2 && out && block * 64 + k < cols) {
    const int waves = (int)blockDim.x / 64;
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kMaxWaves; ++w) t += w < waves ? sums[w][which][k] : 0.f;
    st_param<T>(out, params_f32, block * 64 + k, t);
  }
}

// The first `col_blocks` workgroups take columns, the others rows.
template <typename T, int LPR, int EPT>
__global__ void __launch_bounds__(kMaxBlock)
layernorm_bwd_few_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x,
                         int64_t ldx, const float* __restrict__ mean,
                         const float* __restrict__ rstd, const void* __restrict__ gamma,
                         bool params_f32, int64_t rows, int cols, int row_waves, int col_blocks,
                         T* __restrict__ dx, void* __restrict__ dgamma,
                         void* __restrict__ dbeta) {
  const int block = blockIdx.x;
  if (block < col_blocks)
    sum_cols(block, dy, lddy, x, ldx, mean, rstd, rows, cols, params_f32, dgamma, dbeta);
  else
    dx_rows<T, LPR, EPT>(block - col_blocks, (int)gridDim.x - col_blocks, dy, lddy, x, ldx, mean,
                         rstd, gamma, params_f32, rows, cols, row_waves, dx);
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

// The kernel of a row of `cols` elements, the waves of a row where it has whole ones, and the
// lanes of a row. A lane's elements are 8, 16 or 32: with 16 a wave's 128 registers hold what the
// kernels keep.
struct Shape { int lpr, ept, waves, lanes; };
Shape row_shape(int64_t cols) {
  if (cols <= 16 * 8) return {16, 8, 0, 16};
  if (cols <= 64 * 8) return {64, 8, 1, 64};
  if (cols <= 64 * 16) return {64, 16, 1, 64};
  const int ept = cols <= kMaxBlock * 16 ? 16 : 32;
  const int waves = (int)((cols + 64 * ept - 1) / (64 * ept));
  return {0, ept, waves, 64 * waves};
}

// Rows of a turn: as many as the workgroup's size takes whole.
int groups_of(const Shape& k, int block) { return std::max(1, block / k.lanes); }

int64_t bwd_blocks(int64_t rows, int64_t cols) {
  const int64_t per = groups_of(row_shape(cols), kBwdBlock), want = (rows + per - 1) / per;
  return std::max<int64_t>(1, std::min(want, kBwdGrid));
}

template <typename T, int LPR, int EPT, Cache LOAD>
hipError_t fwd(const LayerNormArgs& a, const Shape& k, hipStream_t s) {
  const int groups = groups_of(k, kFwdBlock);
  const int64_t blocks = std::min<int64_t>((a.rows + groups - 1) / groups, kFwdGrid);
  hipLaunchKernelGGL((layernorm_fwd_kernel<T, LPR, EPT, LOAD>), dim3((unsigned)blocks),
                     dim3((unsigned)(groups * k.lanes)), 0, s, static_cast<const T*>(a.x), a.ldx,
                     a.gamma, a.beta, a.param_dtype == kF32, a.rows, (int)a.cols, k.waves, a.eps,
                     static_cast<T*>(a.y), a.mean, a.rstd);
  return hipGetLastError();
}

// RAGGED: the width is no whole number of pieces. Without the code for that, the kernels have
// registers to spare (8000x2048 f32 40.2 us, with it 47.2 us).
template <typename T, int LPR, int EPT, Cache LOAD, Cache STORE, bool RAGGED>
hipError_t bwd_kernel(const LayerNormArgs& a, const Shape& k, hipStream_t s) {
  const int64_t blocks = bwd_blocks(a.rows, a.cols);
  float* part = blocks > 1 ? a.workspace : nullptr;
  const int part_ld = (int)((a.cols + 3) / 4 * 4);
  hipLaunchKernelGGL((layernorm_bwd_kernel<T, LPR, EPT, LOAD, STORE, RAGGED>),
                     dim3((unsigned)blocks), dim3((unsigned)(groups_of(k, kBwdBlock) * k.lanes)), 0,
                     s, static_cast<const T*>(a.dy), a.lddy, static_cast<const T*>(a.x), a.ldx, a.mean,
                     a.rstd, a.gamma, a.param_dtype == kF32, a.rows, (int)a.cols, k.waves,
                     static_cast<T*>(a.y), a.dgamma, a.dbeta, part, part_ld);
  return hipGetLastError();
}

template <typename T, int LPR, int EPT, Cache LOAD, Cache STORE>
hipError_t bwd(const LayerNormArgs& a, const Shape& k, hipStream_t s) {
  return a.cols % Piece<T>::N ? bwd_kernel<T, LPR, EPT, LOAD, STORE, true>(a, k, s)
                              : bwd_kernel<T, LPR, EPT, LOAD, STORE, false>(a, k, s);
}

template <typename T, int LPR, int EPT>
hipError_t bwd_columns(const LayerNormArgs& a, const Shape& k, hipStream_t s) {
  const int groups = groups_of(k, kBwdBlock);
  const int64_t row_blocks = a.y ? (a.rows + groups - 1) / groups : 0;
  const int64_t col_blocks = a.dgamma || a.dbeta ? (a.cols + 63) / 64 : 0;
  hipLaunchKernelGGL((layernorm_bwd_few_kernel<T, LPR, EPT>),
                     dim3((unsigned)(row_blocks + col_blocks)),
                     dim3((unsigned)(groups * k.lanes)), 0, s, static_cast<const T*>(a.dy), a.lddy,
                     static_cast<const T*>(a.x), a.ldx, a.mean, a.rstd, a.gamma,
                     a.param_dtype == kF32, a.rows, (int)a.cols, k.waves, (int)col_blocks,
                     static_cast<T*>(a.y), a.dgamma, a.dbeta);
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

// Few rows take layernorm_bwd_few_kernel. The second reading costs by the rows, the partial sums
// by the width and another launch: 33x3776 bf16 4.6 us (with partial sums 9.7), 203x13184 9.2
// (19.7), 1000x512 6.5 (8.1), 2000x4096 15.7 (17.5), 1600x8192 21.5 (27.3), but 2000x512 11.6 (8.2)
// and 3000x4096 22.3 (21.2); 500x72 f32 5.5 (8.0), 1021x5003 21.3 (29.0), but 1000x1300 14.9
// (12.1). Above kFewBytes the caches do not hold dy and x until then (600x16384 f32 38.8 us, 35.1).
//
// Up to 16384 columns this takes all that bwd_blocks gives to one workgroup, no rows at all among
// it: that is one turn, at most 64 rows and 16384 elements.
constexpr int64_t kFewBytes = 32 << 20;
bool by_columns(int64_t rows, int64_t cols, int64_t elem) {
  return row_shape(cols).ept <= 16 && rows * elem <= 2000 + cols / 2 &&
         rows * cols * elem <= kFewBytes;
}

template <typename T, int LPR, int EPT>
hipError_t by_size(const LayerNormArgs& a, const Shape& k, bool backward, hipStream_t s) {
  const int64_t bytes = a.rows * a.cols * (int64_t)sizeof(T);
  if (!backward)
    return bytes <= kKeepRows ? fwd<T, LPR, EPT, kKeep>(a, k, s)
                              : fwd<T, LPR, EPT, kStream>(a, k, s);
  if constexpr (EPT <= 16)
    if (by_columns(a.rows, a.cols, sizeof(T))) return bwd_columns<T, LPR, EPT>(a, k, s);
  if (bytes <= kKeepGrad) return bwd<T, LPR, EPT, kKeep, kKeep>(a, k, s);
  return bytes <= kKeepRows ? bwd<T, LPR, EPT, kStream, kKeep>(a, k, s)
                            : bwd<T, LPR, EPT, kStream, kStream>(a, k, s);
}

template <typename T>
hipError_t by_shape(const LayerNormArgs& a, bool backward, hipStream_t s) {
  const Shape k = row_shape(a.cols);
  if (k.lpr == 16) return by_size<T, 16, 8>(a, k, backward, s);
  if (k.lpr == 64)
    return k.ept == 8 ? by_size<T, 64, 8>(a, k, backward, s)
                      : by_size<T, 64, 16>(a, k, backward, s);
  return k.ept == 16 ? by_size<T, 0, 16>(a, k, backward, s) : by_size<T, 0, 32>(a, k, backward, s);
}

}  // namespace

int64_t layernorm_bwd_workspace(int64_t rows, int64_t cols) {
  // for either size of element: by_columns with the larger takes the fewer sizes
  if (by_columns(rows, cols, sizeof(float))) return 0;
  const int64_t b = bwd_blocks(rows, cols);
  return b > 1 ? 2 * b * ((cols + 3) / 4 * 4) * (int64_t)sizeof(float) : 0;
}

namespace {
int64_t elem_size(int dtype) { return dtype == kF32 ? 4 : 2; }
}  // namespace

hipError_t launch_layernorm(const LayerNormArgs& a, bool backward, hipStream_t s) {
  const hipError_t e = a.dtype == kBF16  ? by_shape<BF16>(a, backward, s)
                       : a.dtype == kF16 ? by_shape<F16>(a, backward, s)
                                         : by_shape<float>(a, backward, s);
  if (e != hipSuccess || !backward || !a.workspace) return e;
  if (by_columns(a.rows, a.cols, elem_size(a.dtype))) return e;
  if (a.param_dtype == kBF16) return bwd_params<BF16>(a, s);
  return a.param_dtype == kF16 ? bwd_params<F16>(a, s) : bwd_params<float>(a, s);
}

}  // namespace fp8lin
