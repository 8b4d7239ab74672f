// Tokens to their experts and back: the stable sort of the (token, choice) pairs by expert,
// the rows' exchange in both directions, and its gradients.
//
// Pair i = t * topk + j sends token t to expert idx[i]; an index outside [0, experts) drops
// the pair. Expert e's rows start at offsets[e] in the sorted buffer, in the order of their
// pairs, and fill a multiple of `multiple` rows (FP8 GEMMs take token counts in multiples of
// 16). slot[i] is the pair's row or -1; source[r] is row r's pair or -1 for a padding row.
//
//   dispatch      xs[slot[t, j]] = x[t], padding rows 0
//   combine       y[t] = sum_j w[t, j] ys[slot[t, j]]          (w = 1: dispatch's gradient)
//   combine_bwd   dys[slot[t, j]] = w[t, j] dy[t], padding rows 0;
//                 dw[t, j] = sum_c dy[t, c] ys[slot[t, j], c]
//
// The exchanges only move rows, so memory bounds them: each token row is read once and
// written to its rows (no gather that reads it topk times), each sorted row is read or
// written once. slot and source come from the caller, so every entry is checked against the
// buffers before it is used as an address.
#include <algorithm>

#include "launch.h"
#include "rows.h"

namespace fp8lin {

namespace {

// ------------------------------------------------------------------------------ sort

constexpr int kSortBlock = 1024, kSortWaves = kSortBlock / 64;
constexpr int64_t kSortChunk = 16384;     // pairs per workgroup, up to kSortGrid workgroups
constexpr int64_t kSortGrid = 256;

__device__ __forceinline__ int expert_of(int32_t v, int experts) {
  return v >= 0 && v < experts ? v : -1;
}
__device__ __forceinline__ int expert_of(int64_t v, int experts) {
  return v >= 0 && v < experts ? (int)v : -1;
}

// Pairs [p0, p1) of workgroup b; wave w of it walks [w0, w1), 64 pairs a step.
struct Span { int64_t p0, p1; };
__device__ __forceinline__ Span wave_span(int64_t pairs, int64_t chunk) {
  const int64_t per = chunk / kSortWaves;                 // chunk is a multiple of 64 * waves
  const int64_t a = (int64_t)blockIdx.x * chunk + (int64_t)(threadIdx.x / 64) * per;
  const int64_t b = a + per;
  return {a < pairs ? a : pairs, b < pairs ? b : pairs};
}

// Count this wave's pairs by expert into cnt[experts] (LDS, this wave's own).
template <typename I>
__device__ __forceinline__ void count_span(const I* idx, Span sp, int experts, int* cnt) {
  const int lane = threadIdx.x % 64;
  for (int64_t p = sp.p0 + lane; p < sp.p1; p += 64) {
    const int e = expert_of(idx[p], experts);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
}

// Per-workgroup counts by expert, for a sort over several workgroups.
template <typename I>
__global__ void __launch_bounds__(kSortBlock)
moe_count_kernel(const I* __restrict__ idx, int64_t pairs, int64_t chunk, int experts,
                 int32_t* __restrict__ block_counts) {
  __shared__ int cnt[kMoeMaxExperts];
  for (int e = threadIdx.x; e < experts; e += kSortBlock) cnt[e] = 0;
  __syncthreads();
  count_span(idx, wave_span(pairs, chunk), experts, cnt);
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kSortBlock)
    block_counts[(int64_t)blockIdx.x * experts + e] = cnt[e];
}

// The sort. A stable rank is: pairs of the same expert in earlier workgroups, in earlier
// waves of this workgroup, in earlier steps of this wave, and in lower lanes of this step.
// The last comes from one ballot per bit of the expert index: the lanes that agree in every
// bit are the same expert's. Counts are integers, so nothing depends on the atomics' order.
template <typename I>
__global__ void __launch_bounds__(kSortBlock)
moe_sort_kernel(const I* __restrict__ idx, int64_t pairs, int64_t chunk, int experts, int bits,
                int multiple, int64_t rows, const int32_t* __restrict__ block_counts,
                int32_t* __restrict__ slot, int32_t* __restrict__ source,
                int32_t* __restrict__ counts, int32_t* __restrict__ offsets) {
  extern __shared__ int lds[];                 // next[waves][experts], then total[experts]
  __shared__ int wave_sum[kSortWaves];
  int* next = lds;
  int* total = lds + kSortWaves * experts;     // the expert's pairs, then its padded end
  const int t = threadIdx.x, lane = t % 64, wave = t / 64;
  for (int i = t; i < kSortWaves * experts; i += kSortBlock) next[i] = 0;
  __syncthreads();
  const Span sp = wave_span(pairs, chunk);
  count_span(idx, sp, experts, next + wave * experts);
  __syncthreads();
  // thread e: expert e's pairs over all workgroups and before this one
  int tot = 0, before = 0;
  if (t < experts) {
    if (gridDim.x == 1) {
      for (int w = 0; w < kSortWaves; ++w) tot += next[w * experts + t];
    } else {
      for (int b = 0; b < (int)gridDim.x; ++b) {
        const int c = block_counts[(int64_t)b * experts + t];
        tot += c;
        if (b < (int)blockIdx.x) before += c;
      }
    }
  }
  const int padded = (tot + multiple - 1) / multiple * multiple;
  // inclusive prefix of the padded counts over the threads
  int pre = padded;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(pre, off, 64);
    if (lane >= off) pre += o;
  }
  if (lane == 63) wave_sum[wave] = pre;
  __syncthreads();
  for (int w = 0; w < wave; ++w) pre += wave_sum[w];
  const int start = pre - padded;
  if (t < experts) {
    int at = start + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = next[w * experts + t];
      next[w * experts + t] = at;
      at += c;
    }
    total[t] = pre;
    if (blockIdx.x == 0) {
      counts[t] = tot;
      offsets[t + 1] = pre;
      if (t == 0) offsets[0] = 0;
    }
    // this expert's padding rows, by one workgroup
    if (t % (int)gridDim.x == (int)blockIdx.x)
      for (int r = start + tot; r < pre; ++r) source[r] = -1;
  }
  __syncthreads();
  // rows past the last expert's
  for (int64_t r = total[experts - 1] + (int64_t)blockIdx.x * kSortBlock + t; r < rows;
       r += (int64_t)gridDim.x * kSortBlock)
    source[r] = -1;
  volatile int* mine = next + wave * experts;
  for (int64_t p0 = sp.p0; p0 < sp.p1; p0 += 64) {
    const int64_t p = p0 + lane;
    const bool in = p < sp.p1;
    const int e = in ? expert_of(idx[p], experts) : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t m = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? m : ~m;
    }
    int row = -1;
    if (e >= 0) {
      const int rank = __popcll(same & ((1ull << lane) - 1));
      row = mine[e] + rank;
      // the wave runs in step: every lane has read the counter before the lowest adds to it
      __builtin_amdgcn_wave_barrier();
      if (rank == 0) mine[e] = row + __popcll(same);
      source[row] = (int32_t)p;
    }
    __builtin_amdgcn_wave_barrier();
    if (in) slot[p] = row;
  }
}

// -------------------------------------------------------------------------- exchanges

constexpr int kMoveBlock = 256, kMovePieces = 4;           // 4 KiB of a row per wave
constexpr int kMoveBytes = 64 * 16 * kMovePieces;
constexpr int kZeroRows = 8;                               // rows checked by a wave

// 16 bytes of a row of `bytes` bytes (a multiple of 2) at byte b; the row's last piece may be
// cut off at its end.
__device__ __forceinline__ piece_t ld_bytes(const uint8_t* row, int64_t b, int64_t bytes) {
  if (b + 16 <= bytes) return ld_piece(row + b);
  piece_t v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (b + 2 * i < bytes)
      v[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + b + 2 * i) << (16 * (i & 1));
  return v;
}
__device__ __forceinline__ void st_bytes(uint8_t* row, int64_t b, int64_t bytes, piece_t v) {
  if (b + 16 <= bytes) {
    st_piece(row + b, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (b + 2 * i < bytes)
      *reinterpret_cast<uint16_t*>(row + b + 2 * i) = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
}

// Zero the padding rows among rows [r0, r0 + kZeroRows), bytes [b0, b0 + kMoveBytes).
__device__ __forceinline__ void zero_padding(const int32_t* source, int64_t r0, int64_t rows,
                                             int64_t b0, int64_t bytes, uint8_t* out) {
  const int lane = threadIdx.x % 64;
  const int64_t r = r0 + lane;
  const bool pad = lane < kZeroRows && r < rows && source[r] < 0;
  uint64_t m = __ballot(pad);
  while (m) {
    const int i = __ffsll((unsigned long long)m) - 1;
    m &= m - 1;
    uint8_t* row = out + (r0 + i) * bytes;
#pragma unroll
    for (int v = 0; v < kMovePieces; ++v)
      st_bytes(row, b0 + (v * 64 + lane) * 16, bytes, piece_t{0, 0, 0, 0});
  }
}

// One wave per (token, 4 KiB of the row): loaded once, stored to each of the token's rows.
// The waves after those zero the padding rows.
__global__ void __launch_bounds__(kMoveBlock)
moe_dispatch_kernel(const uint8_t* __restrict__ x, int64_t ld_bytes_x,
                    const int32_t* __restrict__ slot, const int32_t* __restrict__ source,
                    int64_t tokens, int topk, int64_t rows, int64_t bytes, int64_t chunks,
                    uint8_t* __restrict__ xs) {
  const int lane = threadIdx.x % 64;
  int64_t u = (int64_t)blockIdx.x * (kMoveBlock / 64) + threadIdx.x / 64;
  if (u >= tokens * chunks) {
    u -= tokens * chunks;
    const int64_t r0 = u / chunks * kZeroRows;
    if (r0 < rows) zero_padding(source, r0, rows, u % chunks * kMoveBytes, bytes, xs);
    return;
  }
  const int64_t t = u / chunks, b0 = u % chunks * kMoveBytes;
  piece_t v[kMovePieces];
#pragma unroll
  for (int i = 0; i < kMovePieces; ++i)
    v[i] = ld_bytes(x + t * ld_bytes_x, b0 + (i * 64 + lane) * 16, bytes);
  for (int j = 0; j < topk; ++j) {
    const int r = slot[t * topk + j];
    if (r < 0 || r >= rows) continue;
#pragma unroll
    for (int i = 0; i < kMovePieces; ++i)
      st_bytes(xs + r * bytes, b0 + (i * 64 + lane) * 16, bytes, v[i]);
  }
}

constexpr int kSumPieces = 2;                              // 16-byte pieces of a row per lane

// One wave per (token, 2 KiB of the row): the token's rows, four in flight, summed in the
// order of the choices in float32 and rounded once.
template <typename T>
__global__ void __launch_bounds__(kMoveBlock)
moe_combine_kernel(const T* __restrict__ ys, int64_t ldys, const int32_t* __restrict__ slot,
                   const float* __restrict__ weights, int64_t tokens, int topk, int64_t rows,
                   int cols, int chunks, T* __restrict__ y) {
  constexpr int N = Piece<T>::N, U = 4;
  const int lane = threadIdx.x % 64;
  const int64_t u = (int64_t)blockIdx.x * (kMoveBlock / 64) + threadIdx.x / 64;
  if (u >= tokens * chunks) return;
  const int64_t t = u / chunks;
  const int c0 = ((int)(u % chunks) * kSumPieces * 64 + lane) * N;
  float acc[kSumPieces][N];
#pragma unroll
  for (int i = 0; i < kSumPieces; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) acc[i][n] = 0.f;
  for (int j0 = 0; j0 < topk; j0 += U) {
    piece_t v[U][kSumPieces];
    float w[U];
    bool live[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int j = j0 + q;
      const int r = j < topk ? slot[t * topk + j] : -1;
      live[q] = r >= 0 && r < rows;
      w[q] = live[q] && weights ? weights[t * topk + j] : 1.f;
#pragma unroll
      for (int i = 0; i < kSumPieces; ++i)
        v[q][i] = live[q] ? ld_row(ys + r * ldys, c0 + i * 64 * N, cols) : piece_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (!live[q]) continue;
#pragma unroll
      for (int i = 0; i < kSumPieces; ++i) {
        float f[N];
        unpack(v[q][i], f, T{});
#pragma unroll
        for (int n = 0; n < N; ++n) acc[i][n] += w[q] * f[n];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kSumPieces; ++i)
    st_row(y + t * cols, c0 + i * 64 * N, cols, pack(acc[i], T{}));
}

constexpr int kDotChoices = 8;                             // choices per walk over the row

// One workgroup per token: it reads dy[t] once per 8 choices, writes w dy to their rows and
// sums dy ys of each (lanes, then waves, in a fixed order). The workgroups after the tokens'
// zero the padding rows.
template <typename T>
__global__ void __launch_bounds__(kMoveBlock)
moe_combine_bwd_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ ys,
                       int64_t ldys, const int32_t* __restrict__ slot,
                       const int32_t* __restrict__ source, const float* __restrict__ weights,
                       int64_t tokens, int topk, int64_t rows, int cols, int chunks,
                       T* __restrict__ dys, float* __restrict__ dw) {
  constexpr int N = Piece<T>::N, J = kDotChoices, WAVES = kMoveBlock / 64;
  __shared__ float part[WAVES][J];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int64_t t = blockIdx.x;
  if (t >= tokens) {
    const int64_t u = (t - tokens) * WAVES + wave;
    const int64_t r0 = u / chunks * kZeroRows;
    if (r0 < rows)
      zero_padding(source, r0, rows, u % chunks * kMoveBytes, (int64_t)cols * sizeof(T),
                   reinterpret_cast<uint8_t*>(dys));
    return;
  }
  const T* g = dy + t * lddy;
  for (int j0 = 0; j0 < topk; j0 += J) {
    int r[J];
    float w[J], dot[J];
#pragma unroll
    for (int q = 0; q < J; ++q) {
      const int j = j0 + q;
      r[q] = j < topk ? slot[t * topk + j] : -1;
      if (r[q] >= rows) r[q] = -1;
      w[q] = r[q] >= 0 ? weights[t * topk + j] : 0.f;
      dot[q] = 0.f;
    }
    for (int c = threadIdx.x * N; c < cols; c += kMoveBlock * N) {
      float fg[N];
      unpack(ld_row(g, c, cols), fg, T{});
#pragma unroll
      for (int q = 0; q < J; ++q) {
        if (r[q] < 0) continue;
        float fy[N], o[N];
        unpack(ld_row(ys + r[q] * ldys, c, cols), fy, T{});
#pragma unroll
        for (int n = 0; n < N; ++n) {
          dot[q] += fg[n] * fy[n];
          o[n] = w[q] * fg[n];
        }
        st_row(dys + (int64_t)r[q] * cols, c, cols, pack(o, T{}));
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < J; ++q) {
      const float d = lanes_sum<64>(dot[q]);
      if (lane == 0) part[wave][q] = d;
    }
    __syncthreads();
    if (threadIdx.x < J && j0 + (int)threadIdx.x < topk) {
      float d = 0.f;
#pragma unroll
      for (int k = 0; k < WAVES; ++k) d += part[k][threadIdx.x];
      dw[t * topk + j0 + threadIdx.x] = d;
    }
  }
}

int64_t sort_chunk(int64_t pairs) {
  // whole steps of every wave; more than kSortGrid chunks of kSortChunk become longer chunks
  int64_t c = kSortChunk;
  if (pairs > c * kSortGrid) c = (pairs + kSortGrid - 1) / kSortGrid;
  return (c + kSortBlock - 1) / kSortBlock * kSortBlock;
}

template <typename I>
hipError_t sort_launch(const MoeSortArgs& a, hipStream_t s) {
  const int64_t chunk = sort_chunk(a.pairs);
  const unsigned blocks = (unsigned)std::max<int64_t>(1, (a.pairs + chunk - 1) / chunk);
  int bits = 0;
  while ((1 << bits) < a.experts) ++bits;
  const I* idx = static_cast<const I*>(a.idx);
  if (blocks > 1) {
    hipLaunchKernelGGL((moe_count_kernel<I>), dim3(blocks), dim3(kSortBlock), 0, s, idx, a.pairs,
                       chunk, a.experts, a.workspace);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const unsigned lds = (kSortWaves + 1) * (unsigned)a.experts * sizeof(int);
  hipLaunchKernelGGL((moe_sort_kernel<I>), dim3(blocks), dim3(kSortBlock), lds, s, idx, a.pairs,
                     chunk, a.experts, bits, a.multiple, a.rows, a.workspace, a.slot, a.source,
                     a.counts, a.offsets);
  return hipGetLastError();
}

int64_t zero_units(int64_t rows, int64_t chunks) {
  return (rows + kZeroRows - 1) / kZeroRows * chunks;
}

template <typename T>
hipError_t combine(const MoeArgs& a, hipStream_t s) {
  const int per = kSumPieces * 64 * Piece<T>::N;
  const int chunks = (int)((a.cols + per - 1) / per);
  const int64_t blocks = (a.tokens * chunks + kMoveBlock / 64 - 1) / (kMoveBlock / 64);
  hipLaunchKernelGGL((moe_combine_kernel<T>), dim3((unsigned)blocks), dim3(kMoveBlock), 0, s,
                     static_cast<const T*>(a.ys), a.ldys, a.slot, a.weights, a.tokens, a.topk,
                     a.rows, (int)a.cols, chunks, static_cast<T*>(a.out));
  return hipGetLastError();
}

template <typename T>
hipError_t combine_bwd(const MoeArgs& a, hipStream_t s) {
  const int64_t bytes = a.cols * (int64_t)sizeof(T);
  const int chunks = (int)((bytes + kMoveBytes - 1) / kMoveBytes);
  const int waves = kMoveBlock / 64;
  const int64_t blocks = a.tokens + (zero_units(a.rows, chunks) + waves - 1) / waves;
  hipLaunchKernelGGL((moe_combine_bwd_kernel<T>), dim3((unsigned)blocks), dim3(kMoveBlock), 0, s,
                     static_cast<const T*>(a.x), a.ldx, static_cast<const T*>(a.ys), a.ldys,
                     a.slot, a.source, a.weights, a.tokens, a.topk, a.rows, (int)a.cols, chunks,
                     static_cast<T*>(a.out), a.dw);
  return hipGetLastError();
}

}  // namespace

int64_t moe_sort_workspace(int64_t pairs, int32_t experts) {
  const int64_t chunk = sort_chunk(pairs), blocks = (pairs + chunk - 1) / chunk;
  return blocks > 1 ? blocks * experts * (int64_t)sizeof(int32_t) : 0;
}

hipError_t launch_moe_sort(const MoeSortArgs& a, hipStream_t s) {
  return a.idx_bytes == 8 ? sort_launch<int64_t>(a, s) : sort_launch<int32_t>(a, s);
}

hipError_t launch_moe_dispatch(const MoeArgs& a, hipStream_t s) {
  const int64_t es = a.dtype == kF32 ? 4 : 2, bytes = a.cols * es;
  const int64_t chunks = (bytes + kMoveBytes - 1) / kMoveBytes;
  const int waves = kMoveBlock / 64;
  const int64_t blocks = (a.tokens * chunks + zero_units(a.rows, chunks) + waves - 1) / waves;
  hipLaunchKernelGGL(moe_dispatch_kernel, dim3((unsigned)blocks), dim3(kMoveBlock), 0, s,
                     static_cast<const uint8_t*>(a.x), a.ldx * es, a.slot, a.source, a.tokens,
                     a.topk, a.rows, bytes, chunks, static_cast<uint8_t*>(a.out));
  return hipGetLastError();
}

hipError_t launch_moe_combine(const MoeArgs& a, hipStream_t s) {
  if (a.dtype == kBF16) return combine<BF16>(a, s);
  return a.dtype == kF16 ? combine<F16>(a, s) : combine<float>(a, s);
}

hipError_t launch_moe_combine_bwd(const MoeArgs& a, hipStream_t s) {
  if (a.dtype == kBF16) return combine_bwd<BF16>(a, s);
  return a.dtype == kF16 ? combine_bwd<F16>(a, s) : combine_bwd<float>(a, s);
}

}  // namespace fp8lin
