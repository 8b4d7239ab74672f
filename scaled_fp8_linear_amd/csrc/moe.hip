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
// The exchanges only move rows, so memory bounds them: each token row is read from memory once
// and written to its rows (a gather by sorted rows took 163 us where this takes 120), each
// sorted row is read or written once. slot and source come from the caller, so every entry is
// checked against the buffers before it is used as an address.
#include <algorithm>

#include "launch.h"
#include "moe_rows.h"
#include "rows.h"

namespace fp8lin {

namespace {

// ------------------------------------------------------------------------------ sort

// A workgroup ranks up to kSortBlock * S pairs, S to a lane, in registers; what it costs is the
// instructions of the ranking, about 0.8 us a step on one compute unit. So up to kSortOne pairs
// one workgroup does it all in one launch (4000 pairs 6.1 us); above, chunks of kSortBlock are
// counted first, and every workgroup adds up the counts of all; above kSortDirect of those,
// chunks of kSortLong, whose counts a launch between turns into starts.
constexpr int kSortBlock = 1024, kSortWaves = kSortBlock / 64;
constexpr int kSortSteps = 4, kSortShares = 16;
constexpr int64_t kSortOne = kSortSteps * kSortBlock, kSortLong = kSortOne, kSortDirect = 128;

__device__ __forceinline__ int expert_of(int32_t v, int experts) {
  return v >= 0 && v < experts ? v : -1;
}
__device__ __forceinline__ int expert_of(int64_t v, int experts) {
  return v >= 0 && v < experts ? (int)v : -1;
}

__device__ __forceinline__ int wave_index() {
  return __builtin_amdgcn_readfirstlane((int)threadIdx.x / 64);
}

// Bits of `mask` below this lane's.
__device__ __forceinline__ int lanes_below(uint64_t mask) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                        __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// The experts of this lane's S pairs (-1: none): wave w of the workgroup has the 64 S pairs
// from first_pair on, 64 a step.
template <int S>
__device__ __forceinline__ int64_t first_pair() {
  return ((int64_t)blockIdx.x * kSortWaves + wave_index()) * (64 * S);
}
template <int S, typename I>
__device__ __forceinline__ void ld_experts(const I* idx, int64_t p0, int64_t pairs, int experts,
                                           int (&e)[S]) {
  const int lane = threadIdx.x % 64;
  I v[S];
#pragma unroll
  for (int s = 0; s < S; ++s) v[s] = p0 + s * 64 + lane < pairs ? idx[p0 + s * 64 + lane] : (I)-1;
#pragma unroll
  for (int s = 0; s < S; ++s) e[s] = expert_of(v[s], experts);
}

// counts[block][expert] of the workgroup's pairs.
template <int S, typename I>
__global__ void __launch_bounds__(kSortBlock)
moe_count_kernel(const I* __restrict__ idx, int64_t pairs, int experts,
                 int32_t* __restrict__ block_counts) {
  __shared__ int cnt[kMoeMaxExperts];
  int e[S];
  ld_experts<S>(idx, first_pair<S>(), pairs, experts, e);
  for (int i = threadIdx.x; i < experts; i += kSortBlock) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int s = 0; s < S; ++s)
    if (e[s] >= 0) atomicAdd(&cnt[e[s]], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < experts; i += kSortBlock)
    block_counts[(int64_t)blockIdx.x * experts + i] = cnt[i];
}

// counts[block][expert] become the counts of the blocks before; totals[expert] their sum. A
// lane has an expert, a wave a share of the blocks.
__global__ void __launch_bounds__(kSortBlock)
moe_scan_kernel(int32_t* __restrict__ block_counts, int64_t blocks, int experts,
                int32_t* __restrict__ totals) {
  __shared__ int sum[kSortWaves][64];
  const int lane = threadIdx.x % 64, wave = wave_index(), e = blockIdx.x * 64 + lane;
  const int64_t per = (blocks + kSortWaves - 1) / kSortWaves;
  const int64_t b0 = wave * per < blocks ? wave * per : blocks;
  const int64_t b1 = b0 + per < blocks ? b0 + per : blocks;
  int n = 0;
  if (e < experts)
#pragma unroll 8
    for (int64_t b = b0; b < b1; ++b) n += block_counts[b * experts + e];
  sum[wave][lane] = n;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < wave; ++w) at += sum[w][lane];
  if (e >= experts) return;
  if (wave == kSortWaves - 1) totals[e] = at + n;
  for (int64_t b = b0; b < b1; ++b) {
    const int c = block_counts[b * experts + e];
    block_counts[b * experts + e] = at;
    at += c;
  }
}

// The sort. A pair's row is its expert's start, plus the expert's pairs in earlier workgroups,
// in earlier waves of this workgroup, in earlier steps of this wave, and in lower lanes of its
// step. The last comes from one ballot per bit of the expert index: the lanes that agree in
// every bit are the same expert's. A wave's LDS operations run in order, so a step's counters
// hold the steps before it; nothing depends on the order of the waves.
//
// The pairs of one step go to as many experts, so writing source from there costs a line a
// pair. With more than one step (4000 pairs: 6.9 us) the workgroup's pairs are brought into their
// order in LDS first and written along the rows (6.1 us).
// block_counts: null for a single workgroup; else the counts of the blocks, or with totals
// those of the blocks before each.
template <int S, typename I>
__global__ void __launch_bounds__(kSortBlock)
moe_sort_kernel(const I* __restrict__ idx, int64_t pairs, int experts, int bits, int multiple,
                int64_t rows, const int32_t* __restrict__ block_counts,
                const int32_t* __restrict__ totals, int32_t* __restrict__ slot,
                int32_t* __restrict__ source, int32_t* __restrict__ counts,
                int32_t* __restrict__ offsets) {
  constexpr bool kOrder = S > 1;
  __shared__ int next[kSortWaves * kMoeMaxExperts];        // [waves][experts]
  __shared__ int2 share[kOrder ? 1 : kSortBlock];          // only chunks of one step are added
  __shared__ int2 wave_sum[kSortWaves], pad[kMoeMaxExperts];
  __shared__ int shift[kOrder ? kMoeMaxExperts : 1], end, placed;
  __shared__ uint16_t order_pair[kOrder ? S * kSortBlock : 1];
  __shared__ uint16_t order_expert[kOrder ? S * kSortBlock : 1];
  const int t = threadIdx.x, lane = t % 64, wave = wave_index();
  const int64_t p0 = first_pair<S>();
  int e[S], row[S];
  ld_experts<S>(idx, p0, pairs, experts, e);
  // block counts: lane groups of 2^bits lanes take every `shares`-th block
  const int shares = min(kSortBlock >> bits, kSortShares);
  const int se = t & ((1 << bits) - 1), sg = t >> bits;
  int2 n = {0, 0};                             // all blocks, blocks before this
  if (block_counts && !totals && se < experts && sg < shares) {
#pragma unroll 4
    for (int b = sg; b < (int)gridDim.x; b += shares) {
      const int c = block_counts[(int64_t)b * experts + se];
      n.x += c;
      if (b < (int)blockIdx.x) n.y += c;
    }
  }
  for (int i = t; i < kSortWaves * experts; i += kSortBlock) next[i] = 0;
  if constexpr (!kOrder) share[t] = n;
  __syncthreads();
  // ranks among the wave's own pairs: the lanes of a step that hold the same expert, then the
  // lowest of them adds their number to the wave's counter, steps in order
  uint64_t same[S];
#pragma unroll
  for (int k = 0; k < S; ++k) same[k] = __ballot(e[k] >= 0);
  for (int b = 0; b < bits; ++b) {
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const int bit = (e[k] >> b) & 1;
      const uint64_t m = __ballot(bit);
      same[k] &= bit ? m : ~m;
    }
  }
  int* mine = next + wave * experts;
#pragma unroll
  for (int k = 0; k < S; ++k) {
    row[k] = 0;
    if (e[k] >= 0 && lanes_below(same[k]) == 0)
      row[k] = atomicAdd(&mine[e[k]], __popcll(same[k]));
  }
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const int first = e[k] >= 0 ? __ffsll((unsigned long long)same[k]) - 1 : lane;
    row[k] = __shfl(row[k], first, 64) + lanes_below(same[k]);
  }
  __syncthreads();
  // thread e: expert e's pairs over all workgroups, before this one, and of this one
  int c[kSortWaves], tot = 0, before = 0, own = 0;
  int2 pre = {0, 0};                           // inclusive prefix of the padded and own counts
  int padded = 0;
  if (wave * 64 < experts) {
    if (t < experts) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) {
        c[w] = next[w * experts + t];
        own += c[w];
      }
      if (!block_counts) {
        tot = own;
      } else if (totals) {
        tot = totals[t];
        before = block_counts[(int64_t)blockIdx.x * experts + t];
      } else if constexpr (!kOrder) {
#pragma unroll 8
        for (int g = 0; g < shares; ++g) {
          const int2 k = share[(g << bits) + t];
          tot += k.x;
          before += k.y;
        }
      }
    }
    padded = padded_count(tot, multiple);
    pre = int2{padded, own};
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int x = __shfl_up(pre.x, off, 64), y = kOrder ? __shfl_up(pre.y, off, 64) : 0;
      if (lane >= off) pre.x += x, pre.y += y;
    }
  }
  if (experts > 64) {
    if (lane == 63) wave_sum[wave] = pre;
    __syncthreads();
    if (wave * 64 < experts)
      for (int w = 0; w < wave; ++w) pre.x += wave_sum[w].x, pre.y += wave_sum[w].y;
  }
  if (t < experts) {
    const int start = pre.x - padded, first = start + before;
    int at = kOrder ? pre.y - own : first;
    if constexpr (kOrder) shift[t] = first - at;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      next[w * experts + t] = at;
      at += c[w];
    }
    pad[t] = int2{start + tot, pre.x};
    if (t == experts - 1) {
      end = pre.x;
      placed = pre.y;
    }
    if (blockIdx.x == 0) {
      counts[t] = tot;
      offsets[t + 1] = pre.x;
      if (t == 0) offsets[0] = 0;
    }
  }
  __syncthreads();
  const int64_t block_p0 = (int64_t)blockIdx.x * (kSortBlock * S);
#pragma unroll
  for (int k = 0; k < S; ++k) {
    const int64_t p = p0 + k * 64 + lane;
    if (p >= pairs) break;
    int r = -1;
    if (e[k] >= 0) {
      r = row[k] + next[wave * experts + e[k]];
      if constexpr (kOrder) {
        order_pair[r] = (uint16_t)(p - block_p0);
        order_expert[r] = (uint16_t)e[k];
        r += shift[e[k]];
      } else {
        source[r] = (int32_t)p;
      }
    }
    slot[p] = r;
  }
  // padding rows, 16 lanes an expert, every expert's by one workgroup
  for (int i = t;; i += kSortBlock) {
    const int x = (int)blockIdx.x + (int)gridDim.x * (i / 16);
    if (x >= experts) break;
    each_padding_row(pad[x].x, pad[x].y, i % 16, [&](int r) { source[r] = -1; });
  }
  if constexpr (kOrder) {
    __syncthreads();
    for (int i = t; i < placed; i += kSortBlock)
      source[i + shift[order_expert[i]]] = (int32_t)(block_p0 + order_pair[i]);
  }
  // rows past the last expert's
  for (int64_t r = end + (int64_t)blockIdx.x * kSortBlock + t; r < rows;
       r += (int64_t)gridDim.x * kSortBlock)
    source[r] = -1;
}

// -------------------------------------------------------------------------- exchanges

constexpr int kMoveBlock = 256, kMoveWaves = kMoveBlock / 64;

// Waves of the grid, the same for all lanes (addresses of rows are scalar).
__device__ __forceinline__ uint32_t grid_wave() {
  return blockIdx.x * (uint32_t)kMoveWaves + (uint32_t)wave_index();
}

// A token's choices, one to a lane (topk is at most 64): the row of choice j in lane j, -1 where
// there is none in the buffer. One load for all; a choice's row comes out as a scalar.
static_assert(kMoeMaxTopk <= 64, "a lane holds a choice");
struct Choices {
  int row;
  float weight;
  __device__ __forceinline__ Choices(const int32_t* slot, const float* weights, int64_t token,
                                     int topk, int64_t rows) {
    const int lane = threadIdx.x % 64;
    const int64_t pair = token * topk + lane;
    const int r = lane < topk ? slot[pair] : -1;
    weight = lane < topk && weights ? weights[pair] : 1.f;
    row = r < rows ? r : -1;
  }
  __device__ __forceinline__ int row_of(int j) const {
    return __builtin_amdgcn_readlane(row, j);
  }
  __device__ __forceinline__ float weight_of(int j) const {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
  }
};

// Zeroing the padding rows: a wave checks kRows rows and zeroes those without a pair, PIECES
// 16-byte pieces a lane, one row after the other. More rows a wave are fewer waves that find
// nothing but longer ones that do: dispatch of 300 tokens, 6 of 64, width 512 bf16 3.1 us with 8
// rows a wave and 5.5 us with 64, of 8192 tokens, 8 of 64, width 64 7.4 and 8.3 us.
template <typename T, int PIECES> struct Zero {
  static constexpr int kRows = 8, kCols = 64 * Piece<T>::N * PIECES;
  static int64_t waves(int64_t rows, int64_t cols) {
    return (rows + kRows - 1) / kRows * ((cols + kCols - 1) / kCols);
  }
  static __device__ __forceinline__ void run(uint32_t wave, const int32_t* source, int64_t rows,
                                             int cols, T* out) {
    const uint32_t chunks = (uint32_t)(cols + kCols - 1) / kCols;
    const int lane = threadIdx.x % 64, c0 = (int)(wave % chunks) * kCols;
    const int64_t r0 = (int64_t)(wave / chunks) * kRows, r = r0 + lane;
    uint64_t m = __ballot(lane < kRows && r < rows && source[r] < 0);
    while (m) {
      const int i = __ffsll((unsigned long long)m) - 1;
      m &= m - 1;
#pragma unroll
      for (int v = 0; v < PIECES; ++v)
        st_row<kStream>(out + (r0 + i) * cols, c0 + (v * 64 + lane) * Piece<T>::N, cols,
                        piece_t{0, 0, 0, 0});
    }
  }
};

// One wave per (token, PIECES pieces a lane of the row): loaded once, stored to each of
// the token's rows. The first waves zero the padding rows. Bound by the writes of the
// sorted rows: 8192 tokens to 8 of 64 experts, width 4096 bf16 in 108.6 us, 5.6 TB/s. They
// stream (117.8 us kept, and no size was found where that cost); the tokens' rows are kept, 122
// us with the sort against 136 us streamed.
// The `bytes` first bytes (a multiple of the element, at most 16) of a piece.
template <Cache C, typename T>
__device__ __forceinline__ void st_first(T* p, piece_t v, int bytes) {
  if (bytes >= 16) st_piece<C>(p, v);
  else if (bytes > 0) st_row<C>(p, 0, bytes / (int)sizeof(T), v);
}

// LINES: rows whose width is no whole number of 128-byte lines. A store of a wave then covers
// whole lines of its row, which begin somewhere else in every row, so the token's row is loaded
// (from the cache) for each: 4000 tokens, 7 of 64, width 4097 bf16 with the sort 60.0 us, 71.0
// without (width 4096: 56.2); 1066 tokens, 7 of 91, width 6030 f32 53.7 and 61.9; but 8192 tokens,
// 2 of 8, width 5001 51.9 and 48.4, so from three choices on.
template <typename T, int PIECES, bool LINES>
__global__ void __launch_bounds__(kMoveBlock)
moe_dispatch_kernel(const T* __restrict__ x, int64_t ldx, const int32_t* __restrict__ slot,
                    const int32_t* __restrict__ source, int64_t tokens, int topk, int64_t rows,
                    int cols, uint32_t chunks, uint32_t zeros, T* __restrict__ xs) {
  constexpr int N = Piece<T>::N, kCols = 64 * N * PIECES;
  const int lane = threadIdx.x % 64;
  uint32_t u = grid_wave();
  if (u < zeros) {
    Zero<T, PIECES>::run(u, source, rows, cols, xs);
    return;
  }
  u -= zeros;
  const int64_t t = u / chunks;
  if (t >= tokens) return;
  const int c0 = (int)(u % chunks) * kCols + lane * N;
  const T* src = x + t * ldx;
  const Choices choices(slot, nullptr, t, topk, rows);
  if constexpr (LINES) {
    for (int j = 0; j < topk; ++j) {
      const int r = choices.row_of(j);
      if (r < 0) continue;
      T* dst = xs + (int64_t)r * cols;
      const int before = (int)(((uintptr_t)dst & 127) / sizeof(T));
      piece_t v[PIECES];
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        v[i] = ld_raw<kKeep>(src, max(c0 + i * 64 * N - before, 0), cols);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int c = c0 + i * 64 * N - before, from = max(c, 0);
        st_first<kStream>(elem_at(dst, min(from, cols)), cut<T>(v[i], from, cols),
                          (min(c + N, cols) - from) * (int)sizeof(T));
      }
    }
    return;
  }
  piece_t v[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) v[i] = ld_raw<kKeep>(src, c0 + i * 64 * N, cols);
#pragma unroll
  for (int i = 0; i < PIECES; ++i) v[i] = cut<T>(v[i], c0 + i * 64 * N, cols);
  for (int j = 0; j < topk; ++j) {
    const int r = choices.row_of(j);
    if (r < 0) continue;
    T* dst = xs + (int64_t)r * cols;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) st_row<kStream>(dst, c0 + i * 64 * N, cols, v[i]);
  }
}

// One wave per (token, PIECES pieces a lane of the row): the token's rows, U in flight,
// summed in the order of the choices in float32 and rounded once. Bound by the reads of the
// sorted rows: 8192 tokens, 8 of 64 experts, width 4096 bf16 in 99.5 us, 5.9 TB/s.
template <typename T, int PIECES, int U, Cache C>
__global__ void __launch_bounds__(kMoveBlock)
moe_combine_kernel(const T* __restrict__ ys, int64_t ldys, const int32_t* __restrict__ slot,
                   const float* __restrict__ weights, int64_t tokens, int topk, int64_t rows,
                   int cols, uint32_t chunks, T* __restrict__ y) {
  constexpr int N = Piece<T>::N, kCols = 64 * N * PIECES;
  const int lane = threadIdx.x % 64;
  const uint32_t u = grid_wave();
  const int64_t t = u / chunks;
  if (t >= tokens) return;
  const int c0 = (int)(u % chunks) * kCols + lane * N;
  const Choices choices(slot, weights, t, topk, rows);
  float acc[PIECES][N];
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int n = 0; n < N; ++n) acc[i][n] = 0.f;
  for (int j0 = 0; j0 < topk; j0 += U) {
    piece_t v[U][PIECES];
    int r[U];
#pragma unroll
    for (int q = 0; q < U; ++q) r[q] = j0 + q < topk ? choices.row_of(j0 + q) : -1;
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (r[q] < 0) continue;
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        v[q][i] = ld_raw<C>(ys + r[q] * ldys, c0 + i * 64 * N, cols);
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      if (r[q] < 0) continue;
      const float w = choices.weight_of(j0 + q);
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        float f[N];
        unpack(cut<T>(v[q][i], c0 + i * 64 * N, cols), f, T{});
#pragma unroll
        for (int n = 0; n < N; ++n) acc[i][n] = __builtin_fmaf(w, f[n], acc[i][n]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
    st_row<C>(y + t * cols, c0 + i * 64 * N, cols, pack(acc[i], T{}));
}

// W waves per token read dy[t] once per J choices, write w dy to their rows and sum dy ys of
// each (lanes, then waves, in a fixed order). The first workgroups zero the padding rows. Bound by
// memory: 8192 tokens, 2 of 8, width 4096 bf16 in 58.9 us, 5.7 TB/s.
template <typename T, int W, int J, Cache C>
__global__ void __launch_bounds__(kMoveBlock)
moe_combine_bwd_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ ys,
                       int64_t ldys, const int32_t* __restrict__ slot,
                       const int32_t* __restrict__ source, const float* __restrict__ weights,
                       int64_t tokens, uint32_t zero_blocks, int topk, int64_t rows, int cols,
                       T* __restrict__ dys, float* __restrict__ dw) {
  constexpr int N = Piece<T>::N, PER = kMoveWaves / W;
  __shared__ float part[W][J];
  const int lane = threadIdx.x % 64, wave = wave_index();
  if (blockIdx.x < zero_blocks) {
    Zero<T, W>::run(grid_wave(), source, rows, cols, dys);
    return;
  }
  const int64_t t = (int64_t)(blockIdx.x - zero_blocks) * PER + (W == 1 ? wave : 0);
  if (t >= tokens) return;                       // a whole token's waves
  const int lt = W == 1 ? lane : (int)threadIdx.x;
  const T* g = dy + t * lddy;
  const Choices choices(slot, weights, t, topk, rows);
  for (int j0 = 0; j0 < topk; j0 += J) {
    int r[J];
    float w[J], dot[J];
#pragma unroll
    for (int q = 0; q < J; ++q) {
      r[q] = j0 + q < topk ? choices.row_of(j0 + q) : -1;
      w[q] = r[q] >= 0 ? choices.weight_of(j0 + q) : 0.f;
      dot[q] = 0.f;
    }
    constexpr int STEPS = J <= 4 ? 2 : 1, kStep = W * 64 * N;
    for (int c0 = lt * N; c0 < cols; c0 += STEPS * kStep) {
      piece_t pg[STEPS], py[STEPS][J];
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        pg[k] = ld_raw<C>(g, c0 + k * kStep, cols);
#pragma unroll
        for (int q = 0; q < J; ++q)
          if (r[q] >= 0) py[k][q] = ld_raw<C>(ys + r[q] * ldys, c0 + k * kStep, cols);
      }
#pragma unroll
      for (int k = 0; k < STEPS; ++k) {
        const int c = c0 + k * kStep;
        float fg[N];
        unpack(cut<T>(pg[k], c, cols), fg, T{});
#pragma unroll
        for (int q = 0; q < J; ++q) {
          if (r[q] < 0) continue;
          float fy[N], o[N];
          unpack(cut<T>(py[k][q], c, cols), fy, T{});
#pragma unroll
          for (int n = 0; n < N; ++n) {
            dot[q] = __builtin_fmaf(fg[n], fy[n], dot[q]);
            o[n] = w[q] * fg[n];
          }
          st_row<C>(dys + (int64_t)r[q] * cols, c, cols, pack(o, T{}));
        }
      }
    }
    if constexpr (W == 1) {
#pragma unroll
      for (int q = 0; q < J; ++q) {
        const float d = lanes_sum<64>(dot[q]);
        if (lane == 0 && j0 + q < topk) dw[t * topk + j0 + q] = d;
      }
    } else {
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
        for (int k = 0; k < W; ++k) d += part[k][threadIdx.x];
        dw[t * topk + j0 + threadIdx.x] = d;
      }
    }
  }
}

struct SortPlan { int64_t steps, blocks; bool scan; };
SortPlan sort_plan(int64_t pairs) {
  const int64_t b = (pairs + kSortBlock - 1) / kSortBlock;
  if (b <= 1) return {1, 1, false};
  if (pairs <= kSortOne) return {kSortSteps, 1, false};
  if (b <= kSortDirect) return {1, b, false};
  return {kSortSteps, (pairs + kSortLong - 1) / kSortLong, true};
}

template <int S, typename I>
hipError_t sort_steps(const MoeSortArgs& a, const SortPlan& plan, hipStream_t s) {
  int bits = 0;
  while ((1 << bits) < a.experts) ++bits;
  const I* idx = static_cast<const I*>(a.idx);
  const unsigned blocks = (unsigned)plan.blocks;
  int32_t* block_counts = blocks > 1 ? a.workspace : nullptr;
  int32_t* totals = plan.scan ? a.workspace + plan.blocks * a.experts : nullptr;
  if (block_counts) {
    hipLaunchKernelGGL((moe_count_kernel<S, I>), dim3(blocks), dim3(kSortBlock), 0, s, idx,
                       a.pairs, a.experts, block_counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (totals) {
    hipLaunchKernelGGL(moe_scan_kernel, dim3((unsigned)(a.experts + 63) / 64), dim3(kSortBlock), 0,
                       s, block_counts, plan.blocks, a.experts, totals);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((moe_sort_kernel<S, I>), dim3(blocks), dim3(kSortBlock), 0, s, idx, a.pairs,
                     a.experts, bits, a.multiple, a.rows, block_counts, totals, a.slot, a.source,
                     a.counts, a.offsets);
  return hipGetLastError();
}

template <typename I>
hipError_t sort_launch(const MoeSortArgs& a, hipStream_t s) {
  const SortPlan plan = sort_plan(a.pairs);
  return plan.steps == 1 ? sort_steps<1, I>(a, plan, s) : sort_steps<kSortSteps, I>(a, plan, s);
}

// Chunks of a row of `pieces` pieces a lane.
template <typename T> uint32_t row_chunks(int64_t cols, int pieces) {
  const int per = 64 * Piece<T>::N * pieces;
  return (uint32_t)((cols + per - 1) / per);
}
unsigned move_blocks(int64_t waves) { return (unsigned)((waves + kMoveWaves - 1) / kMoveWaves); }

// Waves that are on the card at once. A launch of no more is bound by a wave's own waits.
constexpr int64_t kResidentWaves = 256 * 32;

template <typename T, int PIECES, bool LINES>
hipError_t dispatch_rows(const MoeArgs& a, hipStream_t s) {
  // a row's lines begin up to a line before it
  const uint32_t chunks = row_chunks<T>(a.cols + (LINES ? 128 / (int)sizeof(T) : 0), PIECES);
  const int64_t zeros = Zero<T, PIECES>::waves(a.rows, a.cols);
  const unsigned blocks = move_blocks(a.tokens * chunks + zeros);
  hipLaunchKernelGGL((moe_dispatch_kernel<T, PIECES, LINES>), dim3(blocks), dim3(kMoveBlock), 0, s,
                     static_cast<const T*>(a.x), a.ldx, a.slot, a.source, a.tokens, a.topk, a.rows,
                     (int)a.cols, chunks, (uint32_t)zeros, static_cast<T*>(a.out));
  return hipGetLastError();
}
// One piece a lane where that fits the row or the card (8192 tokens, 8 of 64, width 64 bf16:
// 7.4 us, with four pieces 10.4 us; one token, width 4096 2.9 and 3.8 us); else four, 2 % faster
// for 8192 tokens of width 4096.
template <typename T>
hipError_t dispatch(const MoeArgs& a, hipStream_t s) {
  const int64_t chunks = row_chunks<T>(a.cols, 1);
  if (chunks <= 1 || a.tokens * chunks <= kResidentWaves) return dispatch_rows<T, 1, false>(a, s);
  const bool lines = a.topk > 2 && a.cols * sizeof(T) % 128 != 0;
  return lines ? dispatch_rows<T, 4, true>(a, s) : dispatch_rows<T, 4, false>(a, s);
}

// Tensors of rows up to 96 MiB together are kept in the caches, larger ones stream. Measured over
// three sets of tensors in turn: the combine of 4096 tokens, 8 of 64, width 1024 bf16 (72 MiB)
// takes 13.6 us kept and 15.1 us streamed, with 2 of 8 and width 4096 (97 MiB) 21.5 and 18.8 us;
// the combine's gradient of 2000 tokens, 2 of 8, width 4096 (78 MiB) 14.9 and 16.9 us, of 4096
// tokens (160 MiB) 35.1 and 31.7 us.
constexpr int64_t kKeepBytes = 96 << 20;
bool keeps(const MoeArgs& a, int64_t rows) {
  return rows * a.cols * (a.dtype == kF32 ? 4 : 2) <= kKeepBytes;
}

template <typename T, int PIECES, int U, Cache C>
hipError_t combine_rows(const MoeArgs& a, hipStream_t s) {
  const uint32_t chunks = row_chunks<T>(a.cols, PIECES);
  hipLaunchKernelGGL((moe_combine_kernel<T, PIECES, U, C>), dim3(move_blocks(a.tokens * chunks)),
                     dim3(kMoveBlock), 0, s, static_cast<const T*>(a.ys), a.ldys, a.slot,
                     a.weights, a.tokens, a.topk, a.rows, (int)a.cols, chunks,
                     static_cast<T*>(a.out));
  return hipGetLastError();
}
// Where the waves do not all fit on the card at once, two pieces of two rows in flight: more
// leave fewer waves on a unit (4096 tokens, 8 of 64, width 1024 f32: two rows 25.1 us, four 30.8
// us, one 25.5 us). Where they do, a wave's own waits count: one piece of eight rows.
template <typename T>
hipError_t combine(const MoeArgs& a, hipStream_t s) {
  if (!keeps(a, a.rows + a.tokens)) return combine_rows<T, 2, 2, kStream>(a, s);
  const bool resident = a.tokens * row_chunks<T>(a.cols, 1) <= kResidentWaves;
  return resident ? combine_rows<T, 1, 8, kKeep>(a, s) : combine_rows<T, 2, 2, kKeep>(a, s);
}

template <typename T, int W, int J, Cache C>
hipError_t combine_bwd_rows(const MoeArgs& a, hipStream_t s) {
  const int64_t per = kMoveWaves / W;
  const uint32_t zero_blocks = move_blocks(Zero<T, W>::waves(a.rows, a.cols));
  const unsigned blocks = zero_blocks + (unsigned)((a.tokens + per - 1) / per);
  hipLaunchKernelGGL((moe_combine_bwd_kernel<T, W, J, C>), dim3(blocks), dim3(kMoveBlock), 0, s,
                     static_cast<const T*>(a.x), a.ldx, static_cast<const T*>(a.ys), a.ldys,
                     a.slot, a.source, a.weights, a.tokens, zero_blocks, a.topk, a.rows,
                     (int)a.cols, static_cast<T*>(a.out), a.dw);
  return hipGetLastError();
}
template <typename T, int W, Cache C>
hipError_t combine_bwd_choices(const MoeArgs& a, hipStream_t s) {
  // choices a walk over the row: 8192 tokens, 8 of 64, width 4096 bf16 226 us with eight, 235 us
  // with two walks of four; two steps of a row in flight only up to four (223 us with eight there,
  // but 1000 tokens of width 2048 17.2 us against 15.1)
  if (a.topk <= 2) return combine_bwd_rows<T, W, 2, C>(a, s);
  return a.topk <= 4 ? combine_bwd_rows<T, W, 4, C>(a, s) : combine_bwd_rows<T, W, 8, C>(a, s);
}
template <typename T, Cache C>
hipError_t combine_bwd_waves(const MoeArgs& a, hipStream_t s) {
  // rows of up to two pieces a lane take one wave: four would leave most lanes idle
  return a.cols <= 2 * 64 * Piece<T>::N ? combine_bwd_choices<T, 1, C>(a, s)
                                        : combine_bwd_choices<T, kMoveWaves, C>(a, s);
}
template <typename T>
hipError_t combine_bwd(const MoeArgs& a, hipStream_t s) {
  return keeps(a, 2 * a.rows + a.tokens) ? combine_bwd_waves<T, kKeep>(a, s)
                                         : combine_bwd_waves<T, kStream>(a, s);
}

}  // namespace

int64_t moe_sort_workspace(int64_t pairs, int32_t experts) {
  const SortPlan plan = sort_plan(pairs);
  if (plan.blocks == 1) return 0;
  return (plan.blocks + (plan.scan ? 1 : 0)) * experts * (int64_t)sizeof(int32_t);
}

hipError_t launch_moe_sort(const MoeSortArgs& a, hipStream_t s) {
  return a.idx_bytes == 8 ? sort_launch<int64_t>(a, s) : sort_launch<int32_t>(a, s);
}

hipError_t launch_moe_dispatch(const MoeArgs& a, hipStream_t s) {
  // only moved, so 2-byte elements of either type are the same
  return a.dtype == kF32 ? dispatch<float>(a, s) : dispatch<BF16>(a, s);
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
