// Products of the experts' rows with block scales, all experts in one launch.
//
//   forward, input gradient   y[r, n] = sum_kb sx[r, kb] sw[e, n / 128, kb] S_kb[r, n],
//                             S_kb the sum over the 128 codes of K block kb, e the expert of row r
//   weight gradient           dw[e][n, k] = sum_b sg[n, b] sx[k, b] S_b[n, k], S_b the sum over
//                             the 128 rows of row block b, b over the expert's blocks
//
// Rows come sorted by expert: expert e's are offsets[e] .. offsets[e] + counts[e], on the device.
// Both are clamped to the tensors, so that no value of theirs leads outside of them.
//
// A v_mfma_f32_16x16x128_f8f6f4 started from zero is one block's partial sum S, folded into the
// float32 accumulators with its scales.
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "mfma_tile.h"

namespace fp8lin {

namespace {

constexpr int kBlock = 128;                  // codes per scale
constexpr int kCus = 256;                    // compute units

// The rows of expert e: first, one past the last, one past its padding.
struct Span { int64_t first, end, next; };
__device__ __forceinline__ Span expert_span(const int32_t* offsets, const int32_t* counts, int e,
                                            int64_t rows) {
  const int64_t a = min(max((int64_t)offsets[e], (int64_t)0), rows);
  const int64_t b = min(max((int64_t)offsets[e + 1], a), rows);
  return {a, min(a + max((int64_t)counts[e], (int64_t)0), b), b};
}

__device__ __forceinline__ v4f mfma(v8i b, v8i a) {
  const v4f z = {};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, z, 0, 0, 0, 0, 0, 0);
}

// The spans of rows: 0 before the first expert, 1 .. experts the experts, experts + 1 after the last.
__device__ __forceinline__ Span span_of(const GroupedArgs& a, int i) {
  if (i == 0) return {0, 0, expert_span(a.offsets, a.counts, 0, a.rows).first};
  if (i <= a.experts) return expert_span(a.offsets, a.counts, i - 1, a.rows);
  const int64_t b = expert_span(a.offsets, a.counts, a.experts - 1, a.rows).next;
  return {b, b, a.rows};
}
constexpr int kMaxSpans = kMoeMaxExperts + 2;

// ---------------------------------------------------------------------------
// Streams: small pieces of the output, each by the 4 waves of a workgroup, for what the tiles below
// do not fill the card with: an expert's few rows, where the time is that of reading the weights
// once, and outputs of few tiles. An item is 32 rows of the first operand (columns of y; n) by XR of
// the second (rows of y; in the weight gradient k). A wave takes a quarter of the item's K blocks
// and streams them through a ring of D slots of its own in LDS, loaded straight from memory, so that
// neither registers nor barriers limit what is under way, and goes on with the next item's blocks
// while the waves' sums are added up through LDS. What bounds it: the weights from memory for few
// rows (two experts' 14336 x 4096 for a token, 117 MB, 25.4 us: 4.6 TB/s; loaded to registers 29 us
// with 2 blocks ahead, 39 with 4: a line arrives in two halves, which the L1 cannot hold for long
// enough); else the way from L2 (64 rows of 128 codes for 32 x 32 sums, near 12 TB/s).
//
// XR 8, D 2, two workgroups a CU: up to 8 rows an expert. A slot holds 8 rows of x; lanes of rows
// past them multiply another row's codes, for nobody. XR 32, D 1, three workgroups a CU: the rest
// (also for a token it reads the weights of 4096 x 14336 in 32.8 us to 27.5). One block under way a
// wave is enough there (12 waves a CU, 8.4 KB each): with two and one workgroup a CU 17.6 us instead
// of 16.4 at 1024 x 4096 with 75 rows an expert, 20.3 instead of 14.5 at 1024 x 1024 with 250; with
// 16 rows an item 42.9 instead of 35.1 at 1024 x 4096 with 250 rows.
constexpr int kStreamWaves = 4, kStreamThreads = 64 * kStreamWaves;

template <int BROWS, int XR, int D>
__global__ void __launch_bounds__(kStreamThreads)
grouped_stream_kernel(GroupedArgs a) {
  constexpr bool kGrad = BROWS == 1;                     // weight gradient
  constexpr int MT = (XR + 15) / 16, NT = 2;             // 16x16 tiles
  constexpr int kRows = XR, kCols = 16 * NT;
  constexpr int kW = kCols * kBlock, kX = kRows * kBlock, kSc = 256;
  constexpr int kSlot = kW + kX + (kGrad ? 2 : 1) * kSc;
  constexpr int kInstW = kCols / 8, kInstX = kRows / 8;
  constexpr int kPer = kInstW + kInstX + (kGrad ? 2 : 1);      // loads of a block
  constexpr int kPitch = kCols + 1;
  static_assert(kRows <= 64 && kCols <= 64 && (XR == 8 || XR % 16 == 0), "a lane a row's scale");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kStreamWaves * D * kSlot];
  __shared__ float sums[kStreamWaves][kRows * kPitch];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r16 = lane & 15, g4 = lane >> 4;
  const int col_blocks = (int)(a.N / kCols);
  const int row_blocks = kGrad ? (int)(a.K / kRows) : 0;      // of an expert's gradient
  const int kblocks = (int)((kGrad ? a.rows : a.K) / kBlock); // of an operand's row
  const uint32_t ldx = (uint32_t)(kGrad ? a.rows : a.K);      // bytes
  const uint32_t ldw = (uint32_t)(kGrad ? a.rows : a.ldw);
  uint8_t* const ring = smem + wave * D * kSlot;
  const int spans = kGrad ? a.experts : a.experts + 2;

  // The items in the order of spans, rows, columns; this workgroup's are every gridDim.x-th. A lane
  // holds one of 64 spans at a time.
  struct Item { int span, first, end, m0, n0; };         // span -1: no more
  struct Cursor {
    int base;                                            // spans base .. base + 63 are held
    Span l;
    int items, upto;                                     // of the lane's span, and with those before
    int at;                                              // ours within the 64 spans' items
  };
  auto spans_from = [&](Cursor& c, int base) __attribute__((always_inline)) {
    c.base = base;
    c.l = {0, 0, 0};
    const bool in = base + lane < spans;
    if (in) c.l = kGrad ? expert_span(a.offsets, a.counts, base + lane, a.rows)
                        : span_of(a, base + lane);
    c.items = (kGrad ? (in ? row_blocks : 0) : (int)(c.l.end - c.l.first + kRows - 1) / kRows) *
              col_blocks;
    c.upto = c.items;
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
      const int o = __shfl_up(c.upto, off, 64);
      if (lane >= off) c.upto += o;
    }
  };
  auto next_item = [&](Cursor& c) __attribute__((always_inline)) -> Item {
    uint64_t later = __ballot(c.upto > c.at);
    while (later == 0) {
      if (c.base + 64 >= spans) return {-1, 0, 0, 0, 0};
      c.at -= __builtin_amdgcn_readlane(c.upto, 63);
      spans_from(c, c.base + 64);
      later = __ballot(c.upto > c.at);
    }
    const int from = __builtin_ctzll(later);
    const int first = __builtin_amdgcn_readlane((int)c.l.first, from);
    const int end = __builtin_amdgcn_readlane((int)c.l.end, from);
    const int in = c.at - __builtin_amdgcn_readlane(c.upto - c.items, from);
    c.at += (int)gridDim.x;
    const int m = in / col_blocks * kRows;
    return {c.base + from, first, end, kGrad ? m : first + m, in % col_blocks * kCols};
  };
  // an item's K blocks, and this wave's of them
  struct Blocks { int first, all, from, n; };
  auto blocks_of = [&](const Item& w) __attribute__((always_inline)) -> Blocks {
    Blocks b = {0, kblocks, 0, 0};
    if constexpr (kGrad) {
      b.first = w.first / kBlock;
      b.all = w.end > w.first ? (w.end + kBlock - 1) / kBlock - b.first : 0;
    }
    b.from = b.all * wave / kStreamWaves;
    b.n = b.all * (wave + 1) / kStreamWaves - b.from;
    return b;
  };

  const int lrow = lane >> 3;                            // 8 rows of 128 bytes an instruction
  auto chunk = [&](int row) { return 16u * ((lane & 7) ^ row_swizzle(row & 15)); };
  v4i rsW, rsX, rsS, rsT;                                // of the item that is loaded
  int pb = 0, pn = 0;                                    // its next block of this wave's, and the end
  Cursor pc, cc;                                         // the loading and the adding side's
  auto seek = [&]() __attribute__((always_inline)) {     // the next item with blocks for this wave
    Item w = next_item(pc);
    Blocks b = blocks_of(w);
    if constexpr (kGrad)
      while (w.span >= 0 && b.n == 0) {
        w = next_item(pc);
        b = blocks_of(w);
      }
    const bool none = w.span < 0;                        // empty resources
    pb = b.from, pn = none ? 0x7FFFFFFF : b.from + b.n;
    if constexpr (kGrad) {
      const uint32_t in_row = (uint32_t)b.all * kBlock;
      const int64_t k0 = (int64_t)b.first * kBlock;
      rsW = make_rsrc(a.w + w.n0 * a.rows + k0, none ? 0u : (uint32_t)(kCols - 1) * ldw + in_row);
      rsX = make_rsrc(a.x + w.m0 * a.rows + k0, none ? 0u : (uint32_t)(kRows - 1) * ldx + in_row);
      rsT = make_rsrc(a.sw + (int64_t)w.n0 * kblocks + b.first,
                      none ? 0u : (uint32_t)((kCols - 1) * kblocks + b.all) * 4u);
      rsS = make_rsrc(a.sx + (int64_t)w.m0 * kblocks + b.first,
                      none ? 0u : (uint32_t)((kRows - 1) * kblocks + b.all) * 4u);
    } else {
      const uint32_t live = (uint32_t)min(w.end - w.m0, kRows);
      const int e = none ? 0 : w.span - 1;
      rsW = make_rsrc(a.w + e * a.stride_w + w.n0 * a.ldw,
                      none ? 0u : (uint32_t)(kCols - 1) * ldw + (uint32_t)a.K);
      rsX = make_rsrc(a.x + (int64_t)w.m0 * a.K, none ? 0u : live * ldx);
      rsS = make_rsrc(a.sx + (int64_t)w.m0 * kblocks, none ? 0u : live * (uint32_t)kblocks * 4u);
    }
  };
  auto load = [&](uint32_t lds) __attribute__((always_inline)) {
    const uint32_t k0 = (uint32_t)pb * kBlock;
#pragma unroll
    for (int q = 0; q < kInstW; ++q) {
      const int row = 8 * q + lrow;
      dma16_so(rsW, (uint32_t)row * ldw + chunk(row), k0, lds + 1024u * q);
    }
#pragma unroll
    for (int q = 0; q < kInstX; ++q) {
      const int row = 8 * q + lrow;
      dma16_so(rsX, (uint32_t)row * ldx + chunk(row), k0, lds + kW + 1024u * q);
    }
    // a lane a row: lanes past the tile's rows read what nobody uses
    const uint32_t at = ((uint32_t)lane * (uint32_t)kblocks + (uint32_t)pb) * 4u;
    dma4(rsS, at, lds + kW + kX);
    if constexpr (kGrad) dma4(rsT, at, lds + kW + kX + kSc);
    if (++pb >= pn) seek();
  };

  const int xrow = XR < 16 ? r16 % XR : r16;
  auto frag = [&](uint32_t at, int row) __attribute__((always_inline)) {   // a lane's 32 codes
    const int sw = row_swizzle(row);
    const v4u lo = lds16(at + (uint32_t)row * kBlock + 16 * ((2 * g4) ^ sw));
    const v4u hi = lds16(at + (uint32_t)row * kBlock + 16 * ((2 * g4 + 1) ^ sw));
    return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  auto ldf = [&](uint32_t at) __attribute__((always_inline)) {
    return *(const __attribute__((address_space(3))) float*)(uintptr_t)at;
  };

  spans_from(pc, 0);
  pc.at = (int)blockIdx.x;
  cc = pc;
  seek();
  for (int d = 0; d < D; ++d) load(lds_addr(ring + d * kSlot));
  uint32_t slot = 0;
  for (Item w = next_item(cc); w.span >= 0; w = next_item(cc)) {
    const Blocks bl = blocks_of(w);
    // as constants, so that scalar loads fetch them, which do not count among the blocks' loads
    const auto* const wscale = (const __attribute__((address_space(4))) float*)(uintptr_t)(
        a.sw + (int64_t)(w.span - 1) * a.stride_sw + w.n0 / kBlock * a.ldsw + bl.from);
    v4f acc[MT][NT] = {};
    for (int b = 0; b < bl.n; ++b) {
      const float g = kGrad ? 1.f : wscale[b];
      wait_vm<(D - 1) * kPer>();
      const uint32_t at = lds_addr(ring) + slot * kSlot, sat = at + kW + kX;
      v8i W[NT], X[MT];
      float f[MT], h[kGrad ? 4 * NT : 1];
#pragma unroll
      for (int j = 0; j < NT; ++j) W[j] = frag(at + 16 * j * kBlock, r16);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        X[i] = frag(at + kW + 16 * i * kBlock, xrow);
        f[i] = ldf(sat + 64 * i + 4 * xrow) * g;
      }
      if constexpr (kGrad)
#pragma unroll
        for (int j = 0; j < 4 * NT; ++j)
          h[j] = ldf(sat + kSc + 64 * (j / 4) + 16 * g4 + 4 * (j % 4));
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot has been read
      load(at);
      slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const v4f p = mfma(W[j], X[i]);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][j][r] = fmaf(p[r], kGrad ? f[i] * h[4 * j + r] : f[i], acc[i][j][r]);
        }
    }
    if (XR % 16 == 0 || r16 < XR) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            sums[wave][(16 * i + r16) * kPitch + 16 * j + 4 * g4 + r] = acc[i][j][r];
    }
    // barriers of LDS only: the next item's loads stay under way
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const int live = kGrad ? kRows : min(w.end - w.m0, kRows);
    for (int q = 2 * t; q < live * kCols; q += 2 * kStreamThreads) {
      // two neighbours of a row of the output
      const int m = kGrad ? q % kRows : q / kCols, n = kGrad ? q / kRows : q % kCols;
      constexpr int kNext = kGrad ? kPitch : 1;
      float lo = 0.f, hi = 0.f;
#pragma unroll
      for (int v = 0; v < kStreamWaves; ++v)
        lo += sums[v][m * kPitch + n], hi += sums[v][m * kPitch + n + kNext];
      uint16_t* const y = kGrad ? a.y + ((int64_t)w.span * a.N + w.n0 + n) * a.K + w.m0 + m
                                : a.y + (int64_t)(w.m0 + m) * a.N + w.n0 + n;
      *reinterpret_cast<uint32_t*>(y) = pack_bf16x2(lo, hi);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
  // rows of nobody: the waves share the spans that have some
  if constexpr (!kGrad) {
    const int me = (int)blockIdx.x * kStreamWaves + wave, waves = (int)gridDim.x * kStreamWaves;
    for (int base = 0; base < spans; base += 64) {
      Cursor z;
      spans_from(z, base);
      const bool has = z.l.next > z.l.end;
      const uint64_t m = __ballot(has);
      const int with = __builtin_popcountll(m), step = min(with, waves);
      const int rank = __builtin_popcountll(m & ((1ull << lane) - 1));
      if (with == 0) continue;
      const int64_t sharers = (waves - me % step + step - 1) / step;
      for (int i = me % step; i < with; i += step) {
        const int from = __builtin_ctzll(__ballot(has && rank == i));
        const int end = __builtin_amdgcn_readlane((int)z.l.end, from);
        const int next = __builtin_amdgcn_readlane((int)z.l.next, from);
        uint4* const y = reinterpret_cast<uint4*>(a.y + (int64_t)end * a.N);
        const int64_t pieces = (int64_t)(next - end) * (a.N / 8);
        for (int64_t q = me / step * 64 + lane; q < pieces; q += sharers * 64)
          y[q] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // no load may land after exit
}

// Pieces of bm rows that the output's rows come in, with an expert's last one about half full. In y,
// rows that are a multiple of 128 are taken to have room for every expert's padding to that, which
// nobody multiplies; `max_rows` may say that there are less.
template <int BROWS>
int64_t row_pieces(const GroupedArgs& a, int64_t bm) {
  if (BROWS == 1) return a.experts * ((a.N + bm - 1) / bm);
  const int64_t live = a.rows % 128 ? a.rows : max(a.rows - 127 * (int64_t)a.experts, a.rows / 128);
  return min(live / bm + (a.experts + 1) / 2, a.experts * ((a.max_rows + bm - 1) / bm));
}

template <int BROWS, int XR, int D>
hipError_t launch_stream(const GroupedArgs& a, hipStream_t s) {
  constexpr int64_t kWgs = XR == 8 ? 2 * kCus : 3 * kCus;
  const int64_t items = a.N / 32 * (BROWS == 1 ? a.experts * (a.K / XR) : (a.rows + XR - 1) / XR);
  hipLaunchKernelGGL((grouped_stream_kernel<BROWS, XR, D>), dim3((unsigned)min(items, kWgs)),
                     dim3(kStreamThreads), 0, s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Tiles of the output by 8 waves, two per SIMD, each of RT x 4 16x16 tiles: 256 x 256 (RT = 8), or
// 128 x 256 (RT = 4) with a third slot; or 128 x 128 by 4 waves, two workgroups a CU, for weight
// gradients, whose scales leave no room for that slot (8 experts of 1024 x 1024 over 60000 rows 125
// us to 141 with 128 x 256; of 27 experts of 6272 x 128 16.1 to 20.3). A K stage is 128 codes per
// MFMA in one of kSlots LDS slots. Within a stage, fragments, folds and loads go as in
// gemm_fp8_mx16bw_kernel: a wave holds the stage's 4 B fragments and streams its A rows through a
// ring of 4, two ahead; the barrier comes RT - 2 rows into the stage, once all of its A rows are
// read, publishes stage s + 1 and frees the stage's slot for stage s + kSlots.
//
// What differs is where the work comes from. A workgroup walks its tiles (listed in LDS, some at a
// time) as one stream of stages: the loads run kSlots stages ahead of the multiplying side, of
// whichever tile they belong to, each with its own buffer resources, so that experts may lie anywhere
// in 64 bits and a row past the expert's end reads zeros. A tile has any number of stages; fewer than
// kSlots are filled up with stages of zeros. A row's scales of 4 stages come in one 16-byte load a
// lane into one of kSlots LDS regions when a tile reaches stage 4 i; where less than 4 are left the
// load takes in what follows in memory, or zeros past the tensor's end (the range check goes by
// dwords), and nobody reads that.
//
// BROWS 128: rows of experts times their weights (one B scale per 128 columns). Rows of no expert
// are tiles without stages, whose outputs are 0. BROWS 1: weight gradients (a B scale per column).
//
// What bounds it: the matrix cores, as in the dense kernel; the in-order wait of a tile's first
// stages for the last tile's stores costs a further 9 to 12 % (y of 16384 rows of 8 experts, 14336 x
// 4096: 913 us, 2107 TFLOP/s, 856 in a copy without the stores; dw 1141, 1036 without).
constexpr int kStageK = 128;

template <int BROWS, int RT, int kSlots, int kTileWaves>
__global__ void __launch_bounds__(64 * kTileWaves, 8 / kTileWaves)
grouped_tile_kernel(GroupedArgs a) {
  constexpr int kTileThreads = 64 * kTileWaves, kTileWgs = kCus * 8 / kTileWaves;
  constexpr int WN = kTileWaves / 2, CT = 4, WTN = 16 * CT, WTM = 16 * RT, BM = 2 * WTM;
  constexpr int BN = WTN * WN;
  constexpr int kRing = 4;
  constexpr int SB = (BM + BN) * kStageK;               // bytes of a slot
  // scales: 16 bytes for each of BM rows and then BN columns, or blocks of them
  constexpr int kScaleLanes = (BM + BN / BROWS + 63) / 64 * 64, kRegion = 16 * kScaleLanes;
  constexpr int kRowsPerInst = 1024 / kStageK;          // 8
  constexpr int kInstA = BM / (kRowsPerInst * kTileWaves), kInstB = BN / (kRowsPerInst * kTileWaves);
  constexpr int kDma = kInstA + kInstB;
  constexpr int kStores = RT * CT / 2;                  // of a wave's epilogue
  constexpr int kMf = RT * CT, kBarrierAt = (RT - 2) * CT, kTail = kMf - kBarrierAt;
  constexpr int L = 2;                                  // fold lag (MFMAs)
  constexpr int kGroup = 4, kGroupM = 8;
  constexpr bool PF = BROWS == 128;                     // scales read a stage ahead
  static_assert(RT % kRing == 0 && kDma <= kTail, "tile");
  constexpr int kYoung = (kSlots - 2) * (kDma + 1);     // loads younger than the next stage's
  constexpr int kBatch = kSlots == 3 || kTileWaves == 4 ? 32 : 128;        // tiles of a workgroup's list
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kSlots * SB +
                                                            (kSlots + 1) * kRegion];
  __shared__ int first_tile[BROWS == 128 ? kMaxSpans + 1 : 1];   // spans: row tiles before it
  uint8_t* const regions = smem + kSlots * SB;          // kSlots, and one of zeros

  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int cols = BROWS == 128 ? (int)a.N : (int)a.K;  // of the output
  const int tiles_n = (cols + BN - 1) / BN;
  const int kblocks = (int)(BROWS == 128 ? a.K : a.rows) / kStageK;   // of an operand's row
  const uint32_t lda = (uint32_t)(BROWS == 128 ? a.K : a.rows);       // bytes
  const uint32_t ldb = (uint32_t)(BROWS == 128 ? a.ldw : a.rows);
  const uint32_t ldsb = (uint32_t)(BROWS == 128 ? a.ldsw : kblocks);  // elements
  const int64_t ldd = cols;

  // the spans of rows: before the first expert, the experts, after the last
  const int spans = BROWS == 128 ? a.experts + 2 : a.experts;
  auto span = [&](int i) -> Span {
    return BROWS == 128 ? span_of(a, i) : expert_span(a.offsets, a.counts, i, a.rows);
  };
  const int tiles_m = BROWS == 128 ? 0 : ((int)a.N + BM - 1) / BM;    // of an expert's gradient
  for (int i = t; i < kRegion / 16; i += kTileThreads)
    reinterpret_cast<uint4*>(regions + kSlots * kRegion)[i] = make_uint4(0, 0, 0, 0);
  if constexpr (BROWS == 128) {
    for (int i = t; i < spans; i += kTileThreads) {
      const Span s = span(i);
      first_tile[i + 1] = (int)((s.next - s.first + BM - 1) / BM);
    }
    if (t == 0) first_tile[0] = 0;
    __syncthreads();
    if (wave == 0) {                           // running sums, 64 spans at a time
      int base = 0;
      for (int i0 = 0; i0 < spans; i0 += 64) {
        int v = i0 + lane < spans ? first_tile[i0 + lane + 1] : 0;
#pragma unroll
        for (int off = 1; off < 64; off *= 2) {
          const int o = __shfl_up(v, off, 64);
          if (lane >= off) v += o;
        }
        if (i0 + lane < spans) first_tile[i0 + lane + 1] = base + v;
        base += __shfl(v, 63, 64);
      }
    }
    __syncthreads();
  }
  const int row_tiles = BROWS == 128 ? __builtin_amdgcn_readfirstlane(first_tile[spans])
                                     : spans * tiles_m;
  const int total = row_tiles * tiles_n;
  // Workgroups are dispatched round-robin over the 8 XCDs: 32 consecutive tiles at a time go to
  // one XCD, whose L2 then serves the rows and columns that they share.
  const int wg = (int)(blockIdx.x & 7) * (kTileWgs / 8) + (int)(blockIdx.x >> 3);
  const int count = wg < total ? (total - wg + kTileWgs - 1) / kTileWgs : 0;

  // The workgroup's tiles, up to kBatch at a time, worked out by a lane each: the divisions and
  // 64-bit sums of it would not fit beside the accumulators.
  struct Tile {
    int nk, m0, n0, e;                         // stages, first row and column, expert
    int rows, live, ncols, kb0;                // rows of the output, those with products, columns,
  };                                           // first K block
  __shared__ __attribute__((aligned(16))) Tile list[kBatch];
  auto make_tile = [&](int ti) __attribute__((always_inline)) {
    const int id = ti * kTileWgs + wg;
    Tile w;
    int i, local, mt;
    if constexpr (BROWS == 128) {
      const int rt = id / tiles_n;
      int lo = 0, hi = spans;                  // the last span that begins at or before rt
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (first_tile[mid] <= rt) lo = mid;
        else hi = mid;
      }
      i = lo;
      mt = first_tile[i + 1] - first_tile[i];
      local = id - first_tile[i] * tiles_n;
    } else {
      i = id / (tiles_m * tiles_n);
      mt = tiles_m;
      local = id - i * tiles_m * tiles_n;
    }
    const int group = local / (kGroupM * tiles_n), first = group * kGroupM;
    const int gs = min(mt - first, kGroupM), in = local - first * tiles_n;
    const int m = (first + in % gs) * BM;
    w.n0 = in / gs * BN;
    w.ncols = min(cols - w.n0, BN);
    const Span s = span(i);
    if constexpr (BROWS == 128) {
      w.e = i - 1;
      w.m0 = (int)s.first + m;
      w.rows = (int)min(s.next - w.m0, (int64_t)BM);
      w.live = (int)max(min(s.end - w.m0, (int64_t)BM), (int64_t)0);
      w.kb0 = 0;
      w.nk = w.live > 0 ? kblocks : 0;
    } else {
      w.e = i;
      w.m0 = m;
      w.rows = w.live = min((int)a.N - m, BM);
      w.kb0 = (int)(s.first / kBlock);
      w.nk = s.end > s.first ? (int)((s.end + kBlock - 1) / kBlock) - w.kb0 : 0;
      if (w.nk == 0) w.live = 0;
    }
    list[ti % kBatch] = w;
  };
  auto tile_of = [&](int ti) __attribute__((always_inline)) -> Tile {         // in scalar registers
    const v4i* q = reinterpret_cast<const v4i*>(&list[ti % kBatch]);
    const v4i lo = q[0], hi = q[1];
    auto u = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
    return {u(lo[0]), u(lo[1]), u(lo[2]), u(lo[3]), u(hi[0]), u(hi[1]), u(hi[2]), u(hi[3])};
  };

  // ---- the loading side
  int batch_end = 0;
  const int lrow = kRowsPerInst * wave + (lane >> 3);
  const int lchunk = (lane & 7) ^ row_swizzle(lrow);
  const uint32_t lane_a = (uint32_t)lrow * lda + 16u * lchunk;
  const uint32_t lane_b = (uint32_t)lrow * ldb + 16u * lchunk;
  const uint32_t inst_a = (uint32_t)(kRowsPerInst * kTileWaves) * lda;
  const uint32_t inst_b = (uint32_t)(kRowsPerInst * kTileWaves) * ldb;
  // lane p of the workgroup loads the scales of tile row p < BM, lane BM + c those of column (or
  // block of columns) c; waves past them load nothing, which writes zeros, to the region of zeros
  const int p = 64 * wave + lane;
  const bool sc_from_a = 64 * wave < BM;
  uint32_t sc_lane = kOutOfRange;              // others are below 2^27
  if (p < BM) sc_lane = (uint32_t)p * (uint32_t)kblocks * 4u;
  else if (p < BM + BN / BROWS) sc_lane = (uint32_t)(p - BM) * ldsb * 4u;
  struct Res { const void *a, *b, *s; uint32_t na, nb, ns; int nk; };  // bases, bytes, stages
  auto res_of = [&](int ti) __attribute__((always_inline)) -> Res {
    if (ti >= batch_end) return {a.x, a.x, a.x, 0, 0, 0, 0};          // nothing: reads zeros
    const Tile w = tile_of(ti);
    const uint32_t in_row = (uint32_t)w.nk * kStageK;
    Res r;
    r.nk = w.nk;
    r.na = (uint32_t)(w.live - 1) * lda + in_row;
    r.nb = (uint32_t)(w.ncols - 1) * ldb + in_row;
    if constexpr (BROWS == 128) {
      r.a = a.x + (int64_t)w.m0 * a.K;
      r.b = a.w + w.e * a.stride_w + (int64_t)w.n0 * a.ldw;
    } else {
      r.a = a.w + (int64_t)w.m0 * a.rows + (int64_t)w.kb0 * kStageK;
      r.b = a.x + (int64_t)w.n0 * a.rows + (int64_t)w.kb0 * kStageK;
    }
    if (sc_from_a) {
      r.s = BROWS == 128 ? a.sx + (int64_t)w.m0 * kblocks
                         : a.sw + (int64_t)w.m0 * kblocks + w.kb0;
      r.ns = ((uint32_t)(w.live - 1) * (uint32_t)kblocks + (uint32_t)w.nk) * 4u;
    } else {
      r.s = BROWS == 128 ? a.sw + w.e * a.stride_sw + w.n0 / kBlock * a.ldsw
                         : a.sx + (int64_t)w.n0 * kblocks + w.kb0;
      r.ns = ((uint32_t)(w.ncols / BROWS - 1) * ldsb + (uint32_t)w.nk) * 4u;
    }
    return r;
  };
  auto dma = [&](int d, uint8_t* slot, const Res& r, int kb) __attribute__((always_inline)) {
    const uint32_t k0 = (uint32_t)kb * kStageK, lds = lds_addr(slot) + 1024u * wave;
    // added up here, so that no register holds each sum; a stage past the last block reads zeros
    uint32_t at = kb < r.nk ? (d < kInstA ? lane_a : lane_b) : kOutOfRange;
    asm volatile("" : "+v"(at));
    if (d < kInstA)
      dma16_so(make_rsrc(r.a, r.na), at + d * inst_a, k0, lds + 1024u * kTileWaves * d);
    else
      dma16_so(make_rsrc(r.b, r.nb), at + (d - kInstA) * inst_b, k0,
               lds + BM * kStageK + 1024u * kTileWaves * (d - kInstA));
  };
  // the scales of K blocks kb .. kb + 3 into region rg (zeros if not `on`)
  auto dma_scales = [&](int rg, const Res& r, int kb, bool on) __attribute__((always_inline)) {
    const uint32_t off = on ? 4u * kb : kOutOfRange / 2;
    const uint32_t at = 64 * wave < kScaleLanes ? (uint32_t)(rg * kRegion) + 1024u * wave
                                                : (uint32_t)(kSlots * kRegion);
    dma16(make_rsrc(r.s, r.ns), sc_lane + off, lds_addr(regions) + at);
  };

  // ---- the multiplying side
  const int r16 = lane & 15, g4 = lane >> 4;
  const int sw = row_swizzle(r16);
  const uint32_t fa0 = (uint32_t)(wm * WTM + r16) * kStageK + 16 * ((2 * g4) ^ sw);
  const uint32_t fa1 = (uint32_t)(wm * WTM + r16) * kStageK + 16 * ((2 * g4 + 1) ^ sw);
  const uint32_t fb0 = fa0 + (uint32_t)(BM + wn * WTN - wm * WTM) * kStageK;
  const uint32_t fb1 = fa1 + (uint32_t)(BM + wn * WTN - wm * WTM) * kStageK;
  auto rd = [&](uint32_t lo_at, uint32_t hi_at) __attribute__((always_inline)) {
    const v4u lo = lds16(lo_at);
    const v4u hi = lds16(hi_at);
    return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  struct Bases { uint32_t a0, a1, b0, b1; };
  auto bases = [&](const uint8_t* sm) __attribute__((always_inline)) {
    uint32_t b = lds_addr(sm);
    asm volatile("" : "+s"(b));
    Bases q{b + fa0, b + fa1, b + fb0, b + fb1};
    asm volatile("" : "+v"(q.a0), "+v"(q.a1), "+v"(q.b0), "+v"(q.b1));
    return q;
  };
  auto rdA = [&](const Bases& q, int i) __attribute__((always_inline)) {
    return rd(q.a0 + 16u * i * kStageK, q.a1 + 16u * i * kStageK);
  };
  auto rdB = [&](const Bases& q, int j) __attribute__((always_inline)) {
    return rd(q.b0 + 16u * j * kStageK, q.b1 + 16u * j * kStageK);
  };
  const int pa_lane = wm * WTM + r16;
  const int pb_lane = BROWS == 1 ? BM + wn * WTN + 4 * g4 : BM + wn * WTN / 128;
  typedef const __attribute__((address_space(3))) float lds_f32;
  float fa[RT], fn[PF ? RT : 1], fb[BROWS == 1 ? 4 * CT : 1];
  // the scales of a tile's stage s in region rg: of the lane's rows, times the wave's B scale where
  // there is one, else also of its columns; zeros past the last block
  auto rd_scales = [&](float* fs, int rg, int s, int nk) __attribute__((always_inline)) {
    const uint32_t r = lds_addr(regions) + (uint32_t)((s < nk ? rg : kSlots) * kRegion) +
                       4u * (s % kGroup);
    uint32_t ba = r + 16u * pa_lane, bb = r + 16u * pb_lane;
    asm volatile("" : "+v"(ba), "+v"(bb));
#pragma unroll
    for (int i = 0; i < RT; ++i) fs[i] = *(lds_f32*)(uintptr_t)(ba + 256u * i);
    if constexpr (BROWS == 1) {
#pragma unroll
      for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) fb[4 * j + x] = *(lds_f32*)(uintptr_t)(bb + 256u * j + 16u * x);
    } else {
      const float f = *(lds_f32*)(uintptr_t)bb;
#pragma unroll
      for (int i = 0; i < RT; ++i) fs[i] *= f;
    }
  };

  v4f acc[RT][CT];
  v8i Bq[CT], Aq[kRing];
  auto fold = [&](auto FIRST_, int x, const v4f& P) __attribute__((always_inline)) {
    const int i = x / CT, j = x % CT;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float f = BROWS == 1 ? fa[i] * fb[4 * j + r] : fa[i];
      acc[i][j][r] = decltype(FIRST_)::value ? P[r] * f : fmaf(P[r], f, acc[i][j][r]);
    }
  };
  Res cur, nxt;             // of this tile and of the next with products
  int rg = 0;               // region of this stage's scales; a group of up to 4 stages takes the next
  auto after = [&](int r) { return r + 1 == kSlots ? 0 : r + 1; };
  uint8_t *mine = smem, *other = smem, *third = smem;    // the slots of this stage and the next two
  auto turn = [&]() __attribute__((always_inline)) {
    uint8_t* const m = mine;
    mine = other, other = kSlots == 3 ? third : m, third = m;
  };
  // Stage s of a tile's `ns`, from slot `mine`; `other` holds the next one. STORED (s < kSlots - 1):
  // the last tile's outputs were stored since the next stage's loads were issued, and may stay under
  // way. There is no branch in it: folds that the compiler moves past one keep all products in
  // registers.
  auto stage = [&](auto FIRST_, auto STORED_, int s, int ns, int nk) __attribute__((always_inline)) {
    v4f P[L + 1];
    const v4f z = {};
    const Bases qm = bases(mine);
    Bases qo{};
    if constexpr (!PF) rd_scales(fa, rg, s, nk);
    // the next stage: of the same group of scales, the next group, or the next tile
    const bool last = s + 1 == ns;
    const int rg1 = last || (s + 1) % kGroup == 0 ? after(rg) : rg;
    const int sl = s + kSlots < ns ? s + kSlots : s + kSlots - ns;   // the stage that is loaded
    const Res r = s + kSlots < ns ? cur : nxt;
#pragma unroll
    for (int x = 0; x < kMf; ++x) {
      const int i = x / CT, j = x % CT;
      P[x % (L + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(Bq[j], Aq[i % kRing], z,
                                                                        0, 0, 0, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (x >= L) fold(FIRST_, x - L, P[(x - L) % (L + 1)]);
      if (j == 0 && i + 2 < RT) Aq[(i + 2) % kRing] = rdA(qm, i + 2);
      if (x == kBarrierAt - 1) {
        wait_vm_lgkm<kYoung + (decltype(STORED_)::value ? kStores : 0)>();
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        qo = bases(other);
      }
      if (x >= kBarrierAt) {
        const int y = x - kBarrierAt;
#pragma unroll
        for (int d = y * kDma / kTail; d < (y + 1) * kDma / kTail; ++d) dma(d, mine, r, sl);
        if constexpr (PF)
          if (y == 1) rd_scales(fn, rg1, last ? 0 : s + 1, nk);
        if (y == 0) Aq[0] = rdA(qo, 0);
        if (y == CT) Aq[1] = rdA(qo, 1);
        if (i == RT - 1) Bq[j] = rdB(qo, j);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int x = kMf - L; x < kMf; ++x) fold(FIRST_, x, P[x % (L + 1)]);
    if constexpr (PF) {
#pragma unroll
      for (int i = 0; i < RT; ++i) fa[i] = fn[i];
    }
    // If the loaded stage begins a group of scales, they go into the region after that of the stage
    // before it: with kSlots regions that is neither stage s + 1's, which slower waves still read,
    // nor one of the stages between. Else the load is an empty one, to the region of zeros.
    int rgl = rg1;
    if constexpr (kSlots == 3)
      rgl = s + 2 == ns || (s + 2 < ns && (s + 2) % kGroup == 0) ? after(rg1) : rg1;
    const bool begins = sl % kGroup == 0;
    dma_scales(begins ? after(rgl) : kSlots, r, sl, begins);
    rg = rg1;
  };

  // A lane's 8 neighbouring columns of a row in one 16-byte store; rows and columns outside the
  // tile's are dropped by the range check, rows without products written as 0 whatever their sums.
  auto epilogue = [&](const Tile& w) __attribute__((always_inline)) {
    uint16_t* d = BROWS == 128 ? a.y + (int64_t)w.m0 * ldd + w.n0
                               : a.y + ((int64_t)w.e * a.N + w.m0) * ldd + w.n0;
    const v4i r = make_rsrc(d, (uint32_t)(((int64_t)(w.rows - 1) * ldd + w.ncols) * 2));
    __amdgpu_buffer_rsrc_t rsD = __builtin_amdgcn_make_buffer_rsrc(
        reinterpret_cast<void*>((uint64_t)(uint32_t)r[0] | (uint64_t)(uint32_t)r[1] << 32), 0, r[2],
        kRsrcWord3);
    int mrow = wm * WTM + r16;
    int ncol = wn * WTN + 16 * (g4 & 1) + 8 * (g4 >> 1);
    asm volatile("" : "+v"(mrow), "+v"(ncol));  // nothing of it is kept over the next tile
    const uint32_t base = ((uint32_t)mrow * (uint32_t)ldd + (uint32_t)ncol) * 2u;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const bool live = mrow + 16 * i < w.live;
#pragma unroll
      for (int jp = 0; jp < CT / 2; ++jp) {
        const int j = 2 * jp;
        const uint32_t p0j = pack_bf16x2(acc[i][j][0], acc[i][j][1]);
        const uint32_t p1j = pack_bf16x2(acc[i][j][2], acc[i][j][3]);
        const uint32_t p0k = pack_bf16x2(acc[i][j + 1][0], acc[i][j + 1][1]);
        const uint32_t p1k = pack_bf16x2(acc[i][j + 1][2], acc[i][j + 1][3]);
        const auto w0 = __builtin_amdgcn_permlane16_swap(p0j, p0k, false, false);
        const auto w1 = __builtin_amdgcn_permlane16_swap(p1j, p1k, false, false);
        v4i o = {(int)w0[0], (int)w1[0], (int)w0[1], (int)w1[1]};
        if (!live) o = v4i{0, 0, 0, 0};
        const bool in = mrow + 16 * i < w.rows && ncol + 32 * jp < w.ncols;
        __builtin_amdgcn_raw_buffer_store_b128(
            o, rsD, in ? base + (uint32_t)(16 * i) * (uint32_t)ldd * 2u + 64u * jp : kOutOfRange, 0,
            0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  auto zero_tile = [&](const Tile& w) {
    uint16_t* d = BROWS == 128 ? a.y + (int64_t)w.m0 * ldd + w.n0
                               : a.y + ((int64_t)w.e * a.N + w.m0) * ldd + w.n0;
    const int pieces = w.ncols / 8;            // 16 bytes each
    for (int i = t; i < w.rows * pieces; i += kTileThreads)
      *reinterpret_cast<uint4*>(d + (int64_t)(i / pieces) * ldd + 8 * (i % pieces)) =
          make_uint4(0, 0, 0, 0);
  };

  for (int first = 0; first < count; first += kBatch) {
    batch_end = min(count, first + kBatch);
    if (first > 0) {                           // every wave is through with the last batch
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __syncthreads();
    }
    if (first + t < batch_end) make_tile(first + t);
    __syncthreads();
    auto with_products = [&](int ti) __attribute__((always_inline)) {   // tile ti or a later one
      while (ti < batch_end && tile_of(ti).nk == 0) ++ti;
      return ti;
    };
    // A tile has at least kSlots stages, so that what is loaded kSlots ahead is its own or the next
    // tile's. Stages past its last block multiply zeros with zeros for scales (a scale may be infinite).
    mine = smem, other = smem + SB, third = smem + (kSlots - 1) * SB;
    int ti = with_products(first), tn = with_products(ti + 1);
    cur = res_of(ti), nxt = res_of(tn);
    rg = 0;
    dma_scales(0, cur, 0, true);
#pragma unroll
    for (int k = 0; k < kSlots; ++k)
#pragma unroll
      for (int d = 0; d < kDma; ++d) dma(d, smem + k * SB, cur, k);
    wait_vm<0>();           // all of them: the first barriers do not wait for the others
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    {
      const Bases q = bases(mine);
#pragma unroll
      for (int j = 0; j < CT; ++j) Bq[j] = rdB(q, j);
      Aq[0] = rdA(q, 0);
      Aq[1] = rdA(q, 1);
      if constexpr (PF) rd_scales(fa, 0, 0, 1);
    }
    while (ti < batch_end) {
      const int nk = tile_of(ti).nk, ns = max(nk, kSlots);
      stage(std::true_type{}, std::true_type{}, 0, ns, nk);
      turn();
      if constexpr (kSlots == 3) {
        stage(std::false_type{}, std::true_type{}, 1, ns, nk);
        turn();
      }
      for (int s = kSlots - 1; s < ns; ++s) {
        stage(std::false_type{}, std::false_type{}, s, ns, nk);
        turn();
      }
      epilogue(tile_of(ti));
      ti = tn, tn = with_products(tn + 1);
      cur = nxt, nxt = res_of(tn);
    }
    // rows of no expert, gradients of experts without rows
    for (int z = first; z < batch_end; ++z)
      if (tile_of(z).nk == 0) zero_tile(tile_of(z));
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");   // no load may land after exit
}

}  // namespace

template <int BROWS, int RT, int kSlots, int kWaves>
hipError_t launch_tiles(const GroupedArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((grouped_tile_kernel<BROWS, RT, kSlots, kWaves>), dim3(kCus * 8 / kWaves),
                     dim3(64 * kWaves), 0, s, a);
  return hipGetLastError();
}

// Rounds of the card, `per` workgroups of it, with tiles of bm x bn.
template <int BROWS>
int64_t rounds(const GroupedArgs& a, int64_t bm, int64_t bn, int64_t per) {
  const int64_t n = ((BROWS == 1 ? a.K : a.N) + bn - 1) / bn;
  return (row_pieces<BROWS>(a, bm) * n + per - 1) / per;
}

// A round of the lower tiles takes 5/8 of one of 256 x 256. Measured, lower to higher in us: y of
// 1024 rows of 8 experts, 14336 x 4096, 147 to 147 at 3 rounds to 2; of 4096 rows of 64, 2048 x 1408,
// 59 to 77 at 3 to 2; of 32768 rows, 148 to 137 at 9 to 5. dw of 8 experts, 1024 x 1024 and 1000 rows
// 22.4 to 31.2 at 1 to 1; of 27, 6272 x 128, 16.1 to 19.6 at 3 to 3; of 8, 2048 x 1024 and 7500 rows
// 206 to 191 at 2 to 1.
//
// Where no expert has more than 256 rows a tile of 256 is at most one an expert's, and never the
// faster one (8 experts, 14336 x 4096, 64 rows each: 127 us to 140).
template <int BROWS>
bool low_tiles(const GroupedArgs& a) {
  if (BROWS != 1 && a.max_rows <= 256) return true;
  const int64_t low = BROWS == 1 ? rounds<1>(a, 128, 128, 2 * kCus)
                                 : rounds<128>(a, 128, 256, kCus);
  return 5 * low <= 8 * rounds<BROWS>(a, 256, 256, kCus);
}

// Less than 10 items of a stream a CU take less than a round of tiles (y of 8 experts' 250 rows: 35.1 us
// to 38.7 at 1024 x 4096, 2112 items, 58.2 to 40.4 at 2048 x 4096, 4224; dw of 8 experts, 512 x 512,
// 1000 rows: 14.4 to 20.6, 2048 items; of 4, 1024 x 1024, 4000 rows: 66.0 to 53.8, 4096). The
// contraction's length is not in it, over which the streams read the weights again for every 32 rows.
// Few columns favour them all the same (y of 5 experts' 1104 rows, 768 x 13952, 54 to 104; of 16
// experts' 500, 1024 x 8192, 57 to 76); many do not, and next to the limit the rule then takes the
// slower side: y of 2 experts' 136 rows, 9088 x 10496, 2556 items, 164 to 100; of 4 experts' 100 tokens
// with two choices, 8192 x 4096, 47.0 to 46.3.
template <int BROWS>
bool few_items(const GroupedArgs& a) {
  const int64_t columns = (BROWS == 1 ? a.K : a.N) / 32;
  return row_pieces<BROWS>(a, 32) * columns < 10 * (int64_t)kCus;
}

// Where no expert has more than 64 rows a stream reads the weights about once, and faster (8 experts,
// 14336 x 4096, 16 rows on average: 102 us to 122; 22 of 3456 x 384, 21 rows: 13.8 to 18.6).
hipError_t launch_grouped_gemm(const GroupedArgs& a, hipStream_t s) {
  if (a.max_rows <= 8) return launch_stream<128, 8, 2>(a, s);
  if (a.max_rows <= 64 || a.rows <= 32 * (int64_t)a.experts || few_items<128>(a))
    return launch_stream<128, 32, 1>(a, s);
  return low_tiles<128>(a) ? launch_tiles<128, 4, 3, 8>(a, s) : launch_tiles<128, 8, 2, 8>(a, s);
}

hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s) {
  if (few_items<1>(a)) return launch_stream<1, 32, 1>(a, s);
  return low_tiles<1>(a) ? launch_tiles<1, 4, 2, 4>(a, s) : launch_tiles<1, 8, 2, 8>(a, s);
}

}  // namespace fp8lin
