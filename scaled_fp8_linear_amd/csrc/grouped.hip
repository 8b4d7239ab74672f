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

namespace fp8lin {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(1)));

constexpr int kBlock = 128;                  // codes per scale

// The rows of expert e: first, one past the last, one past its padding.
struct Span { int64_t first, end, next; };
__device__ __forceinline__ Span expert_span(const int32_t* offsets, const int32_t* counts, int e,
                                            int64_t rows) {
  const int64_t a = min(max((int64_t)offsets[e], (int64_t)0), rows);
  const int64_t b = min(max((int64_t)offsets[e + 1], a), rows);
  return {a, min(a + max((int64_t)counts[e], (int64_t)0), b), b};
}

__device__ __forceinline__ v8i frag(const uint8_t* p) {   // a lane's 32 codes
  const v4u_any* q = reinterpret_cast<const v4u_any*>(p);
  const v4u lo = q[0], hi = q[1];
  return v8i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
             (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}
__device__ __forceinline__ v4f mfma(v8i b, v8i a) {
  const v4f z = {};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, z, 0, 0, 0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Few rows per expert: a workgroup makes 32 columns of an expert's rows, its 8 waves taking the
// K blocks in turn, and adds their sums up through LDS. Operands go from memory to registers.
constexpr int kFewWaves = 8, kFewCols = 32, kFewRows = 16;

__global__ void __launch_bounds__(64 * kFewWaves)
grouped_few_kernel(GroupedArgs a) {
  __shared__ float sums[kFewWaves][kFewRows][kFewCols + 1];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int r16 = lane & 15, g4 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * kFewCols;
  const int e = blockIdx.y;
  const int64_t kblocks = a.K / kBlock;
  if (e == a.experts) {                      // the rows past the last expert's and before the first's
    const Span last = expert_span(a.offsets, a.counts, a.experts - 1, a.rows);
    const Span head = expert_span(a.offsets, a.counts, 0, a.rows);
    for (int64_t i = t; i < (a.rows - last.next) * kFewCols; i += blockDim.x)
      a.y[(last.next + i / kFewCols) * a.N + n0 + i % kFewCols] = 0;
    for (int64_t i = t; i < head.first * kFewCols; i += blockDim.x)
      a.y[i / kFewCols * a.N + n0 + i % kFewCols] = 0;
    return;
  }
  const Span s = expert_span(a.offsets, a.counts, e, a.rows);
  const uint8_t* w = a.w + e * a.stride_w + n0 * a.ldw + 32 * g4;
  const float* sw = a.sw + e * a.stride_sw + n0 / kBlock * a.ldsw;
  for (int64_t m0 = s.first; m0 < s.end; m0 += kFewRows) {
    const bool live = m0 + r16 < s.end;
    const int64_t row = live ? m0 + r16 : s.first;
    const uint8_t* x = a.x + row * a.K + 32 * g4;
    v4f acc[2] = {};
    for (int64_t kb = wave; kb < kblocks; kb += kFewWaves) {
      v8i xa = frag(x + kb * kBlock);
      const float f = (live ? a.sx[row * kblocks + kb] : 0.f) * sw[kb];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const v4f p = mfma(frag(w + (16 * j + r16) * a.ldw + kb * kBlock), xa);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = fmaf(p[r], f, acc[j][r]);
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) sums[wave][r16][16 * j + 4 * g4 + r] = acc[j][r];
    __syncthreads();
    const int m = t / kFewCols, n = t % kFewCols;        // 512 lanes: 16 x 32
    if (m0 + m < s.end) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kFewWaves; ++q) v += sums[q][m][n];
      a.y[(m0 + m) * a.N + n0 + n] = (uint16_t)f32_to_bf16_bits(v);
    }
    __syncthreads();
  }
  for (int64_t i = t; i < (s.next - s.end) * kFewCols; i += blockDim.x)   // padding rows
    a.y[(s.end + i / kFewCols) * a.N + n0 + i % kFewCols] = 0;
}

// ---------------------------------------------------------------------------
// Weight gradient: a wave makes 64 x 64 elements of dw, operands from memory to registers.
__global__ void __launch_bounds__(256)
grouped_wgrad_kernel(GroupedArgs a) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int r16 = lane & 15, g4 = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.y * 128 + 64 * (wave >> 1);
  const int64_t k0 = (int64_t)blockIdx.x * 128 + 64 * (wave & 1);
  const int e = blockIdx.z;
  const Span s = expert_span(a.offsets, a.counts, e, a.rows);
  const int64_t rblocks = a.rows / kBlock;
  const int64_t b0 = s.first / kBlock, b1 = s.end > s.first ? (s.end + kBlock - 1) / kBlock : b0;
  v4f acc[4][4] = {};
  for (int64_t b = b0; b < b1; ++b) {
    v8i g[4];
    float sg[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g[j] = frag(a.w + (n0 + 16 * j + r16) * a.rows + b * kBlock + 32 * g4);
#pragma unroll
      for (int r = 0; r < 4; ++r) sg[j][r] = a.sw[(n0 + 16 * j + 4 * g4 + r) * rblocks + b];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = k0 + 16 * i + r16;
      const v8i x = frag(a.x + k * a.rows + b * kBlock + 32 * g4);
      const float sx = a.sx[k * rblocks + b];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4f p = mfma(g[j], x);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = fmaf(p[r], sx * sg[j][r], acc[i][j][r]);
      }
    }
  }
  uint16_t* out = a.y + (int64_t)e * a.N * a.K;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        out[(n0 + 16 * j + 4 * g4 + r) * a.K + k0 + 16 * i + r16] =
            (uint16_t)f32_to_bf16_bits(acc[i][j][r]);
}

}  // namespace

hipError_t launch_grouped_gemm(const GroupedArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(grouped_few_kernel, dim3((unsigned)(a.N / kFewCols), a.experts + 1),
                     dim3(64 * kFewWaves), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const GroupedArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(grouped_wgrad_kernel,
                     dim3((unsigned)(a.K / 128), (unsigned)(a.N / 128), a.experts), dim3(256), 0, s,
                     a);
  return hipGetLastError();
}

}  // namespace fp8lin
