// The router of an expert block: softmax over the experts, the topk choices with their weights,
// the pairs per expert, the balance loss and the z-loss, and the gradient of all of them.
//
// For the logits l[t, e] of the valid tokens (T of them), with p = softmax(l), lse = log sum exp:
//
//     idx[t, :]    the k largest logits in falling order, equal ones by the lower expert
//     w[t, j]      p at idx[t, j], or with `normalize` divided by their sum over j
//     counts[e]    pairs that chose e;  P[e] = (1/T) sum_t p[t, e]
//     losses       { E / (T k) sum_e counts[e] P[e],  (1/T) sum_t lse[t]^2 }
//
// A logit of -inf is a masked expert: never chosen, p = 0. A row without any other has idx -1,
// w 0, lse -inf, and adds nothing to P and to the losses. NaN ranks above every number; a row with it
// or with +inf has NaN for p of every expert that is not masked.
//
// G consecutive lanes hold a token's logits, NV each, so the sums and maxima are DPP steps of log2 G.
// A choice is the maximum of the unsigned keys that order like the logits; for 16-bit types the key's
// lower half is the complement of the expert, which makes the same maximum also break ties. The sums
// of p stay in the lanes that own the expert until a workgroup's tokens are done, and pairs are counted
// in LDS; the workgroups' partial sums are added by a second launch in a fixed order (integer atomics
// alone: the same inputs give the same bits).
//
// What bounds it: up to some 2000 tokens the launches (64 tokens, 2 of 8 experts 4.6 us; two launches
// 8.8). Beyond, the instructions of the choices rather than memory: 32768 tokens, 8 of 256, bf16 27.0
// us, of which 6.4 are the bytes' and a launch's. A lane so keeps its keys unchanged (34 us when each
// choice took its key out and counted the pair in registers), and a token has few lanes (the gradient,
// which has no choices to make, has more).
#include "common.h"
#include "launch.h"
#include "rows.h"

namespace fp8lin {

namespace {

constexpr int kRouteThreads = 512, kRouteWaves = kRouteThreads / 64;
constexpr int kRouteBwdThreads = 256;
constexpr int64_t kRouteMaxBlocks = 256;
constexpr float kLog2e = 1.4426950408889634f;

template <int CTRL> __device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// Maximum over groups of LANES consecutive lanes; every lane gets it.
template <int LANES> __device__ __forceinline__ uint32_t lanes_max_u32(uint32_t v) {
  if constexpr (LANES >= 2) v = max(v, dpp_u<0xB1>(v));
  if constexpr (LANES >= 4) v = max(v, dpp_u<0x4E>(v));
  if constexpr (LANES >= 8) v = max(v, dpp_u<0x141>(v));
  if constexpr (LANES >= 16) v = max(v, dpp_u<0x140>(v));
  if constexpr (LANES >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max((uint32_t)r[0], (uint32_t)r[1]);
  }
  if constexpr (LANES >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max((uint32_t)r[0], (uint32_t)r[1]);
  }
  return v;
}

template <int LANES> __device__ __forceinline__ float lanes_max(float v) {
  if constexpr (LANES >= 2) v = __builtin_fmaxf(v, dpp<0xB1>(v));
  if constexpr (LANES >= 4) v = __builtin_fmaxf(v, dpp<0x4E>(v));
  if constexpr (LANES >= 8) v = __builtin_fmaxf(v, dpp<0x141>(v));
  if constexpr (LANES >= 16) v = __builtin_fmaxf(v, dpp<0x140>(v));
  if constexpr (LANES >= 32) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (LANES >= 64) {
    const uint32_t u = __float_as_uint(v);
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    v = __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}

// Unsigned keys that order like the numbers (-0 as +0, NaN above all); 0 stands for -inf, which
// cannot be chosen. B: the bits of the number, in 16 or 32 bits; INF: those of infinity.
template <typename B, B INF> __device__ __forceinline__ B order_key(B b) {
  constexpr B kSign = (B)((B)1 << (8 * sizeof(B) - 1));
  const B mag = (B)(b & (B)~kSign);
  B k = (b & kSign) ? (B)~b : (B)(b | kSign);
  k = mag == 0 ? kSign : k;
  k = b == (B)(kSign | INF) ? (B)0 : k;
  return mag > INF ? (B)~(B)0 : k;
}
template <typename B> __device__ __forceinline__ B key_bits(B k) {   // of a key that is not 0
  constexpr B kSign = (B)((B)1 << (8 * sizeof(B) - 1));
  return (k & kSign) ? (B)(k ^ kSign) : (B)~k;                       // NaN's is a NaN again
}
template <typename T> struct Logit;
template <> struct Logit<BF16> { using Bits = uint16_t; static constexpr Bits kInf = 0x7F80; };
template <> struct Logit<F16> { using Bits = uint16_t; static constexpr Bits kInf = 0x7C00; };
template <> struct Logit<float> { using Bits = uint32_t; static constexpr Bits kInf = 0x7F800000u; };

template <typename T> __device__ __forceinline__ T masked_logit() {
  using B = typename Logit<T>::Bits;
  return __builtin_bit_cast(T, (B)(Logit<T>::kInf | (B)((B)1 << (8 * sizeof(B) - 1))));
}

// A token's experts over G lanes, NV each: pieces of V neighbouring experts, piece after piece
// over the lanes, so that a group's loads are whole lines.
template <int G, int NV> struct Lanes {
  static constexpr int V = NV < 4 ? NV : 4;
  static constexpr int kMaxK = G * NV < kMoeMaxTopk ? G * NV : kMoeMaxTopk;
  static constexpr int kSlots = (kMaxK + G - 1) / G;            // choices per lane
  static __device__ __forceinline__ int expert(int gl, int i) {
    return i / V * (G * V) + gl * V + i % V;
  }
};

// A lane's logits, -inf past the last expert and in rows that are not live.
template <int G, int NV, typename T>
__device__ __forceinline__ void load_logits(const T* row, int gl, int E, bool live, T (&x)[NV]) {
  using L = Lanes<G, NV>;
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = masked_logit<T>();
  if (!live) return;
#pragma unroll
  for (int i = 0; i < NV; i += L::V) {
    const int c = L::expert(gl, i);
    if (c + L::V <= E) {
      __builtin_memcpy(&x[i], row + c, L::V * sizeof(T));
    } else {
#pragma unroll
      for (int j = 0; j < L::V; ++j)
        if (c + j < E) x[i + j] = row[c + j];
    }
  }
}

// The losses from a workgroup's sums over the experts, cp (a lane's part of sum_e counts[e] prob[e])
// and over the tokens, z (the whole). All lanes of at most 16 waves call it.
__device__ __forceinline__ void write_losses(float* lds, float cp, float z, float scale,
                                             int64_t valid, float* losses) {
  const int t = threadIdx.x, waves = (blockDim.x + 63) / 64;
  cp = lanes_sum<64>(cp);
  if ((t & 63) == 0) lds[t >> 6] = cp;
  __syncthreads();
  if (t == 0) {
    float s = 0.f;
    for (int w = 0; w < waves; ++w) s += lds[w];
    losses[0] = valid > 0 ? s * scale : 0.f;
    losses[1] = valid > 0 ? z / (float)valid : 0.f;
  }
}

// LDS written by lanes of this wave is read by others of it: the hardware keeps a wave's LDS
// operations in order, the fence keeps the compiler's order the same.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A workgroup's sums for an expert: of p, and its pairs.
struct Part { float p; int c; };

template <typename T, int G, int NV>
__global__ void __launch_bounds__(kRouteThreads)
moe_route_kernel(const T* __restrict__ logits, int64_t ldl, int64_t tokens, int64_t valid, int E,
                 int k, bool normalize, int32_t* __restrict__ idx, float* __restrict__ weights,
                 float* __restrict__ lse, int32_t* __restrict__ counts,
                 float* __restrict__ losses, Part* __restrict__ part, float* __restrict__ zpart,
                 uint32_t* __restrict__ arrived, float loss_scale) {
  using L = Lanes<G, NV>;
  using Bits = typename Logit<T>::Bits;
  constexpr bool k16 = sizeof(T) == 2;
  constexpr int kTokens = kRouteThreads / G;                    // of a step
  __shared__ float sums[kRouteWaves][G * NV];
  __shared__ int s_cnt[G * NV];                                 // pairs of an expert
  __shared__ int s_choice[k16 ? 1 : kTokens][k16 ? 1 : L::kMaxK];   // a token's experts
  __shared__ float s_z[kRouteWaves], s_red[16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, gl = lane % G;
  float psum[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) psum[i] = 0.f;
  float zsum = 0.f;
  for (int e = t; e < G * NV; e += kRouteThreads) s_cnt[e] = 0;
  __syncthreads();

  // whole waves stay in the loop, so that the lane exchanges see every lane
  for (int64_t base = (int64_t)blockIdx.x * kTokens; base < tokens;
       base += (int64_t)gridDim.x * kTokens) {
    const int64_t tok = base + t / G;
    const bool live = tok < valid;
    T raw[NV];
    load_logits<G>(logits + tok * ldl, gl, E, live, raw);
    float x[NV];
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = to_f32(raw[i]);
      key[i] = order_key<Bits, Logit<T>::kInf>(__builtin_bit_cast(Bits, raw[i]));
      if (k16 && key[i]) key[i] = key[i] << 16 | (uint32_t)(0xFFFF - L::expert(gl, i));
    }
    uint32_t rec[L::kSlots], first = 0u;       // keys of this lane's choices j = s G + gl
#pragma unroll
    for (int s = 0; s < L::kSlots; ++s) rec[s] = 0u;
    uint32_t above = 0u;                       // 16 bits: the last choice, keys below it are left
    for (int j = 0; j < k; ++j) {
      // modulo 2^32 a key k < above has k - above >= 2^32 - above, one of at least `above` less
      uint32_t m = key[0] - above;
#pragma unroll
      for (int i = 1; i < NV; ++i) m = max(m, key[i] - above);
      const uint32_t gm = lanes_max_u32<G>(m) + above;
      if (j == 0) first = gm;
#pragma unroll
      for (int s = 0; s < L::kSlots; ++s)
        if (j == s * G + gl) rec[s] = gm;
      if constexpr (k16) {
        above = max(gm, 1u);
      } else {
        // the lane's lowest expert with the maximum; where lanes share it, only the lowest of them
        uint32_t low = 0u;
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
          if (key[i] == gm) low = (uint32_t)(0xFFFF - L::expert(gl, i));
        if (__builtin_popcountll(__ballot(low != 0u)) != 64 / G)
          low = lanes_max_u32<G>(low) == low ? low : 0u;
        if (low != 0u && gm != 0u) s_choice[t / G][j] = 0xFFFF - (int)low;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          key[i] = low == (uint32_t)(0xFFFF - L::expert(gl, i)) ? 0u : key[i];
      }
    }
    if constexpr (!k16) wave_lds_fence();
    auto value = [](uint32_t q) __attribute__((always_inline)) {       // of a key of the loop
      if (q == 0u) return -INFINITY;
      if constexpr (k16) return to_f32(__builtin_bit_cast(T, key_bits((Bits)(q >> 16))));
      else return __uint_as_float(key_bits(q));
    };
    const float top = value(first);
    int rec_e[L::kSlots];
    float rec_v[L::kSlots];
#pragma unroll
    for (int s = 0; s < L::kSlots; ++s) {
      rec_v[s] = value(rec[s]);
      rec_e[s] = -1;
      if (rec[s] != 0u) {
        if constexpr (k16) rec_e[s] = 0xFFFF - (int)(rec[s] & 0xFFFFu);
        else rec_e[s] = s_choice[t / G][s * G + gl];
        atomicAdd(&s_cnt[rec_e[s]], 1);
      }
    }
    if constexpr (!k16) wave_lds_fence();      // read before the next step's choices are written
    const bool none = top == -INFINITY;        // no expert left (not so for NaN)
    float total = 0.f, wsum = 0.f, w[L::kSlots];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = none ? 0.f : __builtin_amdgcn_exp2f((x[i] - top) * kLog2e);
      total += x[i];
    }
    total = lanes_sum<G>(total);
    const float inv = none ? 0.f : __builtin_amdgcn_rcpf(total);
#pragma unroll
    for (int i = 0; i < NV; ++i) psum[i] += x[i] * inv;
#pragma unroll
    for (int s = 0; s < L::kSlots; ++s) {
      w[s] = rec_e[s] < 0 ? 0.f : __builtin_amdgcn_exp2f((rec_v[s] - top) * kLog2e);
      wsum += w[s];
    }
    wsum = lanes_sum<G>(wsum);
    const float f = !normalize ? inv : none ? 0.f : __builtin_amdgcn_rcpf(wsum);
    const float row_lse = none ? -INFINITY : top + __logf(total);
    if (gl == 0 && !none) zsum += row_lse * row_lse;
    if (tok < tokens) {
#pragma unroll
      for (int s = 0; s < L::kSlots; ++s) {
        const int j = s * G + gl;
        if (j < k) {
          idx[tok * k + j] = rec_e[s];
          weights[tok * k + j] = rec_e[s] < 0 ? 0.f : w[s] * f;     // f may be NaN
        }
      }
      if (gl == 0) lse[tok] = live ? row_lse : 0.f;
    }
  }

  // the workgroup's sums: over the groups of a wave, then over the waves
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int off = 32; off >= G; off >>= 1) psum[i] += __shfl_xor(psum[i], off, 64);
    if (lane < G) sums[wave][L::expert(gl, i)] = psum[i];
  }
  zsum = lanes_sum<64>(zsum);
  if (lane == 0) s_z[wave] = zsum;
  __syncthreads();
  float z = 0.f;
#pragma unroll
  for (int w = 0; w < kRouteWaves; ++w) z += s_z[w];
  float cp = 0.f;
  for (int e = t; e < E; e += kRouteThreads) {
    Part s = {0.f, s_cnt[e]};
#pragma unroll
    for (int w = 0; w < kRouteWaves; ++w) s.p += sums[w][e];
    if (gridDim.x == 1) {
      counts[e] = s.c;
      cp += (float)s.c * s.p;
    } else {
      part[(int64_t)blockIdx.x * E + e] = s;
    }
  }
  if (gridDim.x == 1) {
    write_losses(s_red, cp, z, loss_scale, valid, losses);
  } else if (t == 0) {
    zpart[blockIdx.x] = z;
    if (blockIdx.x == 0) *arrived = 0u;
  }
}

// Adds the partial sums of `blocks` workgroups, kLossExperts experts a workgroup: a lane takes two
// experts' sums of every 32nd block, 8 loads at a time, since a workgroup's time is that of the
// round trips it takes (6.7 us with one expert a lane and 4 rounds of 8, 3.9 with one). With several
// workgroups the last one to arrive adds their parts of the losses up, in their order; the forward
// kernel has set `arrived` to 0.
constexpr int kLossExperts = 64, kLossThreads = 1024;
struct LossPart { uint32_t arrived; float cp[kMoeMaxExperts / kLossExperts]; };

__global__ void __launch_bounds__(kLossThreads)
moe_route_losses_kernel(const Part* __restrict__ part, const float* __restrict__ zpart, int blocks,
                        int E, int32_t* __restrict__ counts, float* __restrict__ losses,
                        LossPart* last, int64_t valid, float loss_scale) {
  constexpr int kPairs = kLossExperts / 2, kWays = kLossThreads / kPairs, kAhead = 8;
  __shared__ Part sums[kWays][kLossExperts];
  __shared__ float s_red[16], s_z[16];
  const int t = threadIdx.x, c = 2 * (t % kPairs), r = t / kPairs;
  const int e = blockIdx.x * kLossExperts + c;
  Part s[2] = {{0.f, 0}, {0.f, 0}};
  for (int b0 = r; b0 < blocks; b0 += kAhead * kWays) {
    Part v[kAhead][2];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int b = b0 + i * kWays;
      v[i][0] = v[i][1] = {0.f, 0};
      if (b < blocks && e + 2 <= E) __builtin_memcpy(v[i], part + (int64_t)b * E + e, 16);
      else if (b < blocks && e < E) v[i][0] = part[(int64_t)b * E + e];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) s[j].p += v[i][j].p, s[j].c += v[i][j].c;
  }
  sums[r][c] = s[0], sums[r][c + 1] = s[1];
  float z = lanes_sum<64>(t < blocks ? zpart[t] : 0.f);
  static_assert(kRouteMaxBlocks <= kLossThreads, "one lane a block");
  if ((t & 63) == 0) s_z[t >> 6] = z;
  __syncthreads();
  z = 0.f;
  for (int w = 0; w < kLossThreads / 64; ++w) z += s_z[w];
  float cp = 0.f;
  if (t < kLossExperts && blockIdx.x * kLossExperts + t < E) {
    Part q = {0.f, 0};
    for (int i = 0; i < kWays; ++i) q.p += sums[i][t].p, q.c += sums[i][t].c;
    counts[blockIdx.x * kLossExperts + t] = q.c;
    cp = (float)q.c * q.p;
  }
  if (gridDim.x == 1) {
    write_losses(s_red, cp, z, loss_scale, valid, losses);
    return;
  }
  if (t >= 64) return;                         // the sums of cp are the first wave's
  cp = lanes_sum<64>(cp);
  if (t != 0) return;
  __hip_atomic_store(&last->cp[blockIdx.x], cp, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint32_t before = __hip_atomic_fetch_add(&last->arrived, 1u, __ATOMIC_ACQ_REL,
                                                 __HIP_MEMORY_SCOPE_AGENT);
  if (before + 1 != gridDim.x) return;
  float total = 0.f;
  for (unsigned i = 0; i < gridDim.x; ++i)
    total += __hip_atomic_load(&last->cp[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  losses[0] = valid > 0 ? total * loss_scale : 0.f;
  losses[1] = valid > 0 ? z / (float)valid : 0.f;
}

// dl[t, e] = p (A (c[e] - sum_e p c) + B lse - [not normalized] sum_j w dw)
//            + [e = idx[t, j]] w_j (dw_j - [normalized] sum_j w dw)
// with A = dlosses[0] E / (T^2 k) and B = dlosses[1] 2 / T, c the counts. The softmax is made again
// from the row itself: exp(l - lse) would lose what lse rounds off, all of log E in a row of the
// type's lowest values. The choices' terms reach the lanes that own the experts through LDS, a row
// of it for each token, within the wave.
template <typename T, int G, int NV>
__global__ void __launch_bounds__(kRouteBwdThreads)
moe_route_bwd_kernel(const T* __restrict__ logits, int64_t ldl, int64_t tokens, int64_t valid,
                     int E, int k, bool normalize, const float* __restrict__ lse,
                     const int32_t* __restrict__ idx, const float* __restrict__ weights,
                     const int32_t* __restrict__ counts, const float* __restrict__ dweights,
                     const float* __restrict__ dlosses, float a_scale, float b_scale,
                     T* __restrict__ dlogits) {
  using L = Lanes<G, NV>;
  constexpr int kTokens = kRouteBwdThreads / G;
  __shared__ __attribute__((aligned(16))) float rows[kTokens][G * NV];
  const int t = threadIdx.x, lane = t & 63, gl = lane % G;
  const int64_t tok = (int64_t)blockIdx.x * kTokens + t / G;
  const bool live = tok < valid;
  T x[NV];
  load_logits<G>(logits + tok * ldl, gl, E, live, x);
  const float A = dlosses ? dlosses[0] * a_scale : 0.f;
  const float B = dlosses ? dlosses[1] * b_scale : 0.f;
  const float l = live ? lse[tok] : 0.f;
  float* const row = rows[t / G];
  float dot = 0.f;
  if (dweights) {
    int e[L::kSlots];
    float w[L::kSlots], dw[L::kSlots];
#pragma unroll
    for (int s = 0; s < L::kSlots; ++s) {
      const int j = s * G + gl;
      e[s] = -1, w[s] = 0.f, dw[s] = 0.f;
      if (live && j < k) {
        e[s] = idx[tok * k + j];
        w[s] = weights[tok * k + j];
        dw[s] = dweights[tok * k + j];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; i += L::V)
#pragma unroll
      for (int j = 0; j < L::V; ++j) row[L::expert(gl, i) + j] = 0.f;
#pragma unroll
    for (int s = 0; s < L::kSlots; ++s) {
      if (e[s] < 0 || e[s] >= E) e[s] = -1, w[s] = 0.f, dw[s] = 0.f;
      dot += w[s] * dw[s];
    }
    dot = lanes_sum<G>(dot);
    wave_lds_fence();                          // the zeros of this wave's rows come first
#pragma unroll
    for (int s = 0; s < L::kSlots; ++s)
      if (e[s] >= 0) unsafeAtomicAdd(&row[e[s]], w[s] * (dw[s] - (normalize ? dot : 0.f)));
    wave_lds_fence();
  }
  float top = to_f32(x[0]);
#pragma unroll
  for (int i = 1; i < NV; ++i) top = __builtin_fmaxf(top, to_f32(x[i]));
  top = lanes_max<G>(top);
  if (top == -INFINITY) top = 0.f;             // then the sum is 0, or NaN where the row has one
  float p[NV], pc = 0.f, total = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    p[i] = __builtin_amdgcn_exp2f((to_f32(x[i]) - top) * kLog2e);
    total += p[i];
  }
  total = lanes_sum<G>(total);
  const bool none = total == 0.f;              // no expert left: p = 0
  const float inv = none ? 0.f : __builtin_amdgcn_rcpf(total);
  const float rest = none ? 0.f : B * l - (normalize ? 0.f : dot);
  float d[NV];
  if (dlosses) {
    float c[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = L::expert(gl, i);
      c[i] = e < E ? (float)counts[e] : 0.f;
      pc += p[i] * c[i];
    }
    pc = lanes_sum<G>(pc) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = p[i] * inv * fmaf(A, c[i] - pc, rest);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = p[i] * inv * rest;
  }
  // a masked expert's is 0 also where the rest of the row is not finite
#pragma unroll
  for (int i = 0; i < NV; ++i) d[i] = to_f32(x[i]) == -INFINITY ? 0.f : d[i];
  if (dweights) {
#pragma unroll
    for (int i = 0; i < NV; i += L::V)
#pragma unroll
      for (int j = 0; j < L::V; ++j) d[i + j] += row[L::expert(gl, i) + j];
  }
  if (tok >= tokens) return;
#pragma unroll
  for (int i = 0; i < NV; i += L::V) {
    const int c = L::expert(gl, i);
    T o[L::V];
#pragma unroll
    for (int j = 0; j < L::V; ++j) o[j] = from_f32<T>(d[i + j]);
    T* const out = dlogits + tok * E + c;
    if (c + L::V <= E) {
      __builtin_memcpy(out, o, sizeof(o));
    } else {
#pragma unroll
      for (int j = 0; j < L::V; ++j)
        if (c + j < E) out[j] = o[j];
    }
  }
}

// Lanes of a token and experts of a lane. A round of the forward's choice takes NV steps and log2 G
// exchanges for 64 / G tokens, so wider rows take more lanes, but not all of a wave. The backward
// has no rounds and gains by more waves: 16384 rows of 256 in f32 take 12.5 us with 16 lanes a
// token, 11.6 with 32, 10.7 with 64.
template <bool BWD, typename F>
hipError_t by_experts(int E, F f) {
  auto with = [&](auto g, auto nv) { return f(g, nv); };
#define FP8LIN_LANES(G, NV) \
  with(std::integral_constant<int, G>{}, std::integral_constant<int, NV>{})
  if (E <= 8) return FP8LIN_LANES(8, 1);
  if (E <= 16) return FP8LIN_LANES(16, 1);
  if (E <= 32) return FP8LIN_LANES(16, 2);
  if (E <= 64) return FP8LIN_LANES(16, 4);
  if (E <= 128) return FP8LIN_LANES(32, 4);
  if (E <= 256) return with(std::integral_constant<int, BWD ? 64 : 32>{},
                            std::integral_constant<int, BWD ? 4 : 8>{});
  return FP8LIN_LANES(64, 8);
#undef FP8LIN_LANES
}

template <typename F> hipError_t by_dtype(int dtype, F f) {
  if (dtype == kBF16) return f(BF16{});
  if (dtype == kF16) return f(F16{});
  return f(0.0f);
}

// Steps of a workgroup's tokens.
int64_t route_steps(int64_t tokens, int32_t E) {
  const int64_t per = kRouteThreads / (E <= 8 ? 8 : E <= 64 ? 16 : E <= 256 ? 32 : 64);
  return (tokens + per - 1) / per;
}
int64_t route_blocks(int64_t steps) {
  return steps <= 2 ? 1 : steps < kRouteMaxBlocks ? steps : kRouteMaxBlocks;
}
// Whether one workgroup takes them all and writes the losses: a step's time goes with the choices,
// that of a second launch is 4 to 5 us (7.3 us to 9.1 for 8 steps of 2 of 7 experts, 11.8 to 8.8 for
// 16; 7.3 to 8.6 for 4 steps of 10 of 16, 9.9 to 8.8 for 6; 7.9 to 8.7 for 4 steps of 3 of 125, 10.9
// to 8.8 for 4 of 8 of 64).
bool one_workgroup(int64_t steps, int32_t E, int32_t k) {
  return steps <= 2 || steps * (k + 2) <= (E <= 16 ? 48 : 24);
}

}  // namespace

int64_t moe_route_workspace(int64_t tokens, int32_t experts) {
  const int64_t blocks = route_blocks(route_steps(tokens, experts));
  return blocks == 1 ? 0 : blocks * (experts * (int64_t)sizeof(Part) + 4) + (int64_t)sizeof(LossPart);
}

hipError_t launch_moe_route(const MoeRouteArgs& a, hipStream_t s) {
  const int64_t steps = route_steps(a.tokens, a.experts);
  const int64_t blocks = one_workgroup(steps, a.experts, a.topk) ? 1 : route_blocks(steps);
  const double t = (double)(a.valid > 0 ? a.valid : 1);
  const float scale = (float)((double)a.experts / (t * t * a.topk));
  Part* const part = reinterpret_cast<Part*>(a.workspace);
  float* const zpart = blocks == 1 ? nullptr : reinterpret_cast<float*>(part + blocks * a.experts);
  LossPart* const last = blocks == 1 ? nullptr : reinterpret_cast<LossPart*>(zpart + blocks);
  hipError_t e = by_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_experts<false>(a.experts, [&](auto g, auto nv) {
      hipLaunchKernelGGL((moe_route_kernel<T, decltype(g)::value, decltype(nv)::value>),
                         dim3((unsigned)blocks), dim3(kRouteThreads), 0, s,
                         static_cast<const T*>(a.logits), a.ldl, a.tokens, a.valid, a.experts,
                         a.topk, a.normalize, a.idx, a.weights, a.lse, a.counts, a.losses,
                         part, zpart, blocks == 1 ? nullptr : &last->arrived, scale);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess || blocks == 1) return e;
  hipLaunchKernelGGL(moe_route_losses_kernel,
                     dim3((unsigned)((a.experts + kLossExperts - 1) / kLossExperts)),
                     dim3(kLossThreads), 0, s, part, zpart, (int)blocks, a.experts, a.counts,
                     a.losses, last, a.valid, scale);
  return hipGetLastError();
}

// A launch has fewer than 2^32 threads: more tokens (2^25 of more than 128 experts) take several.
constexpr int64_t kRouteBwdMaxBlocks = (int64_t)1 << 23;

hipError_t launch_moe_route_bwd(const MoeRouteArgs& a, hipStream_t s) {
  const double t = (double)(a.valid > 0 ? a.valid : 1);
  const float sa = (float)((double)a.experts / (t * t * a.topk)), sb = (float)(2.0 / t);
  return by_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_experts<true>(a.experts, [&](auto g, auto nv) {
      constexpr int G = decltype(g)::value, kTokens = kRouteBwdThreads / G;
      for (int64_t t0 = 0; t0 < a.tokens; t0 += kRouteBwdMaxBlocks * kTokens) {
        const int64_t n = min(a.tokens - t0, kRouteBwdMaxBlocks * kTokens), pairs = t0 * a.topk;
        hipLaunchKernelGGL((moe_route_bwd_kernel<T, G, decltype(nv)::value>),
                           dim3((unsigned)((n + kTokens - 1) / kTokens)), dim3(kRouteBwdThreads), 0, s,
                           static_cast<const T*>(a.logits) + t0 * a.ldl, a.ldl, n, a.valid - t0,
                           a.experts, a.topk, a.normalize, a.lse + t0, a.idx + pairs,
                           a.weights + pairs, a.counts, a.dweights ? a.dweights + pairs : nullptr,
                           a.dlosses, sa, sb, static_cast<T*>(a.dlogits) + t0 * a.experts);
        if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
      }
      return hipSuccess;
    });
  });
}

}  // namespace fp8lin
