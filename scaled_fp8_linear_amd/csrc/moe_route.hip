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
// w 0, lse -inf, and adds nothing to P and to the losses. NaN ranks above every number.
//
// G consecutive lanes hold a token's logits, NV each (expert = lane NV + i), so the sums and
// maxima are DPP steps of log2 G. A choice is the maximum of the unsigned keys that order like
// the logits; for 16-bit types the key's lower half is the complement of the expert, which makes
// the same maximum also break ties. The counts and sums of p stay in the lanes that own the
// expert until a workgroup's tokens are done; the workgroups' partial sums are added by a second
// launch in a fixed order (no atomics: the same inputs give the same bits).
#include "common.h"
#include "launch.h"
#include "rows.h"

namespace fp8lin {

namespace {

constexpr int kRouteThreads = 256;
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
  if (mag > INF) return (B)~(B)0;
  if (b == (B)(kSign | INF)) return (B)0;
  if (mag == 0) return kSign;
  return (b & kSign) ? (B)~b : (B)(b | kSign);
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

// A lane's logits, -inf past the last expert and in rows that are not live.
template <int NV, typename T>
__device__ __forceinline__ void load_logits(const T* row, int c0, int E, bool live, T (&x)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = masked_logit<T>();
  if (!live) return;
  if (c0 + NV <= E) {
    __builtin_memcpy(x, row + c0, sizeof(x));
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c0 + i < E) x[i] = row[c0 + i];
  }
}

template <int G, int NV> struct Lanes {
  static constexpr int kGroups = kRouteThreads / G;             // tokens of a workgroup's step
  static constexpr int kMaxK = G * NV < kMoeMaxTopk ? G * NV : kMoeMaxTopk;
  static constexpr int kSlots = (kMaxK + G - 1) / G;            // choices per lane
};

// counts[e] and prob[e] (sums over the tokens) -> counts and the two losses; all lanes of the
// workgroup (at most 1024) call it. `lds`: 16 floats.
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

template <typename T, int G, int NV>
__global__ void __launch_bounds__(kRouteThreads)
moe_route_kernel(const T* __restrict__ logits, int64_t ldl, int64_t tokens, int64_t valid, int E,
                 int k, bool normalize, int32_t* __restrict__ idx, float* __restrict__ weights,
                 float* __restrict__ lse, int32_t* __restrict__ counts,
                 float* __restrict__ losses, float* __restrict__ part, float loss_scale) {
  using L = Lanes<G, NV>;
  using Bits = typename Logit<T>::Bits;
  constexpr bool k16 = sizeof(T) == 2;
  __shared__ float s_prob[kRouteThreads / 64][G * NV];
  __shared__ int s_cnt[kRouteThreads / 64][G * NV];
  __shared__ float s_z[kRouteThreads / 64], s_red[16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, gl = lane % G;
  const int c0 = gl * NV;
  float psum[NV];
  int cnt[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) psum[i] = 0.f, cnt[i] = 0;
  float zsum = 0.f;

  // whole waves stay in the loop, so that the lane exchanges see every lane
  for (int64_t base = (int64_t)blockIdx.x * L::kGroups; base < tokens;
       base += (int64_t)gridDim.x * L::kGroups) {
    const int64_t tok = base + t / G;
    const bool live = tok < valid;
    T raw[NV];
    load_logits<NV>(logits + tok * ldl, c0, E, live, raw);
    float x[NV];
    uint32_t key[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = to_f32(raw[i]);
      key[i] = order_key<Bits, Logit<T>::kInf>(__builtin_bit_cast(Bits, raw[i]));
      if (k16 && key[i]) key[i] = key[i] << 16 | (uint32_t)(0xFFFF - (c0 + i));
    }
    float top = -INFINITY, inv_total = 0.f, row_lse = -INFINITY, wsum = 0.f;
    int rec_idx[L::kSlots];
    float rec_w[L::kSlots];
#pragma unroll
    for (int s = 0; s < L::kSlots; ++s) rec_idx[s] = -1, rec_w[s] = 0.f;
    for (int j = 0; j < k; ++j) {
      uint32_t m = key[0];
#pragma unroll
      for (int i = 1; i < NV; ++i) m = max(m, key[i]);
      const uint32_t gm = lanes_max_u32<G>(m);
      int e;
      float v;
      if constexpr (k16) {
        e = 0xFFFF - (int)(gm & 0xFFFFu);
        v = to_f32(__builtin_bit_cast(T, key_bits((Bits)(gm >> 16))));
      } else {
        // the lowest expert among the lanes that hold the maximum
        uint32_t low = 0u;
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
          if (key[i] == gm) low = (uint32_t)(0xFFFF - (c0 + i));
        e = 0xFFFF - (int)lanes_max_u32<G>(low);
        v = __uint_as_float(key_bits(gm));
      }
      if (gm == 0) e = -1, v = -INFINITY;
      if (j == 0) {
        top = v;
        float total = 0.f, px[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          px[i] = gm == 0 ? 0.f : __builtin_amdgcn_exp2f((x[i] - top) * kLog2e);
          total += px[i];
        }
        total = lanes_sum<G>(total);
        if (gm != 0) {
          inv_total = 1.0f / total;
          row_lse = top + __logf(total);
          if (gl == 0) zsum += row_lse * row_lse;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) psum[i] += px[i] * inv_total;
      }
      const float w = e < 0 ? 0.f : __builtin_amdgcn_exp2f((v - top) * kLog2e);
      wsum += w;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (e == c0 + i) key[i] = 0u, cnt[i] += 1;
#pragma unroll
      for (int s = 0; s < L::kSlots; ++s)
        if (j == s * G + gl) rec_idx[s] = e, rec_w[s] = w;
    }
    if (tok < tokens) {
      const float f = !normalize ? inv_total : wsum == 0.f ? 0.f : 1.0f / wsum;
#pragma unroll
      for (int s = 0; s < L::kSlots; ++s) {
        const int j = s * G + gl;
        if (j < k) {
          idx[tok * k + j] = rec_idx[s];
          weights[tok * k + j] = rec_w[s] * f;
        }
      }
      if (gl == 0) lse[tok] = live ? row_lse : 0.f;
    }
  }

  // the workgroup's sums: over the groups of a wave, then over the waves
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int off = 32; off >= G; off >>= 1) {
      psum[i] += __shfl_xor(psum[i], off, 64);
      cnt[i] += __shfl_xor(cnt[i], off, 64);
    }
    if (lane < G) s_prob[wave][c0 + i] = psum[i], s_cnt[wave][c0 + i] = cnt[i];
  }
  zsum = lanes_sum<64>(zsum);
  if (lane == 0) s_z[wave] = zsum;
  __syncthreads();
  const float z = s_z[0] + s_z[1] + s_z[2] + s_z[3];
  float cp = 0.f;
  for (int e = t; e < E; e += kRouteThreads) {
    const float p = s_prob[0][e] + s_prob[1][e] + s_prob[2][e] + s_prob[3][e];
    const int c = s_cnt[0][e] + s_cnt[1][e] + s_cnt[2][e] + s_cnt[3][e];
    if (gridDim.x == 1) {
      counts[e] = c;
      cp += (float)c * p;
    } else {
      part[(int64_t)blockIdx.x * E + e] = p;
      reinterpret_cast<int32_t*>(part)[((int64_t)gridDim.x + blockIdx.x) * E + e] = c;
    }
  }
  if (gridDim.x == 1) {
    write_losses(s_red, cp, z, loss_scale, valid, losses);
  } else if (t == 0) {
    part[2 * (int64_t)gridDim.x * E + blockIdx.x] = z;
  }
}

// Adds the partial sums of `blocks` workgroups: lanes t, t + E', t + 2 E', ... (E' = E rounded up
// to a power of two) take an expert's blocks in turn, and one of them adds their sums up.
__global__ void __launch_bounds__(1024)
moe_route_losses_kernel(const float* __restrict__ part, int blocks, int E, int width,
                        int32_t* __restrict__ counts, float* __restrict__ losses, int64_t valid,
                        float loss_scale) {
  __shared__ float s_p[1024], s_red[16];
  __shared__ int s_c[1024];
  const int32_t* cpart = reinterpret_cast<const int32_t*>(part) + (int64_t)blocks * E;
  const float* zpart = part + 2 * (int64_t)blocks * E;
  const int t = threadIdx.x, e = t % width, r = t / width, ways = 1024 / width;
  float p = 0.f;
  int c = 0;
  if (e < E)
    for (int b = r; b < blocks; b += ways) {
      p += part[(int64_t)b * E + e];
      c += cpart[(int64_t)b * E + e];
    }
  s_p[t] = p, s_c[t] = c;
  float z = 0.f;
  for (int b = t; b < blocks; b += 1024) z += zpart[b];
  __syncthreads();
  float cp = 0.f;
  if (t < E) {
    p = 0.f, c = 0;
    for (int i = 0; i < ways; ++i) p += s_p[i * width + t], c += s_c[i * width + t];
    counts[t] = c;
    cp = (float)c * p;
  }
  __syncthreads();
  z = lanes_sum<64>(z);
  if ((t & 63) == 0) s_p[t >> 6] = z;
  __syncthreads();
  z = 0.f;
  for (int w = 0; w < 16; ++w) z += s_p[w];
  write_losses(s_red, cp, z, loss_scale, valid, losses);
}

// dl[t, e] = p (A (c[e] - sum_e p c) + B lse - [not normalized] sum_j w dw)
//            + [e = idx[t, j]] w_j (dw_j - [normalized] sum_j w dw)
// with A = dlosses[0] E / (T^2 k) and B = dlosses[1] 2 / T, c the counts.
template <typename T, int G, int NV>
__global__ void __launch_bounds__(kRouteThreads)
moe_route_bwd_kernel(const T* __restrict__ logits, int64_t ldl, int64_t tokens, int64_t valid,
                     int E, int k, bool normalize, const float* __restrict__ lse,
                     const int32_t* __restrict__ idx, const float* __restrict__ weights,
                     const int32_t* __restrict__ counts, const float* __restrict__ dweights,
                     const float* __restrict__ dlosses, float a_scale, float b_scale,
                     T* __restrict__ dlogits) {
  using L = Lanes<G, NV>;
  const int t = threadIdx.x, lane = t & 63, gl = lane % G, c0 = gl * NV;
  const float A = dlosses ? dlosses[0] * a_scale : 0.f;
  const float B = dlosses ? dlosses[1] * b_scale : 0.f;
  float c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) c[i] = c0 + i < E ? (float)counts[c0 + i] : 0.f;
  const int64_t tok = (int64_t)blockIdx.x * L::kGroups + t / G;
  const bool live = tok < valid;
  T x[NV];
  load_logits<NV>(logits + tok * ldl, c0, E, live, x);
  // The softmax is made again from the row itself: exp(l - lse) would lose what lse rounds off,
  // all of log E in a row of the type's lowest values.
  float top = to_f32(x[0]);
  bool any = top > -INFINITY || top != top;
#pragma unroll
  for (int i = 1; i < NV; ++i) {
    const float v = to_f32(x[i]);
    any |= v > -INFINITY || v != v;
    top = __builtin_fmaxf(top, v);
  }
  top = lanes_max<G>(top);
  const bool none = lanes_max_u32<G>(any) == 0u;    // no expert left: p = 0
  const float l = none ? 0.f : lse[tok];
  int rec_idx[L::kSlots];
  float rec_w[L::kSlots], rec_v[L::kSlots], dot = 0.f;
#pragma unroll
  for (int s = 0; s < L::kSlots; ++s) {
    const int j = s * G + gl;
    rec_idx[s] = -1, rec_w[s] = 0.f, rec_v[s] = 0.f;
    if (live && j < k && dweights) {
      const int e = idx[tok * k + j];
      if (e >= 0 && e < E)
        rec_idx[s] = e, rec_w[s] = weights[tok * k + j], rec_v[s] = dweights[tok * k + j];
    }
    dot += rec_w[s] * rec_v[s];
  }
  dot = lanes_sum<G>(dot);
  float p[NV], pc = 0.f, total = 0.f, d[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    p[i] = none ? 0.f : __builtin_amdgcn_exp2f((to_f32(x[i]) - top) * kLog2e);
    pc += p[i] * c[i];
    total += p[i];
  }
  total = lanes_sum<G>(total);
  total = none ? 0.f : 1.0f / total;
  pc = lanes_sum<G>(pc) * total;
#pragma unroll
  for (int i = 0; i < NV; ++i) p[i] *= total;
  const float rest = none ? 0.f : B * l - (normalize ? 0.f : dot);
#pragma unroll
  for (int i = 0; i < NV; ++i) d[i] = p[i] * (A * (c[i] - pc) + rest);
  if (dweights) {
#pragma unroll
    for (int s = 0; s < L::kSlots; ++s) {
      const float g = rec_w[s] * (rec_v[s] - (normalize ? dot : 0.f));
      for (int j = 0; j < G && s * G + j < k; ++j) {
        const int from = (lane & ~(G - 1)) | j;
        const int e = __shfl(rec_idx[s], from, 64);
        const float v = __shfl(g, from, 64);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (e == c0 + i) d[i] += v;
      }
    }
  }
  if (tok >= tokens) return;
  T* out = dlogits + tok * E + c0;
  T o[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] = from_f32<T>(d[i]);
  if (c0 + NV <= E) {
    __builtin_memcpy(out, o, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c0 + i < E) out[i] = o[i];
  }
}

// Lanes of a token and experts of a lane.
template <typename F>
hipError_t by_experts(int E, F f) {
  if (E <= 8) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (E <= 16) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 1>{});
  if (E <= 32) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
  if (E <= 64) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 4>{});
  if (E <= 128) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
  if (E <= 256) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
}

template <typename F> hipError_t by_dtype(int dtype, F f) {
  if (dtype == kBF16) return f(BF16{});
  if (dtype == kF16) return f(F16{});
  return f(0.0f);
}

int group_lanes(int E) { return E <= 8 ? 8 : E <= 64 ? 16 : E <= 128 ? 32 : 64; }

// Workgroups of the forward: one that also writes the losses for few tokens, else up to 256.
constexpr int64_t kRouteMaxBlocks = 256;
int64_t route_blocks(int64_t tokens, int32_t E) {
  const int64_t per = kRouteThreads / group_lanes(E);
  const int64_t steps = (tokens + per - 1) / per;
  if (steps <= 2) return 1;
  return steps < kRouteMaxBlocks ? steps : kRouteMaxBlocks;
}

}  // namespace

int64_t moe_route_workspace(int64_t tokens, int32_t experts) {
  const int64_t blocks = route_blocks(tokens, experts);
  return blocks == 1 ? 0 : blocks * (2 * (int64_t)experts + 1) * 4;
}

hipError_t launch_moe_route(const MoeRouteArgs& a, hipStream_t s) {
  const int64_t blocks = route_blocks(a.tokens, a.experts);
  const double t = (double)(a.valid > 0 ? a.valid : 1);
  const float scale = (float)((double)a.experts / (t * t * a.topk));
  hipError_t e = by_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_experts(a.experts, [&](auto g, auto nv) {
      hipLaunchKernelGGL((moe_route_kernel<T, decltype(g)::value, decltype(nv)::value>),
                         dim3((unsigned)blocks), dim3(kRouteThreads), 0, s,
                         static_cast<const T*>(a.logits), a.ldl, a.tokens, a.valid, a.experts,
                         a.topk, a.normalize, a.idx, a.weights, a.lse, a.counts, a.losses,
                         a.workspace, scale);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess || blocks == 1) return e;
  int width = 1;
  while (width < a.experts) width *= 2;
  hipLaunchKernelGGL(moe_route_losses_kernel, dim3(1), dim3(1024), 0, s, a.workspace, (int)blocks,
                     a.experts, width, a.counts, a.losses, a.valid, scale);
  return hipGetLastError();
}

hipError_t launch_moe_route_bwd(const MoeRouteArgs& a, hipStream_t s) {
  const int64_t per = kRouteThreads / group_lanes(a.experts);
  const int64_t blocks = (a.tokens + per - 1) / per;
  if (blocks == 0) return hipSuccess;
  const double t = (double)(a.valid > 0 ? a.valid : 1);
  const float sa = (float)((double)a.experts / (t * t * a.topk)), sb = (float)(2.0 / t);
  return by_dtype(a.dtype, [&](auto tag) {
    using T = decltype(tag);
    return by_experts(a.experts, [&](auto g, auto nv) {
      hipLaunchKernelGGL((moe_route_bwd_kernel<T, decltype(g)::value, decltype(nv)::value>),
                         dim3((unsigned)blocks), dim3(kRouteThreads), 0, s,
                         static_cast<const T*>(a.logits), a.ldl, a.tokens, a.valid, a.experts,
                         a.topk, a.normalize, a.lse, a.idx, a.weights, a.counts, a.dweights,
                         a.dlosses, sa, sb, static_cast<T*>(a.dlogits));
      return hipGetLastError();
    });
  });
}

}  // namespace fp8lin
