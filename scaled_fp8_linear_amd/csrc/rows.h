// Element types and 16-byte row pieces, shared by the kernels that work on rows of bf16,
// f16 or f32 (layer norm, expert dispatch and combine). A piece may start at any element:
// gfx950's global loads and stores take 16 bytes at any byte address, so rows of odd widths
// and strides use the same instructions as aligned ones (and touch one line more).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace fp8lin {

enum DType { kBF16 = 0, kF16 = 1, kF32 = 2 };

struct BF16 { uint16_t u; };
struct F16 { uint16_t u; };

typedef unsigned piece_t __attribute__((ext_vector_type(4)));
typedef unsigned piece_any_t __attribute__((ext_vector_type(4), aligned(2)));

__device__ __forceinline__ piece_t ld_piece(const void* p) {
  return *reinterpret_cast<const piece_any_t*>(p);
}
__device__ __forceinline__ void st_piece(void* p, piece_t v) {
  *reinterpret_cast<piece_any_t*>(p) = v;
}

typedef _Float16 fp8lin_f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float to_f32(BF16 v) { return __uint_as_float((uint32_t)v.u << 16); }
__device__ __forceinline__ float to_f32(F16 v) {
  return (float)__builtin_bit_cast(_Float16, v.u);
}
__device__ __forceinline__ float to_f32(float v) { return v; }

// One rounding to nearest even; NaN stays NaN, f16 overflows to infinity.
template <typename T> __device__ __forceinline__ T from_f32(float f);
template <> __device__ __forceinline__ BF16 from_f32<BF16>(float f) {
  return BF16{__builtin_bit_cast(uint16_t, (__bf16)f)};
}
template <> __device__ __forceinline__ F16 from_f32<F16>(float f) {
  return F16{__builtin_bit_cast(uint16_t, (_Float16)f)};
}
template <> __device__ __forceinline__ float from_f32<float>(float f) { return f; }

// Elements of a 16-byte piece.
template <typename T> struct Piece { static constexpr int N = 16 / (int)sizeof(T); };

__device__ __forceinline__ void unpack(piece_t v, float (&f)[8], BF16) {
#pragma unroll
  for (int i = 0; i < 4; ++i) { f[2 * i] = bf16_lo(v[i]); f[2 * i + 1] = bf16_hi(v[i]); }
}
__device__ __forceinline__ void unpack(piece_t v, float (&f)[8], F16) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t d = v[i];                 // a bit cast of the element itself reads v[0]
    const fp8lin_f16x2 h = __builtin_bit_cast(fp8lin_f16x2, d);
    f[2 * i] = (float)h[0];
    f[2 * i + 1] = (float)h[1];
  }
}
__device__ __forceinline__ void unpack(piece_t v, float (&f)[4], float) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
}

__device__ __forceinline__ piece_t pack(const float (&f)[8], BF16) {
  piece_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  return v;
}
__device__ __forceinline__ piece_t pack(const float (&f)[8], F16) {
  piece_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const fp8lin_f16x2 h = {(_Float16)f[2 * i], (_Float16)f[2 * i + 1]};
    v[i] = __builtin_bit_cast(uint32_t, h);
  }
  return v;
}
__device__ __forceinline__ piece_t pack(const float (&f)[4], float) {
  piece_t v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
  return v;
}

// The piece at column c of a row of `cols` elements: whole, cut off at the row's end (the
// missing elements read as 0), or empty. Nothing past the row is touched.
template <typename T>
__device__ __forceinline__ piece_t ld_row(const T* row, int c, int cols) {
  constexpr int N = Piece<T>::N;
  if (c + N <= cols) return ld_piece(row + c);
  piece_t v = {0u, 0u, 0u, 0u};
  if (c < cols) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < cols) v[i] = __builtin_bit_cast(uint32_t, row[c + i]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < cols) v[i / 2] |= (uint32_t)row[c + i].u << (16 * (i & 1));
    }
  }
  return v;
}
template <typename T>
__device__ __forceinline__ void st_row(T* row, int c, int cols, piece_t v) {
  constexpr int N = Piece<T>::N;
  if (c + N <= cols) {
    st_piece(row + c, v);
  } else if (c < cols) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < cols) reinterpret_cast<uint32_t*>(row)[c + i] = v[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c + i < cols) row[c + i].u = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
  }
}

// Sum over groups of LANES consecutive lanes (a power of two, at most 64): every lane gets
// the same value, added in the same order on every run.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

}  // namespace fp8lin
