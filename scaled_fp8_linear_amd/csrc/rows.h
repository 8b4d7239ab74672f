// Element types and 16-byte row pieces, shared by the kernels that work on rows of bf16,
// f16 or f32 (layer norm, expert dispatch and combine). A piece may start at any element:
// gfx950's global loads and stores take 16 bytes at any byte address, so rows of odd widths
// and strides use the same instructions as aligned ones (and touch one line more).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "common.h"

namespace fp8lin {

enum DType { kBF16 = 0, kF16 = 1, kF32 = 2 };

struct BF16 { uint16_t u; };
struct F16 { uint16_t u; };

typedef unsigned piece_t __attribute__((ext_vector_type(4)));
typedef unsigned piece_any_t __attribute__((ext_vector_type(4), aligned(2)));

typedef unsigned half_piece_any_t __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned dword_any_t __attribute__((aligned(2)));

// Cached pieces, or streaming ones (non-temporal: passed through the caches rather than kept
// there). Which is faster for a tensor that is read or written once depends on the mix of reads
// and writes around it, so each kernel states what it uses and what it measured.
enum Cache { kKeep = 0, kStream = 1 };

template <Cache C>
__device__ __forceinline__ piece_t ld_piece(const void* p) {
  const piece_any_t* q = reinterpret_cast<const piece_any_t*>(p);
  if constexpr (C == kStream) return __builtin_nontemporal_load(q);
  else return *q;
}
template <Cache C>
__device__ __forceinline__ void st_piece(void* p, piece_t v) {
  piece_any_t* q = reinterpret_cast<piece_any_t*>(p);
  if constexpr (C == kStream) __builtin_nontemporal_store((piece_any_t)v, q);
  else *q = v;
}

// row + c for a column 0 <= c < 2^30. Where `row` is the same for a whole wave this is a
// scalar base and a 32-bit lane offset, which the load and store instructions add up.
template <typename T>
__device__ __forceinline__ T* elem_at(T* row, int c) {
  using Byte = std::conditional_t<std::is_const<T>::value, const char, char>;
  uint32_t off = (uint32_t)c * (uint32_t)sizeof(T);
  asm volatile("" : "+v"(off));      // else loops keep the offset widened to 64 bits
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(row) + off);
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

// The piece at column c of a row of `cols` elements, in two steps, so that a kernel can have
// several loads in flight: ld_raw issues one 16-byte load (of the row's last 16 bytes where
// the piece is cut off by the row's end or lies past it), and cut moves a cut-off piece's
// elements down and sets what is past the row to 0, or with FILL kOwn to elements of the row
// (any of them; ld_raw has to be told too). Nothing outside the row is touched; rows shorter
// than a piece (kShort: they may be) are read element by element.
enum Fill { kZero = 0, kOwn = 1 };
template <Cache C, bool kShort = true, Fill FILL = kZero, typename T>
__device__ __forceinline__ piece_t ld_raw(const T* row, int c, int cols) {
  constexpr int N = Piece<T>::N;
  if (!kShort || cols >= N) return ld_piece<C>(elem_at(row, c + N <= cols ? c : cols - N));
  piece_t v = {0u, 0u, 0u, 0u};
  if (c == 0 || FILL == kOwn) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i >= cols && FILL == kZero) continue;
      const T* e = row + (i < cols ? i : 0);
      if constexpr (sizeof(T) == 4) v[i] = __builtin_bit_cast(uint32_t, *e);
      else v[i / 2] |= (uint32_t)e->u << (16 * (i & 1));
    }
  }
  return v;
}
template <typename T, Fill FILL = kZero>
__device__ __forceinline__ piece_t cut(piece_t v, int c, int cols) {
  constexpr int N = Piece<T>::N;
  constexpr bool own = FILL == kOwn;
  if (c + N <= cols || cols < N) return v;
  const int past = (c + N - cols) * (int)sizeof(T);        // bytes past the row's end
  if (past >= 16) return own ? v : piece_t{0u, 0u, 0u, 0u};
  if (past & 8) v = piece_t{v[2], v[3], own ? v[0] : 0u, own ? v[1] : 0u};
  if (past & 4) v = piece_t{v[1], v[2], v[3], own ? v[0] : 0u};
  if constexpr (sizeof(T) == 2) {
    if (past & 2)
      v = piece_t{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16,
                  v[3] >> 16 | (own ? v[0] << 16 : 0u)};
  }
  return v;
}
template <typename T>
__device__ __forceinline__ piece_t ld_row(const T* row, int c, int cols) {
  return cut<T>(ld_raw<kKeep>(row, c, cols), c, cols);
}
template <Cache C, typename T>
__device__ __forceinline__ void st_row(T* row, int c, int cols, piece_t v) {
  constexpr int N = Piece<T>::N;
  T* p = elem_at(row, c);
  if (c + N <= cols) {
    st_piece<C>(p, v);
  } else if (c < cols) {                     // 8, 4 and 2 bytes of what is left
    const int left = (cols - c) * (int)sizeof(T);
    if (left & 8) {
      *reinterpret_cast<half_piece_any_t*>(p) = half_piece_any_t{v[0], v[1]};
      v[0] = v[2], v[1] = v[3];
      p = elem_at(p, 8 / (int)sizeof(T));
    }
    if (left & 4) {
      *reinterpret_cast<dword_any_t*>(p) = v[0];
      v[0] = v[1];
      p = elem_at(p, 4 / (int)sizeof(T));
    }
    if constexpr (sizeof(T) == 2)
      if (left & 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)v[0];
  }
}

// Loads into v have arrived here. Placed before a row's stores, it keeps the wait for a
// prefetched row from also waiting for those stores (both count down one counter).
__device__ __forceinline__ void arrived(piece_t& v) { asm volatile("" : "+v"(v)); }

// Sum over groups of LANES consecutive lanes (a power of two, at most 64): every lane gets
// the same value, added in the same order on every run. Lanes are paired by DPP within 16 and
// by the row swaps beyond, which need neither LDS nor index registers.
template <int CTRL> __device__ __forceinline__ float dpp(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int LANES, int FROM = 1>      // FROM: lanes already summed
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (LANES >= 2 && FROM < 2) v += dpp<0xB1>(v);        // quad_perm 1,0,3,2
  if constexpr (LANES >= 4 && FROM < 4) v += dpp<0x4E>(v);        // quad_perm 2,3,0,1
  if constexpr (LANES >= 8 && FROM < 8) v += dpp<0x141>(v);       // mirror of each 8 lanes
  if constexpr (LANES >= 16 && FROM < 16) v += dpp<0x140>(v);     // mirror of each 16 lanes
  if constexpr (LANES >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (LANES >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return v;
}

}  // namespace fp8lin
