// What the tiled FP8 products share: buffer resources, loads from memory straight into LDS, the LDS
// layout of a 128-byte K stage, and waits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8lin {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_void_ptr;

constexpr int kRsrcWord3 = 0x00020000;     // raw buffer, 32-bit dwords
constexpr uint32_t kOutOfRange = 0x80000000u;

// Buffer resource of a raw byte buffer of `bytes` bytes (reads at or past the end return 0).
__device__ __forceinline__ v4i make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  v4i r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xFFFF);   // stride 0
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = kRsrcWord3;
  return r;
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(lds_void_ptr)p;
}

// XOR swizzle of the 16-byte chunks of a 128-byte LDS row for the 16x16x128 kernels: row r
// stores logical chunk c at physical chunk c ^ row_swizzle(r). A fragment read is a
// ds_read_b128 where lane l takes chunk 2 (l / 16) (+ 1) of row l % 16. gfx950's LDS (64
// banks of 4 bytes, a row pair per 256 bytes) serves such a read in four cycles, one per
// group of 16 lanes; measured with bank-conflict counters, a group is the lanes of one
// half-wave whose bits 2-4 have the same parity ({0-3, 12-15, 20-23, 24-27},
// {4-7, 8-11, 16-19, 28-31}, and those plus 32). This swizzle gives the 16 lanes of each
// group 16 distinct bank quads for both chunks of the fragment (swizzling by (r / 2) % 8,
// right for groups of 16 consecutive lanes, costs a second cycle per read here).
__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 5; }

// 16-byte LDS read at an LDS byte address (a base register plus a constant folds into the
// instruction's offset field)
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(3))) v4u lds_v4u;
__device__ __forceinline__ v4u lds16(uint32_t a) { return *(lds_v4u*)(uintptr_t)a; }

// One 16-byte-per-lane buffer load written straight to LDS at lds + 16 * lane. Issued
// through inline asm so that the compiler does not guard later LDS reads of other
// stages with waits on it; the kernels wait for these loads themselves (vmcnt) before
// the barrier that publishes a stage. Loads complete in order, which keeps every
// compiler-inserted vmcnt wait for ordinary loads correct (at worst stricter).
// The LDS address goes in M0, which the compiler treats as reserved (it warns that the
// clobber may be ignored): no code generated for these kernels reads or writes M0 itself
// (the LDS instructions of gfx950 do not use it), so only these loads set it.
__device__ __forceinline__ void dma16(v4i rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane((int)lds))
               : "memory", "m0");
}

// As dma16, with a wave-uniform byte offset in an SGPR added to the lane's. Callers put
// the whole row offset in the lane's operand (the one the buffer range check is sure to
// test) and only an offset that stays inside a row in the SGPR.
__device__ __forceinline__ void dma16_so(v4i rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(soff), "s"(__builtin_amdgcn_readfirstlane((int)lds))
               : "memory", "m0");
}

// One 4-byte-per-lane buffer load written straight to LDS at lds + 4 * lane.
__device__ __forceinline__ void dma4(v4i rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane((int)lds))
               : "memory", "m0");
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  // this wave's loads older than the newest N have landed
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vm_lgkm() {
  // this wave's loads older than the newest N have landed; its LDS reads are done
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

}  // namespace fp8lin
