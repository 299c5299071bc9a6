// Shared memory and wait helpers of the matrix kernels (gfx950, wave64).
#pragma once
#include "common.h"

namespace muon {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
// ds_read_b64_tr_b16: within each 16-lane group, lane i receives element
// i % 4 of the 4-element reads of lanes i / 4 + 4 q, q = 0..3 (measured).
// With lane s reading row k0 + s / 4 at columns c0 + 4 (s % 4) .. + 3, lane i
// gets column c0 + i at rows k0 .. k0 + 3: a transposed 4 x 16 block.
__device__ __forceinline__ bf16x4 lds_read_tr16(const bf16_t* p) {
  typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(__attribute__((address_space(3))) bf16_t*)p);
}

// The same at an LDS byte address.
__device__ __forceinline__ bf16x4 lds_read_tr16_at(uint32_t at) {
  typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16(reinterpret_cast<lds_bf16x4*>((uintptr_t)at));
}

// A wave-uniform 64-bit value moved to scalar registers (the compiler
// computes uniform divisions in vector registers; these stay live across a
// tile's main loop).
__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint64_t u = (uint64_t)v;
  // readfirstlane returns int: each half goes through uint32_t (no sign extension)
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u) |
                   ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32));
}
template <typename T> __device__ __forceinline__ T* uniform_ptr(T* p) {
  return reinterpret_cast<T*>((uintptr_t)uniform64((int64_t)(uintptr_t)p));
}

// Waits (on this wave's counter) until at most n vector-memory operations
// are outstanding.
__device__ __forceinline__ constexpr int vmcnt_imm(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }

// 16 bytes per lane from global memory (uniform base + per-lane 32-bit byte
// offset) straight into LDS at lds_addr + 16 lane.  Written as asm: the
// compiler neither waits on it nor recycles its address registers early
// (either would serialise the prefetch); the caller waits with vmcnt before
// the data is read.
// M0 is written here and nowhere else in these kernels (the generated code
// holds no other use of it), so clobbering the reserved register is safe.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_dma16(const void* base, uint32_t voff, uint32_t lds_addr) {
  // base and lds_addr are wave-uniform; make that visible to the compiler
  const uint64_t b = (uint64_t)(uintptr_t)base;
  // (readfirstlane returns int: go through uint32_t so the low half is not
  // sign-extended into the high half)
  const uint64_t sb = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)b) |
                      ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) << 32);
  const uint32_t sl = __builtin_amdgcn_readfirstlane(lds_addr);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(voff), "s"(sb), "s"(sl) : "memory", "m0");
}
// The same from a buffer of `bytes` bytes: lanes whose offset lies past its end read nothing (and what arrives
// for them is of no use).  The scalar offset is 0, so that the lane's offset alone is compared with the size.
__device__ __forceinline__ u32x4 buffer_of(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)uniform64((int64_t)(uintptr_t)base);
  return u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, (uint32_t)__builtin_amdgcn_readfirstlane(bytes), 0x00020000u};
}
// A buffer that begins `bytes` bytes later and ends where it did.
__device__ __forceinline__ void advance(u32x4& buffer, uint32_t bytes) {
  const uint64_t b = ((uint64_t)buffer[1] << 32 | buffer[0]) + bytes;
  buffer[0] = (uint32_t)b;
  buffer[1] = (uint32_t)(b >> 32);
  buffer[2] -= bytes;
}
__device__ __forceinline__ void lds_dma16(const u32x4& buffer, uint32_t voff, uint32_t lds_addr) {
  const uint32_t sl = __builtin_amdgcn_readfirstlane(lds_addr);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(voff), "s"(buffer), "s"(sl) : "memory", "m0");
}
// 4 bytes per lane, to lds_addr + 4 lane.
__device__ __forceinline__ void lds_dma4(const u32x4& buffer, uint32_t voff, uint32_t lds_addr) {
  const uint32_t sl = __builtin_amdgcn_readfirstlane(lds_addr);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :: "v"(voff), "s"(buffer), "s"(sl) : "memory", "m0");
}
#pragma clang diagnostic pop

// Workgroup barrier without the release/acquire fences of __syncthreads,
// which would also wait for every outstanding global store and LDS-DMA load;
// the caller waits for what it needs.  This wave's LDS accesses complete
// first, and the compiler moves no memory access across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Registers a and b against lane bit 3 (4): afterwards a holds what lanes with the bit clear had in both, in
// the lanes that had it and in their partners, and b what the others had.
__device__ __forceinline__ void swap_lanes8(u32x4& a, u32x4& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int x = (int)a[i], y = (int)b[i];
    a[i] = (uint32_t)__builtin_amdgcn_update_dpp(x, y, 0x128, 0xf, 0xc, false);   // lanes 8-15 of 16 from 8 below
    b[i] = (uint32_t)__builtin_amdgcn_update_dpp(y, x, 0x128, 0xf, 0x3, false);
  }
}
__device__ __forceinline__ void swap_lanes16(u32x4& a, u32x4& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const auto v = __builtin_amdgcn_permlane16_swap(a[i], b[i], false, false);
    a[i] = v[0];
    b[i] = v[1];
  }
}

}  // namespace muon
