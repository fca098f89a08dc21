// Reads and loads of LDS that the kernels address by hand.
#pragma once

#include "paged_device.hpp"

namespace rrt {

using i16x4 = short __attribute__((ext_vector_type(4)));
using lds_i16x4 = __attribute__((address_space(3))) i16x4;
using lds_u32x4 = __attribute__((address_space(3))) u32x4;
using lds_u32x2 = __attribute__((address_space(3))) u32x2;
using lds_i32 = __attribute__((address_space(3))) int32_t;

__device__ __forceinline__ uint32_t lds_at(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)p;
}
__device__ __forceinline__ u32x4 lds_read16(uint32_t at) { return *(lds_u32x4*)at; }
// Four 16-bit values of one column from four rows: lane i of a group of 16
// gives the address of 4 columns of row i / 4 and gets column i.
__device__ __forceinline__ u32x2 lds_read_tr(uint32_t at) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)at));
}

// Loads straight to LDS: 16 (4) bytes from each active lane's address to `to`
// (wave uniform) + 16 (4) x lane.  No register is written, so nothing but
// wait_loads() below waits for them; as instructions that the compiler knows
// to write LDS, they made it wait for all of them before every transposed read.
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds(const char* from, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(offset), "s"(from) : "memory", "m0");
}
__device__ __forceinline__ void load4_to_lds(const int32_t* from, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(__builtin_amdgcn_readfirstlane(to)), "v"(from) : "memory", "m0");
}
// Waits until all but the last N loads have arrived.
template <int N = 0>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

}  // namespace rrt
