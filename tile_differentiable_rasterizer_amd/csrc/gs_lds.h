// gs_lds.h -- loads from memory straight to LDS, gfx950.  Internal to libgsraster.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gs {

// Sixteen bytes of zeros for the lanes of a load that have nothing to read.
__device__ const uint32_t kZeros[4] __attribute__((aligned(16))) = {0, 0, 0, 0};

// Loads straight to LDS, 16 (or 4) bytes a lane, in a row from `to` (the same for the wavefront).
// They are written as assembly because the compiler orders every LDS read behind the builtin's
// loads, wherever they go, and so would wait for the next tile before it works on this one.  They
// write no register.  Whoever reads what they bring waits first: wait_loads(), then the barrier.
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p);
}
__device__ __forceinline__ void load_to_lds16(const void* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(offset), "s"(base), "s"(to)
               : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds16(const void* p, uint32_t to) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(p), "s"(to) : "memory", "m0");
}
__device__ __forceinline__ void load_to_lds4(const void* base, uint32_t offset, uint32_t to) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :
               : "v"(offset), "s"(base), "s"(to)
               : "memory", "m0");
}
// Waits for the wavefront's own loads to LDS (and every other load).
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }

}  // namespace gs
