// Stages of a product in LDS: loads straight into it, the order of their
// chunks, and what keeps reads and writes of it apart.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// Global -> LDS DMA: lane l's bytes land at lds + 16 l (4 l).  Inline asm, so
// that the compiler does not take the LDS write as pending before every later
// LDS read; ordered by s_waitcnt vmcnt and the stage's barrier.  There are no
// register results, and the address operands are read at issue.  The LDS base
// comes from M0, which has to be written a wait state before (s_nop; the
// compiler does not look inside the asm).
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}

// s_barrier that no memory access moves across (the builtin alone does not
// keep LDS reads behind it).
__device__ __forceinline__ void all_waves() { asm volatile("s_barrier" ::: "memory"); }

// Depends on r % 32 alone, so that a fragment's LDS address is one per-lane
// offset for each step plus a constant for its 32-row block.
__device__ __forceinline__ int swizzle(int r) { return (r ^ ((r & 31) >> 3)) & 7; }

// The same value, which the compiler takes as new: what is computed from it
// once a tile stays there, instead of waiting in registers through the tiles.
__device__ __forceinline__ int renewed(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Orders a wave's own LDS writes before its reads of other lanes' values.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace nvfp4
