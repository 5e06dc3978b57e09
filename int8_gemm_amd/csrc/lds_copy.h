// Global -> LDS copies and the waits of a copy ring, shared by the GEMM kernels.
#pragma once

#include "common.h"

namespace convrot {

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// s_waitcnt on vmcnt only (expcnt, lgkmcnt left unconstrained); gfx9 encoding
template <int V>
__device__ __forceinline__ void wait_vmcnt() {
  static_assert(V >= 0 && V < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((V & 0xF) | (0x7 << 4) | (0xF << 8) | ((V >> 4) << 14));
}

// One 16-byte-per-lane global -> LDS copy (global_load_lds_dwordx4, SGPR base
// + 32-bit VGPR offset): lane i writes LDS bytes [lds_base + 16 i, +16).
// Written as inline asm so that the compiler's waitcnt model (which treats the
// LDS write of the builtin form as pending LDS traffic and drains it around
// every later LDS read) stays out of the way; completion is tracked by the
// explicit vmcnt waits of the K-loop. The instruction has no VGPR result.
// The compiler fills no wait states inside the block. Two are asked for: one
// between a scalar write of M0 and a copy to LDS, and five between a vector
// instruction that writes an SGPR (v_readfirstlane of the base) and a memory
// access that reads it. The scalar copy of the base is the one, and needs none
// itself, so the access reads an SGPR that no vector instruction wrote.
__device__ __forceinline__ void dma16(const int8_t* sbase, uint32_t voff, uint32_t lds_base) {
  const int8_t* base;
  asm volatile("s_mov_b32 m0, %3\n\ts_mov_b64 %0, %2\n\tglobal_load_lds_dwordx4 %1, %0"
               : "=&s"(base)
               : "v"(voff), "s"(sbase), "s"(lds_base)
               : "memory", "m0");
}

// s_waitcnt lgkmcnt(0) only (vmcnt, expcnt left unconstrained)
__device__ __forceinline__ void wait_lgkm0() {
  __builtin_amdgcn_s_waitcnt(0xF | (0x7 << 4) | (0x0 << 8) | (0x3 << 14));
}

// Workgroup barrier without the release/acquire fences of __syncthreads():
// those would force vmcnt(0) and drain the in-flight LDS-DMA stages. The
// empty asm statements keep the compiler from moving memory accesses across.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace convrot
