// direct_load.h -- global memory straight into LDS (gfx950), and waits for it.
#pragma once

#include "device_common.h"

namespace moe {

// One wave-wide direct global->LDS load: lane i's 16 bytes at base + voff land
// at LDS byte address lds_addr + 16*i (gfx950 global_load_lds_dwordx4; the LDS
// address comes from M0).  The wait for it is explicit (s_waitcnt vmcnt), as
// the compiler does not track this load.  M0 is declared clobbered: the
// compiler sets M0 right before each of its own uses.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(uint32_t lds_addr, const void* base, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds_addr), "v"(voff), "s"(base)
               : "memory", "m0");
}
// Same with 4 bytes per lane (global_load_lds_dword): lane i's word lands at
// lds_addr + 4*i.
__device__ __forceinline__ void dma4(uint32_t lds_addr, const void* base, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2"
               :
               : "s"(lds_addr), "v"(voff), "s"(base)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Wait until at most n slices of PER direct loads each are outstanding (n <= N; vmcnt
// takes an immediate, so each count has its own instruction).  LGKM: also drain LDS reads.
template <int PER, int N, bool LGKM>
__device__ __forceinline__ void wait_slices(int n) {
  if constexpr (N == 0) {
    if constexpr (LGKM)
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  } else {
    if (n >= N) {
      if constexpr (LGKM)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N * PER) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N * PER) : "memory");
    } else {
      wait_slices<PER, N - 1, LGKM>(n);
    }
  }
}

__device__ __forceinline__ uint32_t uniform_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_readfirstlane(v);
}

__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  // readfirstlane yields a signed int: widen through uint32_t so the low half is
  // zero-extended (a sign-extended low half would corrupt the upper address bits)
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t*>(lo | (hi << 32));
}

}  // namespace moe
