// Loads that write LDS directly and the waits that belong to them, shared by the
// matrix products (hc_gemm.hip) and the attention kernels.
#pragma once

#include "hc_device.h"

namespace hc {

constexpr uint32_t OUTSIDE = 0x80000000u;  // an offset past every descriptor's end: loads give zeros, stores nothing

__device__ __forceinline__ u32x4 raw_desc(const void* base) {
  const uint64_t b = (uint64_t)base;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32)), 0x7FFFFFF0u, 0x00020000u};
}
// The same with an end: what lies at `bytes` or behind reads as zeros.
__device__ __forceinline__ u32x4 raw_desc(const void* base, uint32_t bytes) {
  u32x4 d = raw_desc(base);
  d[2] = (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes);
  return d;
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) { return (uint32_t)(uintptr_t)(const lds_u8*)p; }
// Lane l: W bytes (16 or 4) from offset off of the descriptor to LDS byte dst + W l (dst
// the same in every lane). Written out because the compiler, which cannot tell the stage
// being filled from the one being read, would wait for the load before every LDS read. m0 is a
// register of the compiler's own (it warns of any asm that writes it): named as written, so that
// no value that the compiler put there itself is taken to have survived.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int W, bool STREAM> __device__ __forceinline__ void lds_load(u32x4 desc, uint32_t off, uint32_t dst) {
  static_assert(W == 16 || W == 4, "width");
  if constexpr (W == 4 && STREAM)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen nt lds"
                 : : "s"(dst), "v"(off), "s"(desc) : "memory", "m0");
  else if constexpr (W == 4)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 : : "s"(dst), "v"(off), "s"(desc) : "memory", "m0");
  else if constexpr (STREAM)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds"
                 : : "s"(dst), "v"(off), "s"(desc) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 : : "s"(dst), "v"(off), "s"(desc) : "memory", "m0");
}
// The same, 16 bytes from an address of each lane's own.
__device__ __forceinline__ void lds_load_from(const void* p, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(dst), "v"(p) : "memory", "m0");
}
#pragma clang diagnostic pop

// What lanes load that have nothing to load: 16 bytes of zeros.
static __device__ __attribute__((aligned(16))) const uint32_t zeros16[4] = {0u, 0u, 0u, 0u};

// Waits until at most N of this wave's loads are in flight (they complete in order).
template <int N> __device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Workgroup barrier once this wave's LDS operations are done; its global loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace hc
