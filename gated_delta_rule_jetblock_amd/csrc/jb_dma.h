// jb_dma.h -- buffer -> LDS transfers that the compiler does not track, and the
// wait that orders them (projection and attention kernels).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace jb {

// s_waitcnt with only the vector-memory count constrained (gfx9 encoding)
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// A raw buffer descriptor over [base, base + bytes): reads past the range
// return zero.  Wave-uniform by construction; readfirstlane says so to the
// register allocator, which then keeps it in scalar registers.
typedef int v4i_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4i_t buf_desc(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return v4i_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
               __builtin_amdgcn_readfirstlane((int)(uint32_t)((b >> 32) & 0xffff)),
               __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}

// Buffer -> LDS load of 16 bytes per lane: the piece at byte voff + soff of the
// buffer lands at LDS byte lds + 16 lane.  Written out so that the compiler
// does not track it: it would otherwise wait for every such load in flight
// before each LDS read of the K loop.  The loop's own s_waitcnt on the
// vector-memory count and its barriers order the slices.  The load has no
// register result, only the LDS bytes it writes; M0 (the LDS base, read when
// the load issues) is restored afterwards.
// The leading s_nop covers a vector-ALU write (readfirstlane) of the
// descriptor or offsets just before, which the compiler cannot see here.
__device__ __forceinline__ void dma16(v4i_t desc, int voff, int soff, uint32_t lds) {
  uint32_t saved;
  asm volatile(
      "s_nop 4\n\ts_mov_b32 %0, m0\n\ts_mov_b32 m0, %4\n\ts_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds\n\ts_mov_b32 m0, %0"
      : "=&s"(saved)
      : "v"(voff), "s"(desc), "s"(soff), "s"(lds)
      : "memory");
}

}  // namespace jb
