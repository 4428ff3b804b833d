// Copies from memory straight into LDS, 16 bytes a lane, for the LDS rings of the int8
// product and the packed attention (gfx950).  Inline asm, so that the compiler does not wait for every
// copy before each LDS read; wait_copies_but waits for what is needed.  lds is the
// wave-uniform LDS byte address of lane 0's destination, lane i writes lds + 16 i.
// m0 is used for nothing else in these kernels; a copy that follows its write
// needs one wait state, which inside inline asm nobody else puts in.
#pragma once
#include "device_common.h"

namespace fp8sm {

typedef int i32x4 __attribute__((ext_vector_type(4)));

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// from a raw buffer: base of rsrc + voff (a lane's) + soff
__device__ __forceinline__ void lds_copy16_buf(uint32_t voff, i32x4 rsrc, int soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Raw buffer descriptor that starts at base (wave-uniform); byte offsets below
// `bytes` are in range, loads beyond it give zeros.  Last word: 32-bit data format,
// no swizzle, no per-lane index.
__device__ __forceinline__ i32x4 raw_buffer(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)b);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}

// Waits until at most N of the wavefront's copies (and loads) are on their way.
template <int N>
__device__ __forceinline__ void wait_copies_but() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)((__attribute__((address_space(3))) const uint8_t*)p);
}

}  // namespace fp8sm
