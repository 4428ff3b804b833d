// Shared by the key/value cache kernels and the attention over it (gfx950).
#pragma once
#include "device_common.h"
#include "launch.h"

namespace fp8sm {

// One sequence of a ragged batch: its rows c0 .. c0 + n - 1 of the token
// arrays, and its cached length with those n tokens as the last ones.
struct Seq {
  int c0, n, len;
};

// The device arrays are data, not checked by the host: whatever they hold, the
// rows lie in [0, T) and the length within the block table's reach.  b is
// wavefront-uniform, and so is the result, in scalar registers: what is decided
// from it is a scalar branch.
__device__ __forceinline__ Seq load_seq(const KvBatch& kb, int b, int block_shift) {
  Seq s;
  const int T = kb.T;
  s.c0 = min(max(__builtin_amdgcn_readfirstlane(kb.cu[b]), 0), T);
  s.n = min(max(__builtin_amdgcn_readfirstlane(kb.cu[b + 1]), s.c0), T) - s.c0;
  s.len = min(max(__builtin_amdgcn_readfirstlane(kb.lens[b]), 0), kb.max_blocks << block_shift);
  return s;
}

// Work slots of a ragged batch without a plan made on the host: sequence b's
// slots start at f(b) = floor(cu[b] * mul / 2^shift) + add * b, which leaves
// room for n * mul / 2^shift + add of them.  Returns the sequence that owns
// slot u (the last b with f(b) <= u) and f(b).  Every lane of the wavefront
// takes part: one round of 64 probes for up to 64 sequences, two for 4096.
__device__ __forceinline__ int find_seq(const KvBatch& kb, int64_t u, int mul, int shift, int add,
                                        int64_t* first) {
  const int lane = threadIdx.x & 63;
  const int T = kb.T, B = kb.B;
  int lo = 0, span = B;
  int64_t f0 = 0;
  while (true) {
    const int step = (span + 63) >> 6;
    const int b = lo + lane * step;
    int64_t f = INT64_MAX;
    if (lane * step < span) {
      const int c = min(max(kb.cu[b], 0), T);
      f = (((int64_t)c * mul) >> shift) + (int64_t)add * b;
    }
    const uint64_t m = __ballot(f <= u);
    const int k = max(0, 63 - (int)__clzll((long long)(m | 1)));
    f0 = __shfl(f, k, 64);
    lo += k * step;
    span = min(step, span - k * step);
    if (step == 1) break;
  }
  *first = (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(f0 >> 32)) << 32) |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)f0));
  return __builtin_amdgcn_readfirstlane(lo);
}

// 2^(e - 127) of a biased exponent byte (0: 2^-127, 255: 2^128 overflows to inf
// only in the product).
__device__ __forceinline__ float exp_byte_value(int e) {
  return e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)e << 23);
}

}  // namespace fp8sm
