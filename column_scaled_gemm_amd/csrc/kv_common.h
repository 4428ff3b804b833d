// Shared by the key/value cache kernels and the attention over it (gfx950).
#pragma once
#include "device_common.h"
#include "launch.h"

namespace fp8sm {

// One sequence of a ragged batch: its rows c0 .. c0 + n - 1 of the token
// arrays, its cached length with those n tokens as the last ones, and the first
// of its work slots.  All wavefront-uniform, in scalar registers.
struct Seq {
  int b, c0, n, len;
  int64_t first;
};

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32) |
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// Work slots of a ragged batch without a plan made on the host: sequence b's
// slots start at f(b) = floor(cu[b] * mul / 2^shift) + add * b, which leaves
// room for n * mul / 2^shift + add of them.  Returns the sequence that owns
// slot u (the last b with f(b) <= u), or sequence 0 with u < first where rows before
// the first sequence leave slots that nobody owns.  Every lane of the wavefront takes part:
// one round of 64 probes for up to 64 sequences, two for 4096; the last round
// brings the sequence's other numbers along.
// The device arrays are data, not checked by the host: whatever they hold, the
// rows lie in [0, T) and the length within the block table's reach.
__device__ __forceinline__ Seq find_seq(const KvBatch& kb, int block_shift, int64_t u, int mul, int shift,
                                        int add) {
  const int lane = threadIdx.x & 63;
  const int T = kb.T, B = kb.B;
  int lo = 0, span = B;
  while (true) {
    const int step = (span + 63) >> 6;
    const int b = lo + lane * step;
    int64_t f = INT64_MAX;
    int c = 0, next = 0, len = 0;
    if (lane * step < span) {
      c = kb.cu[b];
      if (step == 1) {
        next = kb.cu[b + 1];
        len = kb.lens[b];
      }
      c = min(max(c, 0), T);
      f = (((int64_t)c * mul) >> shift) + (int64_t)add * b;
    }
    const uint64_t m = __ballot(f <= u);
    const int k = max(0, 63 - (int)__clzll((long long)(m | 1)));
    lo += k * step;
    if (step > 1) {
      span = min(step, span - k * step);
      continue;
    }
    Seq s;
    s.b = __builtin_amdgcn_readfirstlane(lo);
    s.c0 = __builtin_amdgcn_readlane(c, k);
    s.n = min(max(__builtin_amdgcn_readlane(next, k), s.c0), T) - s.c0;
    s.len = min(max(__builtin_amdgcn_readlane(len, k), 0), kb.max_blocks << block_shift);
    s.first = uniform64((((int64_t)s.c0 * mul) >> shift) + (int64_t)add * s.b);
    return s;
  }
}

// 2^(e - 127) of a biased exponent byte (0: 2^-127, 255: 2^128 overflows to inf
// only in the product).
__device__ __forceinline__ float exp_byte_value(int e) {
  return e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)e << 23);
}

}  // namespace fp8sm
