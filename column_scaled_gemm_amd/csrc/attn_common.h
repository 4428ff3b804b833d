// Shared by the attention kernels (gfx950).
#pragma once
#include "kv_common.h"

namespace fp8sm {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// The running maximum is moved only when a row's scores exceed it by more than
// kSlack (p <= 2^kSlack then), so most steps do not rescale the accumulator.
constexpr float kSlack = 8.0f;
// Where P is rounded to fp16 it is taken 2^kLift times as large: p <= 2^(kSlack +
// kLift) = 2^15, which fp16 holds, and its fixed step below 2^-14 lies at 2^-31 of the
// row's largest p.  Without the lift it is 2^-24, and a tail 16 nats below a token of
// small value is off by 6%, one of 18 nats lost.
constexpr float kLift = 7.0f, kUnlift = 1.0f / 128;
// Up to here m scale rounds by at most 2^-4 and serves as the exponents' reference in one
// fma; beyond, scores are subtracted first.
constexpr float kFarScore = 1 << 20;
constexpr float kLn2 = 0.6931471805599453f;

template <bool F16>
__device__ __forceinline__ uint16_t round16(float v) {
  if constexpr (F16)
    return __builtin_bit_cast(uint16_t, (_Float16)v);
  else
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Grids are one list of workgroups; more than a grid's first dimension takes
// go on in its second.
constexpr uint32_t kGridX = 1 << 16;
__device__ __forceinline__ int64_t workgroup_id() { return blockIdx.x + (int64_t)blockIdx.y * kGridX; }
inline dim3 grid_of(int64_t n) {
  return n <= kGridX ? dim3((uint32_t)n) : dim3(kGridX, (uint32_t)((n + kGridX - 1) / kGridX));
}

// max of a value over the two half-wavefronts
__device__ __forceinline__ float half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

}  // namespace fp8sm
