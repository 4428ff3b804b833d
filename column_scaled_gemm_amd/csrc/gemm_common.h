// Shared by the scaled GEMM kernels (gfx950): the epilogue, the walk over the
// output tiles, and the launchers' choice of the epilogue.
#pragma once
#include "device_common.h"
#include "launch.h"

#include <type_traits>

namespace fp8sm {

typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ uint16_t f32_to_bf16_rne(float f) {
  uint32_t u = __float_as_uint(f);
  u += 0x7FFFu + ((u >> 16) & 1u);
  return (uint16_t)(u >> 16);
}

__device__ __forceinline__ float rowwise_epilogue(float acc, float sa, float sb) {
  const float v = acc * sa;
  return v * sb;
}

// Rowwise epilogue variants: EPI_F16 writes fp16 instead of bf16, EPI_BIAS
// adds bias[c] (a value of the output dtype, widened exactly) in fp32 before
// the final rounding: out = rnd(RN32(RN32(acc * sa) * sb) + bias).
enum { EPI_F16 = 1, EPI_BIAS = 2 };

// Both conversions are the hardware's round-to-nearest-even (overflow to
// +-inf); the bf16 one (v_cvt_pk_bf16_f32) equals f32_to_bf16_rne for every
// fp32 value that is not NaN (checked over all 2^32 patterns on gfx950).
template <int EPI>
__device__ __forceinline__ uint16_t epi_round(float v) {
  if constexpr ((EPI & EPI_F16) != 0)
    return __builtin_bit_cast(uint16_t, (_Float16)v);
  else
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}

template <int EPI>
__device__ __forceinline__ float epi_value(float acc, float sa, float sb,
                                           const uint16_t* __restrict__ bias, int c) {
  float v = rowwise_epilogue(acc, sa, sb);
  if constexpr ((EPI & EPI_BIAS) != 0) {
    if constexpr ((EPI & EPI_F16) != 0)
      v = v + (float)__builtin_bit_cast(_Float16, bias[c]);
    else
      v = v + __uint_as_float((uint32_t)bias[c] << 16);
  }
  return v;
}

// Scale and store one lane's four consecutive outputs of row r (columns c..c+3,
// c a multiple of 4; N % 8 == 0 so all four are in range when c < N).
template <int EPI>
__device__ __forceinline__ void store_row4(uint16_t* __restrict__ C, int64_t ldc, int r, int c,
                                           const f32x4& acc, float sar,
                                           const float* __restrict__ sb, int sb_vec,
                                           const uint16_t* __restrict__ bias) {
  float y[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) y[v] = epi_value<EPI>(acc[v], sar, sb[sb_vec ? c + v : 0], bias, c + v);
  uint32_t lo, hi;
  if constexpr ((EPI & EPI_F16) != 0) {
    lo = (uint32_t)epi_round<EPI>(y[0]) | ((uint32_t)epi_round<EPI>(y[1]) << 16);
    hi = (uint32_t)epi_round<EPI>(y[2]) | ((uint32_t)epi_round<EPI>(y[3]) << 16);
  } else {  // two values per conversion instruction
    lo = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)y[0], (__bf16)y[1]});
    hi = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)y[2], (__bf16)y[3]});
  }
  *reinterpret_cast<uint2*>(C + (int64_t)r * ldc + c) = make_uint2(lo, hi);
}

// The same for two consecutive outputs (columns c, c + 1, c even): one 4-byte
// store.
template <int EPI>
__device__ __forceinline__ void store_row2(uint16_t* __restrict__ C, int64_t ldc, int r, int c,
                                           float a0, float a1, float sar,
                                           const float* __restrict__ sb, int sb_vec,
                                           const uint16_t* __restrict__ bias) {
  const float y0 = epi_value<EPI>(a0, sar, sb[sb_vec ? c : 0], bias, c);
  const float y1 = epi_value<EPI>(a1, sar, sb[sb_vec ? c + 1 : 0], bias, c + 1);
  uint32_t v;
  if constexpr ((EPI & EPI_F16) != 0)
    v = (uint32_t)epi_round<EPI>(y0) | ((uint32_t)epi_round<EPI>(y1) << 16);
  else
    v = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)y0, (__bf16)y1});
  *reinterpret_cast<uint32_t*>(C + (int64_t)r * ldc + c) = v;
}

// Hardware places consecutive workgroups on the 8 XCDs in turn; give each XCD
// a contiguous range of logical tiles (so tiles sharing A / B panels share an
// L2), then walk the logical tiles in groups of kGroupM tile rows.
template <int kGroupM = 8>
__device__ __forceinline__ void tile_coords(int bid, int nbid, int tiles_m, int tiles_n, int& tm,
                                            int& tn) {
  constexpr int kXcd = 8;
  const int xcd = bid % kXcd, idx = bid / kXcd;
  const int lid = xcd * (nbid / kXcd) + min(xcd, nbid % kXcd) + idx;
  const int per_group = kGroupM * tiles_n;
  const int group = lid / per_group;
  const int first_m = group * kGroupM;
  const int gm = min(tiles_m - first_m, kGroupM);
  const int r = lid - group * per_group;
  tm = first_m + r % gm;
  tn = r / gm;
}

static dim3 grid2(int64_t blocks, const GemmArgs& g) {
  return dim3((unsigned)blocks, (unsigned)g.batch.count);
}

// Runs f(std::integral_constant<int, EPI>) for the arguments' epilogue.
template <typename Fn>
static hipError_t with_epi(const GemmArgs& g, Fn&& f) {
  switch ((g.out_f16 ? EPI_F16 : 0) | (g.bias ? EPI_BIAS : 0)) {
    case 0: f(std::integral_constant<int, 0>{}); break;
    case EPI_F16: f(std::integral_constant<int, EPI_F16>{}); break;
    case EPI_BIAS: f(std::integral_constant<int, EPI_BIAS>{}); break;
    default: f(std::integral_constant<int, EPI_F16 | EPI_BIAS>{}); break;
  }
  return hipGetLastError();
}

}  // namespace fp8sm
