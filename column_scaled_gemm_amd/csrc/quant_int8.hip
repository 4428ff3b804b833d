// Per-token int8 quant for gfx950, optionally of silu(gate) * up:
//   a' = max(max|y|, 1e-10), scale = RN32(a' / 127), q = RNE(RN32(y * RN32(127 / a'))).
//
// Rows are read once and held.  Plain rows are bound by memory: 8320 x 5376 bf16 21.8 us,
// 6.2 TB/s read and written (a large copy: 5.1).  Of silu(gate) * up the arithmetic
// bounds, 3.3 .. 3.6 TB/s (8320 x 2048 25 us, 4096 x 7168 44): timing copies without the
// series of e^-g take 66% of the time, without the exact division 90%.
#include "device_common.h"
#include "launch.h"

#include <type_traits>

namespace fp8sm {

// silu(g) = RN32(g / RN32(1 + RN32(e^-g))), the library's definition, computed: e^-g in
// fp64 (x = n ln 2 + r, |r| < 0.35, and the series of e^r to r^11: the next term is below
// 2^-47, and so is what fp64's ln 2 lacks, 216 times) and rounded to fp32 once, but for
// values below 2^-126, which 1 takes in.
__device__ __forceinline__ float silu(float g) {
  const float x = fminf(fmaxf(-g, -150.f), 150.f);  // (e^+-150 is 0 or infinite in fp32)
  const float n = __builtin_rintf(x * 1.442695f);
  const double r = __builtin_fma((double)n, -0.6931471805599453, (double)x);
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  const float e = __builtin_ldexpf((float)p, (int)n);
  return g / (1.0f + e);
}

// The row's multiplier and scale from its largest finite magnitude.
struct Int8Scale {
  float mult, scale;
  __device__ __forceinline__ explicit Int8Scale(float amax) {
    const float a = fmaxf(amax, kAmaxFloor);
    mult = 127.0f / a;
    scale = a / 127.0f;
  }
};

// Codes of eight values.  Adding 1.5 * 2^23 to |v| <= 2^22 rounds to the nearest
// integer, ties to even, and leaves it in the low bits.  FINITE: every value is, and
// then |y * mult| < 127.5.
template <bool FINITE>
__device__ __forceinline__ uint2 to_int8_x8(const float* y, float mult) {
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v = y[i] * mult;
    if constexpr (!FINITE) v = v != v ? 0.f : fminf(fmaxf(v, -127.f), 127.f);
    b[i] = __float_as_uint(v + 12582912.0f);
  }
  uint32_t o[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    // bytes 0 of two registers side by side, then of both pairs
    const uint32_t lo = __builtin_amdgcn_perm(b[4 * k + 1], b[4 * k], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(b[4 * k + 3], b[4 * k + 2], 0x04000c0cu);
    o[k] = lo | hi;
  }
  return make_uint2(o[0], o[1]);
}

template <bool F16, bool FUSED>
__device__ __forceinline__ void row_values(const uint4 gv, const uint4 uv, float* y) {
  widen8<F16>(gv, y);
  if constexpr (FUSED) {
    float u[8];
    widen8<F16>(uv, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = silu(y[i]) * u[i];
  }
}

__device__ __forceinline__ float finite_or_zero(float a) {  // of an absolute value
  return a < INFINITY ? a : 0.f;
}

// W wavefronts (1 or 4) share a row and hold it in registers, NC chunks of eight
// values a lane; chunks past the row's end read its last one and count for nothing.
template <bool F16, bool FUSED, int W, int NC>
__global__ __launch_bounds__(256) void quant_int8_kernel(QuantInt8Args a) {
  __shared__ float top[4], odd[4];
  const int64_t b = blockIdx.y;
  const int64_t M = batch_rows(a.batch.rows, a.M);
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = W == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + w;
  if (row >= M) return;  // (the whole workgroup where four wavefronts share a row)
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + b * a.batch.sx + row * a.ld_x;
  int8_t* q = a.q + b * a.batch.sq + row * a.ld_q;
  const int chunks = (int)(a.K >> 3);
  using Held = std::conditional_t<FUSED, float[8], uint4>;
  Held v[NC];
  int at[NC];
  bool ok[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (W == 4 ? 64 * w : 0) + lane + 64 * W * i;
    ok[i] = c < chunks;
    at[i] = min(c, chunks - 1) * 8;
  }
  uint4 g[NC], u[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    g[i] = load_stream16(x + at[i]);
    if constexpr (FUSED) u[i] = load_stream16(x + a.K + at[i]);
  }
  float amax = 0.f, sum = 0.f;  // sum: NaN as soon as some value is not finite
  if constexpr (FUSED) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      row_values<F16, true>(g[i], u[i], v[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float m = finite_or_zero(fabsf(v[i][k]));
        amax = ok[i] ? fmaxf(amax, m) : amax;
        sum = __builtin_fmaf(v[i][k], 0.f, sum);
      }
    }
  } else {
    // |x| as 16-bit patterns, which order like unsigned integers; the ones from
    // `inf` on are infinities and NaN
    constexpr uint32_t inf = F16 ? 0x7C00u : 0x7F80u;
    u16x2 m2 = {0, 0};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      v[i] = g[i];
      const uint32_t d[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(u16x2, d[k] & 0x7FFF7FFFu));
    }
    uint32_t m = max(m2[0], m2[1]);
    if (m >= inf) {
      sum = __builtin_nanf("");
      m = 0;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint32_t d[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t lo = d[k] & 0x7FFFu, hi = d[k] >> 16 & 0x7FFFu;
          m = max(m, max(lo < inf ? lo : 0u, hi < inf ? hi : 0u));
        }
      }
    }
    amax = F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)m) : __uint_as_float(m << 16);
  }
  amax = group_max<64>(amax);
  bool finite = !__any(sum != sum);
  if constexpr (W == 4) {
    if (lane == 0) {
      top[w] = amax;
      odd[w] = finite ? 0.f : 1.f;
    }
    __syncthreads();
    amax = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    finite = odd[0] + odd[1] + odd[2] + odd[3] == 0.f;
  }
  const Int8Scale s(amax);
  auto store = [&](auto fin) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      uint2 o;
      if constexpr (FUSED) {
        o = to_int8_x8<decltype(fin)::value>(v[i], s.mult);
      } else {
        float y[8];
        widen8<F16>(v[i], y);
        o = to_int8_x8<decltype(fin)::value>(y, s.mult);
      }
      if (ok[i]) store_stream8(q + at[i], o);
    }
  };
  if (finite)
    store(std::true_type{});
  else
    store(std::false_type{});
  if (lane == 0 && (W == 1 || w == 0)) a.scales[b * a.batch.ss + row] = s.scale;
}

// Rows too long for the registers: a workgroup a row, read twice (the second time
// from L2).
template <bool F16, bool FUSED>
__global__ __launch_bounds__(256) void quant_int8_long_kernel(QuantInt8Args a) {
  __shared__ float top[4];
  const int64_t b = blockIdx.y, row = blockIdx.x;
  if (row >= batch_rows(a.batch.rows, a.M)) return;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + b * a.batch.sx + row * a.ld_x;
  int8_t* q = a.q + b * a.batch.sq + row * a.ld_q;
  auto values = [&](int64_t c, float* y) {
    const uint4 g = *reinterpret_cast<const uint4*>(x + c * 8);
    uint4 u = make_uint4(0, 0, 0, 0);
    if constexpr (FUSED) u = *reinterpret_cast<const uint4*>(x + a.K + c * 8);
    row_values<F16, FUSED>(g, u, y);
  };
  float amax = 0.f;
  for (int64_t c = threadIdx.x; c < a.K >> 3; c += 256) {
    float y[8];
    values(c, y);
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, finite_or_zero(fabsf(y[k])));
  }
  amax = group_max<64>(amax);
  if ((threadIdx.x & 63) == 0) top[threadIdx.x >> 6] = amax;
  __syncthreads();
  const Int8Scale s(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
  for (int64_t c = threadIdx.x; c < a.K >> 3; c += 256) {
    float y[8];
    values(c, y);
    store_stream8(q + c * 8, to_int8_x8<false>(y, s.mult));
  }
  if (threadIdx.x == 0) a.scales[b * a.batch.ss + row] = s.scale;
}

template <bool F16, bool FUSED>
static void launch(const QuantInt8Args& a, hipStream_t s) {
  const unsigned nb = (unsigned)a.batch.count;
  auto go = [&](auto w, auto nc) {
    constexpr int W = decltype(w)::value, NC = decltype(nc)::value;
    const unsigned blocks = (unsigned)(W == 4 ? a.M : (a.M + 3) / 4);
    hipLaunchKernelGGL((quant_int8_kernel<F16, FUSED, W, NC>), dim3(blocks, nb), dim3(256), 0, s, a);
  };
  const int64_t chunks = a.K / 8;
  constexpr auto one = std::integral_constant<int, 1>{};
  constexpr auto four = std::integral_constant<int, 4>{};
  if (chunks <= 64) return go(one, one);
  if (chunks <= 128) return go(one, std::integral_constant<int, 2>{});
  if (chunks <= 256) return go(four, one);
  if (chunks <= 512) return go(four, std::integral_constant<int, 2>{});
  if (chunks <= 768) return go(four, std::integral_constant<int, 3>{});
  if (chunks <= 1024) return go(four, four);
  if (chunks <= 1536) return go(four, std::integral_constant<int, 6>{});
  if (chunks <= 2048) return go(four, std::integral_constant<int, 8>{});
  hipLaunchKernelGGL((quant_int8_long_kernel<F16, FUSED>), dim3((unsigned)a.M, nb), dim3(256), 0, s, a);
}

hipError_t launch_quant_int8(const QuantInt8Args& a, hipStream_t s) {
  if (a.fused)
    a.f16 ? launch<true, true>(a, s) : launch<false, true>(a, s);
  else
    a.f16 ? launch<true, false>(a, s) : launch<false, false>(a, s);
  return hipGetLastError();
}

}  // namespace fp8sm
