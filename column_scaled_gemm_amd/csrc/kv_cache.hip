// Between the QKV projection and attention (gfx950): RMS norm and position
// rotation of the query and key heads, and the paged E4M3 key/value cache.
//
// Cache format.  A block is `block` (16, 32, 64, 128) consecutive tokens of
// one sequence; each block and head has one power-of-two scale, kept as the
// biased exponent byte of the library's UE8M0 scales.  For the values x of a
// block and head: a' = max(max|x|, 1e-10), e = ceil(log2(RN32(a' / 448))),
// code = E4M3(x 2^-e), value = code 2^e.  Appending to a block that holds
// tokens takes the larger of its exponent and the new tokens'; where that
// raises it, the held codes are rounded again to the coarser step.  A power of
// two makes that second rounding exact except for bits that fall below the
// smallest code, and makes widening a code exact in bf16.
// K codes are [blocks][heads][block][D].  V codes are
// [blocks][heads][block / 16][D][16]: the matrix instruction of the product
// with V wants consecutive tokens of one channel in a lane, so 16 tokens of a
// channel are one 16-byte load.
#include "kv_common.h"

#include <algorithm>
#include <type_traits>

namespace fp8sm {

// ---------------------------------------------------------------------------
// Norm and rotation.  A head is D / 8 lanes of 8 values, a wavefront takes 64 /
// (D / 8) heads at a time, kRopeU times; the mates of a half-split pair come from
// the lane that loaded them.  Everything between the load and the one final
// rounding is fp32.  Bound by memory: 8320 rows of 112 heads of 128 (477 MB) in 86
// .. 93 us, 5.1 .. 5.5 TB/s.

// Sum over aligned groups of W lanes (8 or 16), in every lane of the group.
template <int W>
__device__ __forceinline__ float group_sum(float v) {
  auto dpp = [](float x, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v += dpp(v, std::integral_constant<int, 0xB1>{});   // lanes 1 0 3 2 of each four
  v += dpp(v, std::integral_constant<int, 0x4E>{});   // lanes 2 3 0 1
  v += dpp(v, std::integral_constant<int, 0x141>{});  // the other four of eight
  if constexpr (W == 16) v += dpp(v, std::integral_constant<int, 0x140>{});  // the other eight
  return v;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (F16) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  } else {
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
  }
}

// 16-byte streaming store, as store_stream8.
__device__ __forceinline__ void store_stream16(void* p, const uint4 v) {
  __builtin_nontemporal_store(u32x4{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4*>(p));
}

constexpr int kRopeU = 4;  // (8320 rows of 112 heads: 1: 119 us, 2: 108, 4: 100)

//
// AXES: pair i turns by row pos[axis(i)][t].  The token's rot cosines and sines are
// gathered into LDS once for the workgroup's heads, while their first reads are on the
// way: 8320 rows of 112 heads on three axes take 86.5 us, 5.57 TB/s, as on one axis.
template <bool F16, int D, bool NORM, bool INTER, bool AXES>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(RopeArgs a) {
  constexpr int LPH = D / 8, HPW = 64 / LPH;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int lh = lane % LPH, sub = lane / LPH;
  const int64_t t = blockIdx.x;
  const int heads = a.Hq + a.Hk, half = a.rot >> 1;
  const uint16_t* x = static_cast<const uint16_t*>(a.x) + t * a.ld_x;
  uint16_t* y = static_cast<uint16_t*>(a.y) + t * a.ld_y;
  const int h0 = (blockIdx.y * 4 + w) * (HPW * kRopeU) + sub;
  if (!AXES && h0 - sub >= heads) return;

  int64_t p = 0;
  float gathered = 0.f;
  if constexpr (AXES) {
    int pa[kMaxAxes];
#pragma unroll
    for (int k = 0; k < kMaxAxes; ++k) {
      pa[k] = a.pos[min(k, a.axes - 1) * a.ld_pos + t];
      if (pa[k] < 0 || pa[k] >= a.max_pos) return;  // (the whole workgroup)
    }
    if ((int)threadIdx.x < a.rot) {
      const int i = threadIdx.x, pair = i < half ? i : i - half;
      const int axis = (int)((pair < 32 ? a.axis_of[0] : a.axis_of[1]) >> (2 * (pair & 31))) & 3;
      const int row = axis == 0 ? pa[0] : axis == 1 ? pa[1] : axis == 2 ? pa[2] : pa[3];
      gathered = a.cos_sin[(int64_t)row * a.rot + i];
    }
  } else if (a.rot) {
    p = a.pos[t];
    if (p < 0 || p >= a.max_pos) return;  // names no row of the table: left as it is
  }
  uint4 v[kRopeU];
#pragma unroll
  for (int u = 0; u < kRopeU; ++u) {
    const int h = min(h0 + u * HPW, heads - 1);
    v[u] = load_stream16(x + (int64_t)h * D + lh * 8);
  }
  __shared__ __attribute__((aligned(16))) float turns[AXES ? D : 1];
  if constexpr (AXES) {
    if ((int)threadIdx.x < a.rot) turns[threadIdx.x] = gathered;
    __syncthreads();
    if (h0 - sub >= heads) return;
  }
  // the lane's pairs: 8 lh + i with 8 lh + i +- half, or adjacent elements
  const bool turned = lh * 8 < a.rot, first = lh * 8 < half;
  float cs[8], sn[8];
  if (turned) {
    const float* row = AXES ? turns : a.cos_sin + p * a.rot;
    if constexpr (INTER) {
      const float4 c = *reinterpret_cast<const float4*>(row + lh * 4);
      const float4 s = *reinterpret_cast<const float4*>(row + half + lh * 4);
      cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
      sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
    } else {
      const float* q = row + (first ? lh * 8 : lh * 8 - half);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 c = *reinterpret_cast<const float4*>(q + 4 * i);
        const float4 s = *reinterpret_cast<const float4*>(q + half + 4 * i);
        cs[4 * i] = c.x, cs[4 * i + 1] = c.y, cs[4 * i + 2] = c.z, cs[4 * i + 3] = c.w;
        sn[4 * i] = s.x, sn[4 * i + 1] = s.y, sn[4 * i + 2] = s.z, sn[4 * i + 3] = s.w;
      }
    }
  }
  const int mate = INTER ? lh : first ? lh + a.rot / 16 : lh - a.rot / 16;
  const int mate_lane = turned ? sub * LPH + mate : lane;
#pragma unroll
  for (int u = 0; u < kRopeU; ++u) {
    const int h = h0 + u * HPW;
    float f[8], g[8];
    widen8<F16>(v[u], f);
    if constexpr (!INTER) {  // the mates' raw values (every lane takes part)
      uint4 o;
      o.x = __shfl(v[u].x, mate_lane, 64);
      o.y = __shfl(v[u].y, mate_lane, 64);
      o.z = __shfl(v[u].z, mate_lane, 64);
      o.w = __shfl(v[u].w, mate_lane, 64);
      widen8<F16>(o, g);
    }
    if constexpr (NORM) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s = __builtin_fmaf(f[i], f[i], s);
      s = group_sum<LPH>(s);
      const float r = 1.0f / sqrtf(__builtin_fmaf(s, 1.0f / D, a.eps));
      const uint16_t* wt = static_cast<const uint16_t*>(h < a.Hq ? a.wq : a.wk);
      float wf[8];
      widen8<F16>(*reinterpret_cast<const uint4*>(wt + lh * 8), wf);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * r * wf[i];
      if constexpr (!INTER) {
        widen8<F16>(*reinterpret_cast<const uint4*>(wt + (turned ? mate : lh) * 8), wf);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = g[i] * r * wf[i];
      }
    }
    if (turned) {
      if constexpr (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float e = f[2 * i], o = f[2 * i + 1];
          f[2 * i] = e * cs[i] - o * sn[i];
          f[2 * i + 1] = o * cs[i] + e * sn[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * cs[i] + (first ? -g[i] : g[i]) * sn[i];
      }
    }
    if (h < heads)
      store_stream16(y + (int64_t)h * D + lh * 8,
                     make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]),
                                pack2<F16>(f[4], f[5]), pack2<F16>(f[6], f[7])));
  }
}

template <bool F16, int D, bool AXES>
static void rope_launch(const RopeArgs& a, hipStream_t s) {
  constexpr int per = 4 * (64 / (D / 8)) * kRopeU;
  const dim3 grid((uint32_t)a.T, (uint32_t)((a.Hq + a.Hk + per - 1) / per));
  if (a.wq || a.wk) {
    if (a.interleaved)
      qk_norm_rope_kernel<F16, D, true, true, AXES><<<grid, 256, 0, s>>>(a);
    else
      qk_norm_rope_kernel<F16, D, true, false, AXES><<<grid, 256, 0, s>>>(a);
  } else {
    if (a.interleaved)
      qk_norm_rope_kernel<F16, D, false, true, AXES><<<grid, 256, 0, s>>>(a);
    else
      qk_norm_rope_kernel<F16, D, false, false, AXES><<<grid, 256, 0, s>>>(a);
  }
}

template <bool AXES>
static void rope_launch_of(const RopeArgs& a, hipStream_t s) {
  if (a.D == 64)
    a.f16 ? rope_launch<true, 64, AXES>(a, s) : rope_launch<false, 64, AXES>(a, s);
  else
    a.f16 ? rope_launch<true, 128, AXES>(a, s) : rope_launch<false, 128, AXES>(a, s);
}

hipError_t launch_qk_norm_rope(const RopeArgs& a, hipStream_t s) {
  a.axes ? rope_launch_of<true>(a, s) : rope_launch_of<false>(a, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Writing.  A unit is one touched block of one sequence, one head, K or V; it
// owns the block's codes and exponent, so nothing is written by two
// wavefronts.  W wavefronts share a unit, TPW tokens each (block = W TPW), and
// hold its new values in registers between finding the largest and encoding: one
// read, one write.  K takes 16-byte loads of a token's channels, V 4-byte loads
// (a whole row of 128 channels a wavefront), so that a lane ends up with 16
// tokens of two channels, 32 contiguous bytes of the cache.  Bound by memory: 8320
// tokens of 56 heads (238 MB in, 119 out) in 65 .. 83 us, 4.3 .. 5.4 TB/s; a copy
// of 2 GiB runs at 4.9.

// bit pattern of |v|, 0 for infinities and NaN: they do not set a scale
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
  return b >= 0x7F800000u ? 0u : b;
}

// v 2^-e as the conversion's operand: clamped to the largest code, NaN kept
__device__ __forceinline__ float code_operand(float v, float mult) {
  const float s = v * mult;
  const float c = fminf(fmaxf(s, -kQMax), kQMax);
  return s == s ? c : s;
}

// four codes of four operands
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// four codes rounded again to a step 2^-s times as fine (mult = 2^s, s <= 0)
__device__ __forceinline__ uint32_t recode4(uint32_t v, float mult) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, true);
  return codes4(lo[0] * mult, lo[1] * mult, hi[0] * mult, hi[1] * mult);
}

// biased exponent of a block whose largest magnitude has these bits (the rule
// of the UE8M0 group quant: adding 0x1FFFFF carries into the exponent field
// exactly when a > 448 2^k)
__device__ __forceinline__ int block_exponent(uint32_t amax_bits) {
  const float a = fmaxf(__uint_as_float(amax_bits), kAmaxFloor);
  return (int)((__float_as_uint(a) + 0x1FFFFFu) >> 23) - 8;
}

// 2^-(e - 127) of a biased exponent: a block written elsewhere may hold up to 254,
// whose factor is below the normal range
__device__ __forceinline__ float encode_factor(int e) { return exp_byte_value(max(254 - e, 0)); }

template <bool F16>
__device__ __forceinline__ void widen2(uint32_t v, float& a, float& b) {
  if constexpr (F16) {
    a = (float)__builtin_bit_cast(_Float16, (uint16_t)(v & 0xFFFFu));
    b = (float)__builtin_bit_cast(_Float16, (uint16_t)(v >> 16));
  } else {
    a = __uint_as_float(v << 16);
    b = __uint_as_float(v & 0xFFFF0000u);
  }
}

struct WriteArgs {
  const uint16_t *k, *v;
  int64_t ld_k, ld_v;
  KvBatch kb;
  KvCache c;
};

// the largest pattern of the W wavefronts of a unit
template <int W>
__device__ __forceinline__ uint32_t unit_max(uint32_t m, uint32_t* red) {
  m = __float_as_uint(group_max<64>(__uint_as_float(m)));
  if constexpr (W > 1) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[w] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) m = max(m, red[w / W * W + i]);
  }
  return m;
}

template <bool F16, int D, int W, int TPW>
__global__ __launch_bounds__(256) void kv_write_kernel(WriteArgs a) {
  __shared__ uint32_t red[4];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int bs = a.c.block_shift, block = W * TPW;
  const Seq s = find_seq(a.kb, bs, blockIdx.x, 1, bs, 2);
  if (blockIdx.x < s.first) return;  // a slot of rows before the first sequence
  const int start = s.len - s.n;  // position of the first new token
  const int lo = max(start, 0);   // of the first one that has a place
  const int j = (lo >> bs) + (int)(blockIdx.x - s.first);
  const int p0 = j << bs;                                // first position of the block
  if (p0 >= s.len || lo >= s.len) return;                // the whole workgroup: no such block
  const int page = a.kb.table[(int64_t)s.b * a.kb.ld_table + j];
  if (page < 0 || page >= a.c.num_blocks) return;        // no place
  const int H = a.c.heads;
  const int half = gridDim.y / 2;                        // K's workgroups, then V's
  const bool is_v = (int)blockIdx.y >= half;
  const int unit = ((int)blockIdx.y - (is_v ? half : 0)) * (4 / W) + w / W;
  const bool live = unit < H;                            // others only meet the barrier
  const int h = live ? unit : 0;
  const int held = max(lo - p0, 0);                      // tokens the block holds already
  const int end = min(s.len - p0, block);                // new ones: held .. end - 1
  uint8_t* ep = (is_v ? a.c.ve : a.c.ke) + (int64_t)page * H + h;
  const int e_old = held ? *ep : 0;
  uint8_t* base = (is_v ? a.c.v : a.c.k) + ((int64_t)page * H + h) * block * D;
  const int t0 = (w % W) * TPW;                          // this wavefront's first token slot
  const uint16_t* src = is_v ? a.v : a.k;
  const int64_t ld = is_v ? a.ld_v : a.ld_k;
  src += ((int64_t)s.c0 + p0 - start) * ld + h * D;      // row of token slot 0

  if (!is_v) {
    constexpr int LPR = D / 8, RPI = 64 / LPR, NL = TPW / RPI;
    const int r = lane / LPR, c = lane % LPR;
    uint4 x[NL];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int p = t0 + i * RPI + r;
      x[i] = make_uint4(0, 0, 0, 0);
      if (live && p >= held && p < end) x[i] = load_stream16(src + p * ld + c * 8);
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      float f[8];
      widen8<F16>(x[i], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max(m, finite_bits(f[k]));
    }
    m = unit_max<W>(m, red);
    const int e = max(block_exponent(m), e_old);
    const float mult = encode_factor(e);
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int p = t0 + i * RPI + r;
      uint8_t* dst = base + p * D + c * 8;
      if (p >= held && p < end) {
        float f[8];
        widen8<F16>(x[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = code_operand(f[k], mult);
        *reinterpret_cast<uint2*>(dst) = make_uint2(codes4(f[0], f[1], f[2], f[3]), codes4(f[4], f[5], f[6], f[7]));
      } else if (p < held && e > e_old) {
        const float re = pow2f(max(e_old - e, -126));
        uint2 o = *reinterpret_cast<const uint2*>(dst);
        o.x = recode4(o.x, re);
        o.y = recode4(o.y, re);
        *reinterpret_cast<uint2*>(dst) = o;
      }
    }
    if (t0 == 0 && lane == 0) *ep = (uint8_t)e;
  } else {
    // a lane takes two channels; for D = 64 the halves of the wavefront take
    // eight tokens each of a run of sixteen
    constexpr int TG = 128 / D, TPL = 16 / TG, NS = TPW / 16;
    const int d = 2 * (lane % (D / 2)), tg = lane / (D / 2);
    uint32_t x[NS][TPL];
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < NS; ++q)
#pragma unroll
      for (int i = 0; i < TPL; ++i) {
        const int p = t0 + q * 16 + tg * TPL + i;
        x[q][i] = 0;
        if (live && p >= held && p < end) x[q][i] = *reinterpret_cast<const uint32_t*>(src + p * ld + d);
      }
#pragma unroll
    for (int q = 0; q < NS; ++q)
#pragma unroll
      for (int i = 0; i < TPL; ++i) {
        float f, g;
        widen2<F16>(x[q][i], f, g);
        m = max(m, max(finite_bits(f), finite_bits(g)));
      }
    m = unit_max<W>(m, red);
    const int e = max(block_exponent(m), e_old);
    const float mult = encode_factor(e);
    if (!live) return;
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      const int p = t0 + q * 16 + tg * TPL;  // the lane's first token
      if (p >= end || (p + TPL <= held && e == e_old)) continue;
      uint32_t o[2][TPL / 4];
#pragma unroll
      for (int i = 0; i < TPL / 4; ++i) {
        float f[4], g[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          widen2<F16>(x[q][4 * i + k], f[k], g[k]);
          f[k] = code_operand(f[k], mult);
          g[k] = code_operand(g[k], mult);
        }
        o[0][i] = codes4(f[0], f[1], f[2], f[3]);
        o[1][i] = codes4(g[0], g[1], g[2], g[3]);
      }
      uint8_t* dst = base + (p / 16) * (16 * D) + d * 16 + tg * TPL;
      if (p < held || p + TPL > end) {  // some tokens of the run are not new
        const float re = pow2f(max(e_old - e, -126));
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < TPL / 4; ++i) {
            const uint32_t was = *reinterpret_cast<const uint32_t*>(dst + 16 * k + 4 * i);
            const uint32_t again = e > e_old ? recode4(was, re) : was;
            uint32_t keep = 0, fresh = 0;  // bytes of held and of new tokens
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int pt = p + 4 * i + t;
              if (pt < held) keep |= 0xFFu << (8 * t);
              if (pt >= held && pt < end) fresh |= 0xFFu << (8 * t);
            }
            o[k][i] = (o[k][i] & fresh) | (again & keep) | (was & ~(keep | fresh));
          }
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if constexpr (TPL == 16)
          *reinterpret_cast<uint4*>(dst + 16 * k) = make_uint4(o[k][0], o[k][1], o[k][2], o[k][3]);
        else
          *reinterpret_cast<uint2*>(dst + 16 * k) = make_uint2(o[k][0], o[k][1]);
      }
    }
    if (t0 == 0 && lane == 0) *ep = (uint8_t)e;
  }
}

// Slots of a batch's touched blocks: f(b) of find_seq with 2 slots a sequence.
static uint32_t block_slots(const KvBatch& kb, int block_shift) {
  return (uint32_t)(((int64_t)kb.T >> block_shift) + 2 * (int64_t)kb.B);
}

template <bool F16, int D>
static void write_launch(const WriteArgs& a, hipStream_t s) {
  const uint32_t slots = block_slots(a.kb, a.c.block_shift), heads = a.c.heads;
  switch (a.c.block_shift) {
    case 4: kv_write_kernel<F16, D, 1, 16><<<dim3(slots, 2 * ((heads + 3) / 4)), 256, 0, s>>>(a); break;
    case 5: kv_write_kernel<F16, D, 1, 32><<<dim3(slots, 2 * ((heads + 3) / 4)), 256, 0, s>>>(a); break;
    case 6: kv_write_kernel<F16, D, 2, 32><<<dim3(slots, 2 * ((heads + 1) / 2)), 256, 0, s>>>(a); break;
    default: kv_write_kernel<F16, D, 4, 32><<<dim3(slots, 2 * heads), 256, 0, s>>>(a); break;
  }
}

hipError_t launch_kv_write(const void* k, const void* v, bool f16, int64_t ld_k, int64_t ld_v,
                           const KvBatch& kb, const KvCache& c, hipStream_t s) {
  const WriteArgs a{static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v), ld_k, ld_v, kb, c};
  if (c.D == 64)
    f16 ? write_launch<true, 64>(a, s) : write_launch<false, 64>(a, s);
  else
    f16 ? write_launch<true, 128>(a, s) : write_launch<false, 128>(a, s);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Reading back: the mirror of the write, one wavefront per 16 tokens of a
// block, head, K or V.  value = code 2^e in fp32 (exact), rounded once to the
// output type.  Bound by memory: 16 x 4096 tokens of 8 heads (134 MB in, 268 out)
// in 61 .. 68 us, 5.9 .. 6.6 TB/s (78 us with plain stores of K's rows).

struct ReadArgs {
  uint16_t *k, *v;  // either may be null
  int64_t ld_k, ld_v;
  KvBatch kb;
  KvCache c;
};

template <bool F16, int D>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadArgs a) {
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Seq s = find_seq(a.kb, a.c.block_shift, blockIdx.x, 1, 4, 2);
  if (blockIdx.x < s.first) return;  // a slot of rows before the first sequence
  const int start = s.len - s.n;
  const int H = a.c.heads;
  const int unit = blockIdx.y * 4 + w;
  if (unit >= 2 * H) return;
  const bool is_v = unit >= H;
  const int h = is_v ? unit - H : unit;
  uint16_t* dst = is_v ? a.v : a.k;
  if (dst == nullptr) return;
  // runs of sixteen from the one that holds the first token (start < 0: those
  // tokens do not exist, their rows are zeros)
  const int p0 = ((start >> 4) + (int)(blockIdx.x - s.first)) << 4;
  if (p0 >= s.len) return;
  const int lo = max(start - p0, 0), end = min(s.len - p0, 16);
  const int64_t ld = is_v ? a.ld_v : a.ld_k;
  dst += ((int64_t)s.c0 + p0 - start) * ld + h * D;  // row of the run's first token
  int page = -1;
  if (p0 >= 0) page = a.kb.table[(int64_t)s.b * a.kb.ld_table + (p0 >> a.c.block_shift)];
  const bool ok = page >= 0 && page < a.c.num_blocks;
  const int64_t ph = (int64_t)(ok ? page : 0) * H + h;
  const float scale = ok ? exp_byte_value((is_v ? a.c.ve : a.c.ke)[ph]) : 0.f;
  const int in = p0 & ((1 << a.c.block_shift) - 1);  // the run's place in its block
  const uint8_t* base = (is_v ? a.c.v : a.c.k) + ((ph << a.c.block_shift) + (ok ? in : 0)) * D;
  auto value = [&](float code) { return ok ? code * scale : 0.f; };
  if (!is_v) {
    constexpr int LPR = D / 8, RPI = 64 / LPR, NL = 16 / RPI;
    const int r = lane / LPR, c = lane % LPR;
    uint2 x[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) x[i] = *reinterpret_cast<const uint2*>(base + (i * RPI + r) * D + c * 8);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int p = i * RPI + r;
      if (p < lo || p >= end) continue;
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int q = (int)(k ? x[i].y : x[i].x);
        const auto lo2 = __builtin_amdgcn_cvt_pk_f32_fp8(q, false);
        const auto hi2 = __builtin_amdgcn_cvt_pk_f32_fp8(q, true);
        o[2 * k] = pack2<F16>(value(lo2[0]), value(lo2[1]));
        o[2 * k + 1] = pack2<F16>(value(hi2[0]), value(hi2[1]));
      }
      store_stream16(dst + p * ld + c * 8, make_uint4(o[0], o[1], o[2], o[3]));
    }
  } else {
    constexpr int TG = 128 / D, TPL = 16 / TG;
    const int d = 2 * (lane % (D / 2)), tg = lane / (D / 2);
    uint32_t x[2][TPL / 4];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < TPL / 4; ++i)
        x[k][i] = *reinterpret_cast<const uint32_t*>(base + (d + k) * 16 + tg * TPL + 4 * i);
#pragma unroll
    for (int i = 0; i < TPL / 4; ++i) {
      const auto a0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[0][i], false);
      const auto a1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[0][i], true);
      const auto b0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[1][i], false);
      const auto b1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[1][i], true);
      const float fa[4] = {a0[0], a0[1], a1[0], a1[1]}, fb[4] = {b0[0], b0[1], b1[0], b1[1]};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int p = tg * TPL + 4 * i + k;
        if (p >= lo && p < end)
          *reinterpret_cast<uint32_t*>(dst + p * ld + d) = pack2<F16>(value(fa[k]), value(fb[k]));
      }
    }
  }
}

template <bool F16, int D>
static void read_launch(const ReadArgs& a, hipStream_t s) {
  kv_read_kernel<F16, D><<<dim3(block_slots(a.kb, 4), (2u * a.c.heads + 3) / 4), 256, 0, s>>>(a);
}

hipError_t launch_kv_read(const KvBatch& kb, const KvCache& c, void* k, void* v, bool f16,
                          int64_t ld_k, int64_t ld_v, hipStream_t s) {
  const ReadArgs a{static_cast<uint16_t*>(k), static_cast<uint16_t*>(v), ld_k, ld_v, kb, c};
  if (c.D == 64)
    f16 ? read_launch<true, 64>(a, s) : read_launch<false, 64>(a, s);
  else
    f16 ? read_launch<true, 128>(a, s) : read_launch<false, 128>(a, s);
  return hipGetLastError();
}

}  // namespace fp8sm
