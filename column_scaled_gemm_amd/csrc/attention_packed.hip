// Attention of whole prompts, packed one behind the other, over their own 16-bit keys
// and values (gfx950).
//
//   out[r] = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q_r . k_t)
//
// over the tokens t of its prompt that row r sees, in one pass with a running maximum
// and sum in fp32, as the attention over the cache does it.  The query heads that
// share a key head are extra rows: row r of a prompt is token r / G and head r % G.
//
// Scores are computed transposed, S^T = K Q^T, so that a lane holds one row's scores
// of consecutive tokens, which is the second operand of O^T = V^T P^T as it stands.
// The first, consecutive tokens of one channel, is what the transposing LDS read
// (ds_read_b64_tr_b16) makes of rows of V: of 16 lanes, lane i gives the place of four
// channels of token i / 4 and gets channel i of four tokens.
//
// P is rounded to the inputs' type for the product with V, half a step of each
// probability (2^-8 in bf16, 2^-11 in fp16, relative to the running maximum less 7 as
// kLift explains), as large as the rounding of the result: the matrix instructions
// take both operands in one type, and V is not moved to another one.  The sum l takes
// the unrounded p.
#include "attn_common.h"
#include "lds_copy.h"

#include <type_traits>

namespace fp8sm {

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kPackedStep = 64;  // tokens a step

template <bool F16>
__device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return (uint32_t)round16<F16>(a) | (uint32_t)round16<F16>(b) << 16;
}

// Of two 16-bit values, a word whose halves are ~0 where the value is infinite or NaN.
template <bool F16>
__device__ __forceinline__ uint32_t odd_halves(uint32_t v) {
  constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  return ((v & e) == e ? 0xFFFFu : 0u) | ((v >> 16 & e) == e ? 0xFFFF0000u : 0u);
}

__host__ __device__ __forceinline__ int64_t packed_slots(const PackedArgs& a, int rows) {
  return (int64_t)a.T * a.G / rows + a.B;
}

// 128 RG rows of one prompt and key head a workgroup, 32 RG a wavefront.
template <bool F16, int D, int RG>
__global__ __launch_bounds__(256, 2 / RG) void attn_packed_kernel(PackedArgs a) {
  constexpr int DT = D / 32, NK = D / 16, ROWS = 128 * RG;
  constexpr int ROWB = 2 * D;                  // bytes of a token's key or value
  constexpr int TILE = kPackedStep * ROWB;     // of a step's keys or values
  constexpr int CPW = TILE / 1024 / 4;         // copies of a wavefront a step, keys and values each
  constexpr int RPC = 1024 / ROWB;             // tokens of a copy
  constexpr int PPR = ROWB / 16;               // 16-byte pieces of a token
  constexpr int NSLOT = 2;
  constexpr float lift = F16 ? kLift : 0.f;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[NSLOT][2][TILE];
  const int tid = threadIdx.x, lane = tid & 63, x = lane & 31, h = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // The list is head, row tile with the last tile (most tokens to see) first, each
  // XCD taking a contiguous part where that leaves none with more work.
  const int64_t slots = packed_slots(a, ROWS), n = slots * a.heads, id = workgroup_id();
  if (id >= n) return;
  const int64_t part = n >> 3, rest = n & 7;
  const int64_t at = a.heads % 8 == 0 || a.heads >= 64 ? (id & 7) * part + min(id & 7, rest) + (id >> 3) : id;
  const int hk = (int)(at / slots);
  const int64_t slot = slots - 1 - (at - hk * slots);
  // (the prompts have no cache: their lengths stand in for cached ones, unused)
  const KvBatch kb{a.cu, a.cu + 1, nullptr, 0, 1, a.T, a.B};
  const Seq s = find_seq(kb, 0, slot, a.G, RG == 1 ? 7 : 8, 1);
  const int rows = s.n * a.G;
  const int64_t r64 = (slot - s.first) * ROWS;
  if (r64 < 0 || r64 >= rows) return;  // (< 0: rows before the first prompt)
  const int r0 = (int)r64;
  const int tok_first = r0 / a.G, tok_last = (min(r0 + ROWS, rows) - 1) / a.G;
  const int t_begin = a.window ? max(tok_first - a.window + 1, 0) : 0;
  const int t_end = a.causal ? tok_last + 1 : s.n;
  const int steps = (t_end - t_begin + kPackedStep - 1) / kPackedStep;

  // rows of the lane, and what they see: [see_lo, see_hi)
  int see_lo[RG], see_hi[RG], tok[RG], head[RG];
  uint4 qf[RG][NK];
#pragma unroll
  for (int i = 0; i < RG; ++i) {
    const int r = r0 + 32 * (RG * w + i) + x;
    const bool ok = r < rows;
    tok[i] = ok ? r / a.G : -1;
    head[i] = hk * a.G + (ok ? r - tok[i] * a.G : 0);
    see_hi[i] = ok ? (a.causal ? tok[i] + 1 : s.n) : 0;
    see_lo[i] = a.window ? max(tok[i] - a.window + 1, 0) : 0;
    const uint16_t* q = a.q + (int64_t)(s.c0 + max(tok[i], 0)) * a.ld_q + (int64_t)head[i] * D;
    const uint32_t flip = a.negate ? 0x80008000u : 0u;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (ok) v = *reinterpret_cast<const uint4*>(q + 16 * k + 8 * h);
      v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
      qf[i][k] = v;
    }
  }
  // what the wavefront's rows see: nothing outside [w_lo, w_hi), everything inside
  // [all_lo, all_hi)
  int w_lo = 0, w_hi = 0, all_lo = 0, all_hi = 0;
  {
    const int a0 = r0 + 32 * RG * w, a1 = min(a0 + 32 * RG, rows);
    if (a0 < a1) {
      const int first = a0 / a.G, last = (a1 - 1) / a.G;
      w_hi = a.causal ? last + 1 : s.n;
      all_hi = a.causal ? first + 1 : s.n;
      w_lo = a.window ? max(first - a.window + 1, 0) : 0;
      all_lo = a.window ? last - a.window + 1 : 0;
    }
  }

  f32x16 o[RG][DT];
  // exponents are (score - before) scale - from; before is 0 but for far scores
  float m[RG], l[RG], from[RG], before[RG];
  bool far[RG];  // of some row of the wavefront
#pragma unroll
  for (int i = 0; i < RG; ++i) {
    m[i] = -INFINITY, l[i] = 0.f, from[i] = 0.f, before[i] = 0.f, far[i] = false;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int k = 0; k < 16; ++k) o[i][d][k] = 0.f;
  }

  // Copies.  LDS takes a copy's pieces in lane order; a lane fetches the piece that
  // belongs at its place, so that rows lie swizzled: piece c of key row r at
  // c ^ kkey(r), the row's number in the order in which lanes read them; of values,
  // pairs of pieces (16 channels) at pair ^ vkey(r).
  const uint32_t lds0 = lds_address(&ring[0][0][0]);
  auto kkey = [](int r) {
    return (r & 3) | (r >> 4 & 1) << 2 | (D == 128 ? (r >> 2 & 1) << 3 : 0);
  };
  auto vkey = [](int r) { return D == 128 ? (r & 3) | (r & 1) << 2 : r & 3; };
  uint32_t koff[CPW], voff[CPW];
#pragma unroll
  for (int c = 0; c < CPW; ++c) {
    const int r = (4 * c + w) * RPC + lane / PPR, p = lane % PPR;
    koff[c] = (uint32_t)(r * a.ld_k) * 2 + 16 * (p ^ kkey(r));
    voff[c] = (uint32_t)(r * a.ld_v) * 2 + 16 * (2 * ((p >> 1) ^ vkey(r)) + (p & 1));
  }
  const uint16_t* kbase = a.k + (int64_t)s.c0 * a.ld_k + (int64_t)hk * D;
  const uint16_t* vbase = a.v + (int64_t)s.c0 * a.ld_v + (int64_t)hk * D;
  auto issue = [&](int i) {
    const int t0 = t_begin + i * kPackedStep;
    // tokens from t_end on are past the buffer's end and come as zeros
    const int64_t last = min(kPackedStep, t_end - t0) - 1;
    const i32x4 rk = raw_buffer(kbase + (int64_t)t0 * a.ld_k, (uint32_t)(last * a.ld_k + D) * 2);
    const i32x4 rv = raw_buffer(vbase + (int64_t)t0 * a.ld_v, (uint32_t)(last * a.ld_v + D) * 2);
    const uint32_t dst = lds0 + (uint32_t)(i % NSLOT) * (2 * TILE);
#pragma unroll
    for (int c = 0; c < CPW; ++c) lds_copy16_buf(koff[c], rk, 0, dst + (uint32_t)(4 * c + w) * 1024);
#pragma unroll
    for (int c = 0; c < CPW; ++c) lds_copy16_buf(voff[c], rv, 0, dst + TILE + (uint32_t)(4 * c + w) * 1024);
  };

  // The lane's key row of 32 tokens: row m of the matrix tile is token
  // 16 ((m >> 2) & 1) + 4 (m >> 3) + m % 4, which leaves lane half h with the
  // consecutive tokens 16 h .. 16 h + 15 in its registers 0 .. 15.
  const int krow = 16 * ((x >> 2) & 1) + 4 * (x >> 3) + (x & 3);
  const int kplace = krow * ROWB + 16 * (h ^ kkey(krow));           // piece 2 u + h: ^ 32 u
  const int li = lane & 15, vrow = 16 * h + (li >> 2);
  const int vplace = vrow * ROWB + 32 * ((x >> 4) ^ vkey(vrow)) + 8 * (li & 3);  // pair 2 d + (x >> 4): ^ 64 d

  auto compute = [&](int i, auto partial_tag) {
    constexpr bool PARTIAL = decltype(partial_tag)::value;
    const int t0 = t_begin + i * kPackedStep;
    const uint8_t* lk = ring[i % NSLOT][0];
    const uint8_t* lv = ring[i % NSLOT][1];
    f32x16 sc[RG][2];
#pragma unroll
    for (int g = 0; g < RG; ++g)
#pragma unroll
      for (int grp = 0; grp < 2; ++grp)
#pragma unroll
        for (int k = 0; k < 16; ++k) sc[g][grp][k] = 0.f;
#pragma unroll
    for (int u = 0; u < NK; ++u)
#pragma unroll
      for (int grp = 0; grp < 2; ++grp) {
        const uint4 c = *reinterpret_cast<const uint4*>(lk + 32 * grp * ROWB + (kplace ^ (32 * u)));
#pragma unroll
        for (int g = 0; g < RG; ++g) sc[g][grp] = mfma32<F16>(c, qf[g][u], sc[g][grp]);
      }
    uint4 p[RG][2][2];
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      float mx = -INFINITY;
#pragma unroll
      for (int grp = 0; grp < 2; ++grp) {
        if constexpr (PARTIAL) {
          const int t = t0 + 32 * grp + 16 * h;
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (t + k < see_lo[g] || t + k >= see_hi[g]) sc[g][grp][k] = -INFINITY;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) mx = fmaxf(mx, sc[g][grp][k]);
      }
      mx = half_max(mx);
      // (also the first finite score of a row: m = -inf).  Each row moves its own maximum
      // only: its bits do not depend on the rows beside it.
      const bool moves = (mx - m[g]) * a.scale_log2 > kSlack;
      if (__any(moves)) {
        const float al = moves ? __builtin_amdgcn_exp2f((m[g] - mx) * a.scale_log2) : 1.f;
        m[g] = moves ? mx : m[g];
        l[g] *= al;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int k = 0; k < 16; ++k) o[g][d][k] *= al;
        from[g] = __builtin_fmaf(m[g] == -INFINITY ? 0.f : m[g], a.scale_log2, -lift);
        const bool away = fabsf(from[g]) >= kFarScore;
        before[g] = away ? m[g] : 0.f;
        if (away) from[g] = -lift;
        far[g] = __any(away);
      }
      if (far[g]) {
#pragma unroll
        for (int grp = 0; grp < 2; ++grp)
#pragma unroll
          for (int k = 0; k < 16; ++k) sc[g][grp][k] -= before[g];
      }
#pragma unroll
      for (int grp = 0; grp < 2; ++grp) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          sc[g][grp][k] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[g][grp][k], a.scale_log2, -from[g]));
          sum += sc[g][grp][k];
        }
        l[g] += sum;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          p[g][grp][j] = make_uint4(pack16<F16>(sc[g][grp][8 * j], sc[g][grp][8 * j + 1]),
                                    pack16<F16>(sc[g][grp][8 * j + 2], sc[g][grp][8 * j + 3]),
                                    pack16<F16>(sc[g][grp][8 * j + 4], sc[g][grp][8 * j + 5]),
                                    pack16<F16>(sc[g][grp][8 * j + 6], sc[g][grp][8 * j + 7]));
      }
    }
#pragma unroll
    for (int grp = 0; grp < 2; ++grp)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          uint2 half[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint8_t* place = lv + (32 * grp + 8 * j + 4 * e) * ROWB + (vplace ^ (64 * d));
            half[e] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)place));
          }
          uint4 c = make_uint4(half[0].x, half[0].y, half[1].x, half[1].y);
          if constexpr (PARTIAL) {
            // An infinite or NaN value that some rows see and others do not: a product
            // with the others' p = 0 would give them NaN too.  Such values become 0,
            // and the rows that see one are found by a product of their own.
            const uint4 odd = make_uint4(odd_halves<F16>(c.x), odd_halves<F16>(c.y), odd_halves<F16>(c.z), odd_halves<F16>(c.w));
            if (__any((odd.x | odd.y | odd.z | odd.w) != 0)) {
              constexpr uint32_t one = F16 ? 0x3C003C00u : 0x3F803F80u;
              const uint4 ones = make_uint4(odd.x & one, odd.y & one, odd.z & one, odd.w & one);
              const int t = t0 + 32 * grp + 16 * h + 8 * j;
#pragma unroll
              for (int g = 0; g < RG; ++g) {
                uint32_t vis[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  vis[k] = ((t + 2 * k < see_lo[g] || t + 2 * k >= see_hi[g] ? 0u : 0xFFFFu) |
                            (t + 2 * k + 1 < see_lo[g] || t + 2 * k + 1 >= see_hi[g] ? 0u : 0xFFFF0000u)) & one;
                f32x16 z;
#pragma unroll
                for (int k = 0; k < 16; ++k) z[k] = 0.f;
                z = mfma32<F16>(ones, make_uint4(vis[0], vis[1], vis[2], vis[3]), z);
#pragma unroll
                for (int k = 0; k < 16; ++k)
                  if (z[k] > 0.f) o[g][d][k] = __builtin_nanf("");
              }
              c.x &= ~odd.x, c.y &= ~odd.y, c.z &= ~odd.z, c.w &= ~odd.w;
            }
          }
#pragma unroll
          for (int g = 0; g < RG; ++g) o[g][d] = mfma32<F16>(c, p[g][grp][j], o[g][d]);
        }
  };

  // Makes step i visible and starts the copies of step i + 1.
  auto advance = [&](int i) {
    wait_copies_but<0>();
    __syncthreads();  // step i is in LDS, and nobody reads step i - 1 any more
    if (i + 1 < steps) issue(i + 1);
  };
  // Steps of which the wavefront's rows see everything are a loop of their own,
  // between two that mask.  Whichever loop a wavefront is in, it passes advance() once
  // for each of the workgroup's steps, so all meet there.
  auto masked = [&](int first, int last) {
    for (int i = first; i < last; ++i) {
      advance(i);
      const int t0 = t_begin + i * kPackedStep;
      if (t0 < w_hi && t0 + kPackedStep > w_lo) compute(i, std::true_type{});
    }
  };
  issue(0);
  const int full = min(max((all_lo - t_begin + kPackedStep - 1) / kPackedStep, 0), steps);
  const int full_end = min(max((all_hi - t_begin) / kPackedStep, full), steps);
  masked(0, full);
  for (int i = full; i < full_end; ++i) {
    advance(i);
    compute(i, std::false_type{});
  }
  masked(full_end, steps);

#pragma unroll
  for (int i = 0; i < RG; ++i) {
    const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l[i]), __float_as_uint(l[i]), false, false);
    const float sum = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
    if (tok[i] < 0) continue;
    const int64_t t = s.c0 + tok[i];
    const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
    uint16_t* dst = a.out + t * a.ld_o + (int64_t)head[i] * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *reinterpret_cast<uint2*>(dst + 32 * d + 8 * v + 4 * h) =
            make_uint2(pack16<F16>(o[i][d][4 * v] * inv, o[i][d][4 * v + 1] * inv),
                       pack16<F16>(o[i][d][4 * v + 2] * inv, o[i][d][4 * v + 3] * inv));
    if (a.lse && h == 0)
      a.lse[t * a.Hq + head[i]] = __builtin_fmaf(m[i], a.scale_log2, __builtin_amdgcn_logf(sum * (F16 ? kUnlift : 1.f))) * kLn2;
  }
}

template <bool F16, int D>
static void packed_launch(const PackedArgs& a, hipStream_t s) {
  attn_packed_kernel<F16, D, 1><<<grid_of(packed_slots(a, 128) * a.heads), 256, 0, s>>>(a);
}

hipError_t launch_attention_packed(const PackedArgs& a, bool f16, hipStream_t s) {
  if (a.D == 64)
    f16 ? packed_launch<true, 64>(a, s) : packed_launch<false, 64>(a, s);
  else
    f16 ? packed_launch<true, 128>(a, s) : packed_launch<false, 128>(a, s);
  return hipGetLastError();
}

}  // namespace fp8sm
