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
//
// 8320 tokens, 56 heads of 128, causal (0.99 TFLOP): 932 .. 972 us, 1.02 .. 1.06 PFLOP/s, where
// a bf16 library product of 16384^3 reaches 1.36.  Bound by the chip's power, the clock
// falls below 2 GHz under this load, and by the matrix pipe (32 products of 32 clocks a step
// and wavefront) beside the vector instructions (about 900 clocks alone, a third of them
// the 32 exponentials): a SIMD's wavefronts have to be at different ones.  What the
// parts cost (timing copies without them, before the priorities): copies 13%,
// exponentials 10%, LDS reads 9%, the second product 17%.  On the way: 1081 us with values tested for infinities at each of
// a masked step's products, 1050 with one test a step and keys read four fragments
// ahead, 1004 with P packed in pairs, 988 with the second walk apart, 949 with the
// wavefronts' priorities, 938 with values read three fragments ahead (960 .. 995 before
// the last two, by the box).  Slower, measured: 64 rows a wavefront, one a SIMD
// (1470), 256 rows a workgroup (977 against 962), rings of three steps (986), 64 rows a
// workgroup (1382), the next step's scores between this step's exponentials (the
// registers of two steps' scores spill), halves of 32 tokens with exponentials between
// the products (1046 against 1025), copies sent off behind the first reads (967 against 944).
#include "attn_common.h"
#include "lds_copy.h"
#include "packed_rows.h"

#include <type_traits>

namespace fp8sm {

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kPackedRows = 128, kPackedStep = 64;  // rows a workgroup, 32 a wavefront; tokens a step
constexpr int kAhead = 4, kAheadV = 3;  // fragments of keys, of values on their way to the registers

template <bool F16>
__device__ __forceinline__ f32x16 mfma32(uint4 a, uint4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Two values rounded to 16 bits, in one instruction for bf16.
template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (F16)
    return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  else
    return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}

// Of two 16-bit values, a word whose halves are ~0 where the value is infinite or NaN.
template <bool F16>
__device__ __forceinline__ uint32_t odd_halves(uint32_t v) {
  constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  return ((v & e) == e ? 0xFFFFu : 0u) | ((v >> 16 & e) == e ? 0xFFFF0000u : 0u);
}

__host__ __device__ __forceinline__ int64_t packed_slots(const PackedArgs& a) {
  return (int64_t)a.T * a.G / kPackedRows + a.B;
}

template <bool F16, int D>
__global__ __launch_bounds__(256, 2) void attn_packed_kernel(PackedArgs a) {
  constexpr int DT = D / 32, NK = D / 16;
  constexpr int ROWB = 2 * D;                  // bytes of a token's key or value
  constexpr int TILE = kPackedStep * ROWB;     // of a step's keys or values
  constexpr int CPW = TILE / 1024 / 4;         // copies of a wavefront a step, keys and values each
  constexpr int RPC = 1024 / ROWB;             // tokens of a copy
  constexpr int PPR = ROWB / 16;               // 16-byte pieces of a token
  constexpr float lift = F16 ? kLift : 0.f;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[2][2][TILE];
  const int lane = threadIdx.x & 63, x = lane & 31, h = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // The list of workgroups: prompts ordered by length too took 73 us against 76 (14 heads of
  // 64 in 7 prompts) and 990 against 1014 (8320 tokens), but up to 46% more with many prompts,
  // whose tiles of one length share no keys.
  const int64_t slots = packed_slots(a), n = slots * a.heads, id = workgroup_id();
  if (id >= n) return;
  int64_t from_last, hk64;
  if (a.side) {
    from_last = id / a.heads;
    hk64 = id - from_last * a.heads;
  } else {
    const int64_t part = n >> 3, rest = n & 7;
    const int64_t at = (id & 7) * part + min(id & 7, rest) + (id >> 3);
    hk64 = at / slots;
    from_last = at - hk64 * slots;
  }
  const int hk = (int)hk64;
  const int64_t slot = slots - 1 - from_last;
  // (the prompts have no cache: their lengths stand in for cached ones, unused)
  const KvBatch kb{a.cu, a.cu + 1, nullptr, 0, 1, a.T, a.B};
  const Seq s = find_seq(kb, 0, slot, a.G, 7, 1);
  const int rows = s.n * a.G;
  const int64_t r64 = (slot - s.first) * kPackedRows;
  if (r64 < 0 || r64 >= rows) return;  // (< 0: rows before the first prompt)
  const int r0 = (int)r64;
  const int tok_first = r0 / a.G, tok_last = (min(r0 + kPackedRows, rows) - 1) / a.G;
  const int t_begin = a.window ? max(tok_first - a.window + 1, 0) : 0;
  const int t_end = a.causal ? tok_last + 1 : s.n;
  const int steps = (t_end - t_begin + kPackedStep - 1) / kPackedStep;

  // the lane's row, and what it sees: [see_lo, see_hi)
  const PackedRow own = packed_row(r0, 32 * w + x, rows, hk, a.G);
  const bool ok = own.ok;
  const int tok = own.tok, head = own.head;
  const int see_hi = ok ? (a.causal ? tok + 1 : s.n) : 0;
  const int see_lo = a.window ? max(tok - a.window + 1, 0) : 0;
  // what the wavefront's rows see: nothing outside [w_lo, w_hi), everything inside
  // [all_lo, all_hi)
  int w_lo = 0, w_hi = 0, all_lo = 0, all_hi = 0;
  {
    const int a0 = r0 + 32 * w, a1 = min(a0 + 32, rows);
    if (a0 < a1) {
      const int first = a0 / a.G, last = (a1 - 1) / a.G;
      w_hi = a.causal ? last + 1 : s.n;
      all_hi = a.causal ? first + 1 : s.n;
      w_lo = a.window ? max(first - a.window + 1, 0) : 0;
      all_lo = a.window ? last - a.window + 1 : 0;
    }
  }

  f32x16 o[DT];
  // exponents are (score - before) scale - from; before is 0 but for far scores
  float m, l, from, before;
  bool far;  // of some row of the wavefront
  // An infinite or NaN value that some rows see and others do not: a product with the
  // others' p = 0 would give them NaN too.  Steps that mask look for one; a workgroup that
  // met one starts again and takes them apart in every step.
  bool odd = false;

  // Copies.  LDS takes a copy's pieces in lane order; a lane fetches the piece that
  // belongs at its place, so that rows lie swizzled: piece c of key row r at
  // c ^ kkey(r), the row's number in the order in which lanes read them; of values,
  // pairs of pieces (16 channels) at pair ^ vkey(r).
  const uint32_t lds0 = lds_address(&ring[0][0][0]);
  auto kkey = [](int r) __attribute__((always_inline)) {
    // (16 lanes read at a time, of rows 8 g + {0 .. 7, 16 .. 23}: all 64 banks; rows of 64
    // channels lie two to a line of banks)
    return D == 128 ? (r & 3) | (r >> 4 & 1) << 2 | (r >> 2 & 1) << 3 : (r >> 1 & 3) | (r >> 4 & 1) << 2;
  };
  auto vkey = [](int r) __attribute__((always_inline)) { return D == 128 ? (r & 3) | (r & 1) << 2 : r & 3; };
  uint32_t koff[CPW], voff[CPW];
#pragma unroll
  for (int c = 0; c < CPW; ++c) {
    const int r = (4 * c + w) * RPC + lane / PPR, p = lane % PPR;
    koff[c] = (uint32_t)(r * a.ld_k) * 2 + 16 * (p ^ kkey(r));
    voff[c] = (uint32_t)(r * a.ld_v) * 2 + 16 * (2 * ((p >> 1) ^ vkey(r)) + (p & 1));
  }
  const uint16_t* kbase = a.k + (int64_t)s.c0 * a.ld_k + (int64_t)hk * D;
  const uint16_t* vbase = a.v + (int64_t)s.c0 * a.ld_v + (int64_t)hk * D;
  auto issue = [&](int i) __attribute__((always_inline)) {
    const int t0 = t_begin + i * kPackedStep;
    // tokens from t_end on are past the buffer's end and come as zeros
    const int64_t last = min(kPackedStep, t_end - t0) - 1;
    const i32x4 rk = raw_buffer(kbase + (int64_t)t0 * a.ld_k, (uint32_t)(last * a.ld_k + D) * 2);
    const i32x4 rv = raw_buffer(vbase + (int64_t)t0 * a.ld_v, (uint32_t)(last * a.ld_v + D) * 2);
    const uint32_t dst = lds0 + (uint32_t)(i & 1) * (2 * TILE);
#pragma unroll
    for (int c = 0; c < CPW; ++c) lds_copy16_buf(koff[c], rk, 0, dst + (uint32_t)(4 * c + w) * 1024);
#pragma unroll
    for (int c = 0; c < CPW; ++c) lds_copy16_buf(voff[c], rv, 0, dst + TILE + (uint32_t)(4 * c + w) * 1024);
  };

  // The first copies leave before the queries are asked for, and those of lanes without
  // a row come from the tile's first one: one trip to memory for all.
  issue(0);
  uint4 qf[NK];
  {
    const uint16_t* q = a.q + (int64_t)(s.c0 + tok) * a.ld_q + (int64_t)head * D;
    const uint32_t flip = a.negate ? 0x80008000u : 0u, keep = ok ? ~0u : 0u;
#pragma unroll
    for (int k = 0; k < NK; ++k) qf[k] = *reinterpret_cast<const uint4*>(q + 16 * k + 8 * h);
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      qf[k].x = (qf[k].x ^ flip) & keep, qf[k].y = (qf[k].y ^ flip) & keep;
      qf[k].z = (qf[k].z ^ flip) & keep, qf[k].w = (qf[k].w ^ flip) & keep;
    }
  }

  // The lane's key row of 32 tokens: row m of the matrix tile is token
  // 16 ((m >> 2) & 1) + 4 (m >> 3) + m % 4, which leaves lane half h with the
  // consecutive tokens 16 h .. 16 h + 15 in its registers 0 .. 15.
  const int krow = 16 * ((x >> 2) & 1) + 4 * (x >> 3) + (x & 3);
  const int kplace = krow * ROWB + 16 * (h ^ kkey(krow));           // piece 2 u + h: ^ 32 u
  const int li = lane & 15, vrow = 16 * h + (li >> 2);
  const int vplace = vrow * ROWB + 32 * ((x >> 4) ^ vkey(vrow)) + 8 * (li & 3);  // pair 2 d + (x >> 4): ^ 64 d

  // One step.  PARTIAL: some row does not see some of its tokens.  CLEAR: values that
  // are infinite or NaN are taken out of the product, see `odd`.
  auto compute = [&](int i, auto partial_tag, auto clear_tag) __attribute__((always_inline)) {
    constexpr bool PARTIAL = decltype(partial_tag)::value, CLEAR = decltype(clear_tag)::value;
    constexpr int KF = 2 * NK, VF = 4 * DT, VA = kAheadV;  // fragments of keys, of values; of those ahead
    const int t0 = t_begin + i * kPackedStep;
    const uint8_t* lk = ring[i & 1][0];
    const uint8_t* lv = ring[i & 1][1];
    uint4 kf[KF], vf[VF];
    // keys: tokens 32 (f % 2) on, channels 16 (f / 2) on
    auto read_k = [&](int f) __attribute__((always_inline)) {
      kf[f] = *reinterpret_cast<const uint4*>(lk + 32 * (f & 1) * ROWB + (kplace ^ (32 * (f >> 1))));
    };
    // values: tokens 32 (f / 2 DT) + 8 (f / DT % 2) on of each half, channels 32 (f % DT) on
    auto read_v = [&](int f) __attribute__((always_inline)) {
      const uint8_t* place = lv + (32 * (f / (2 * DT)) + 8 * (f / DT % 2)) * ROWB + (vplace ^ (64 * (f % DT)));
      uint2 half[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        half[e] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(place + 4 * e * ROWB)));
      vf[f] = make_uint4(half[0].x, half[0].y, half[1].x, half[1].y);
    };
    f32x16 sc[2];
#pragma unroll
    for (int grp = 0; grp < 2; ++grp)
#pragma unroll
      for (int k = 0; k < 16; ++k) sc[grp][k] = 0.f;
#pragma unroll
    for (int f = 0; f < kAhead; ++f) read_k(f);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 0; f < KF; ++f) {
      if (f + kAhead < KF) read_k(f + kAhead);
      sc[f & 1] = mfma32<F16>(kf[f], qf[f >> 1], sc[f & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int f = 0; f < VA; ++f) read_v(f);

    // A SIMD has wavefronts of two or three workgroups.  One that is at its exponentials
    // goes first: the products of another need an issue slot in eight only, and the other
    // way round the vector instructions wait for products (8320 tokens, 56 heads: 995 us
    // without, 949 so, 979 with products first, 988 with one workgroup first throughout).
    __builtin_amdgcn_s_setprio(2);
    float mx = -INFINITY;
#pragma unroll
    for (int grp = 0; grp < 2; ++grp) {
      if constexpr (PARTIAL) {
        const int t = t0 + 32 * grp + 16 * h;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (t + k < see_lo || t + k >= see_hi) sc[grp][k] = -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) mx = fmaxf(mx, sc[grp][k]);
    }
    mx = half_max(mx);
    // (also the first finite score of a row: m = -inf).  Each row moves its own maximum
    // only: its bits do not depend on the rows beside it.
    const bool moves = (mx - m) * a.scale_log2 > kSlack;
    if (__any(moves)) {
      asm volatile("");  // (stays a branch)
      const float al = moves ? __builtin_amdgcn_exp2f((m - mx) * a.scale_log2) : 1.f;
      m = moves ? mx : m;
      l *= al;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int k = 0; k < 16; ++k) o[d][k] *= al;
      from = __builtin_fmaf(m == -INFINITY ? 0.f : m, a.scale_log2, -lift);
      const bool away = fabsf(from) >= kFarScore;
      before = away ? m : 0.f;
      if (away) from = -lift;
      far = __any(away);
    }
    if (far) {
      asm volatile("");
#pragma unroll
      for (int grp = 0; grp < 2; ++grp)
#pragma unroll
        for (int k = 0; k < 16; ++k) sc[grp][k] -= before;
    }
    uint4 p[2][2];
#pragma unroll
    for (int grp = 0; grp < 2; ++grp) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        sc[grp][k] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[grp][k], a.scale_log2, -from));
        sum += sc[grp][k];
      }
      l += sum;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        p[grp][j] = make_uint4(pack16<F16>(sc[grp][8 * j], sc[grp][8 * j + 1]),
                               pack16<F16>(sc[grp][8 * j + 2], sc[grp][8 * j + 3]),
                               pack16<F16>(sc[grp][8 * j + 4], sc[grp][8 * j + 5]),
                               pack16<F16>(sc[grp][8 * j + 6], sc[grp][8 * j + 7]));
    }
    if constexpr (PARTIAL && !CLEAR) {
      if (a.causal) {
        u16x2 most = {0, 0};
#pragma unroll
        for (int k = 0; k < TILE / 1024; ++k) {
          const uint4 c = *reinterpret_cast<const uint4*>(lv + 1024 * k + 16 * lane);
          const uint32_t d[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) most = __builtin_elementwise_max(most, __builtin_bit_cast(u16x2, d[e] & 0x7FFF7FFFu));
        }
        odd |= __any(max(most[0], most[1]) >= (F16 ? 0x7C00 : 0x7F80));
      }
    }
    __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int f = 0; f < VF; ++f) {
      if (f + VA < VF) read_v(f + VA);
      if constexpr (CLEAR) {
        // such values become 0, and the rows that see one are found by a product of their own
        constexpr uint32_t one = F16 ? 0x3C003C00u : 0x3F803F80u;
        uint4& c = vf[f];
        const uint4 bad = make_uint4(odd_halves<F16>(c.x), odd_halves<F16>(c.y), odd_halves<F16>(c.z), odd_halves<F16>(c.w));
        const uint4 ones = make_uint4(bad.x & one, bad.y & one, bad.z & one, bad.w & one);
        const int t = t0 + 32 * (f / (2 * DT)) + 16 * h + 8 * (f / DT % 2);
        uint32_t vis[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          vis[k] = ((t + 2 * k < see_lo || t + 2 * k >= see_hi ? 0u : 0xFFFFu) |
                    (t + 2 * k + 1 < see_lo || t + 2 * k + 1 >= see_hi ? 0u : 0xFFFF0000u)) & one;
        f32x16 z;
#pragma unroll
        for (int k = 0; k < 16; ++k) z[k] = 0.f;
        z = mfma32<F16>(ones, make_uint4(vis[0], vis[1], vis[2], vis[3]), z);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (z[k] > 0.f) o[f % DT][k] = __builtin_nanf("");
        c.x &= ~bad.x, c.y &= ~bad.y, c.z &= ~bad.z, c.w &= ~bad.w;
      }
      o[f % DT] = mfma32<F16>(vf[f], p[f / (2 * DT)][f / DT % 2], o[f % DT]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // Makes step i visible and starts the copies of step i + 1.
  auto advance = [&](int i) __attribute__((always_inline)) {
    wait_copies_but<0>();
    __syncthreads();  // step i is in LDS, and nobody reads step i - 1 any more
    if (i + 1 < steps) issue(i + 1);
  };
  // Steps of which the wavefront's rows see everything are a loop of their own,
  // between two that mask.  Whichever loop a wavefront is in, it passes advance() once
  // for each of the workgroup's steps, so all meet there.
  auto masked = [&](int first, int last, auto clear_tag) __attribute__((always_inline)) {
    for (int i = first; i < last; ++i) {
      advance(i);
      const int t0 = t_begin + i * kPackedStep;
      if (t0 < w_hi && t0 + kPackedStep > w_lo) compute(i, std::true_type{}, clear_tag);
    }
  };
  auto walk = [&](auto clear_tag) __attribute__((always_inline)) {
    m = -INFINITY, l = 0.f, from = 0.f, before = 0.f, far = false;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int k = 0; k < 16; ++k) o[d][k] = 0.f;
    if constexpr (decltype(clear_tag)::value) {
      masked(0, steps, clear_tag);
    } else {
      const int full = min(max((all_lo - t_begin + kPackedStep - 1) / kPackedStep, 0), steps);
      const int full_end = min(max((all_hi - t_begin) / kPackedStep, full), steps);
      masked(0, full, clear_tag);
      for (int i = full; i < full_end; ++i) {
        advance(i);
        compute(i, std::false_type{}, clear_tag);
      }
      masked(full_end, steps, clear_tag);
    }
  };
  walk(std::false_type{});
  if (__builtin_amdgcn_readfirstlane(__syncthreads_or(odd))) {
    issue(0);
    walk(std::true_type{});
  }

  const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
  const float sum = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
  if (!ok) return;
  const int64_t t = s.c0 + tok;
  const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
  uint16_t* dst = a.out + t * a.ld_o + (int64_t)head * D;
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int v = 0; v < 4; ++v)
      *reinterpret_cast<uint2*>(dst + 32 * d + 8 * v + 4 * h) =
          make_uint2(pack16<F16>(o[d][4 * v] * inv, o[d][4 * v + 1] * inv),
                     pack16<F16>(o[d][4 * v + 2] * inv, o[d][4 * v + 3] * inv));
  if (a.lse && h == 0)
    a.lse[t * a.Hq + head] = __builtin_fmaf(m, a.scale_log2, __builtin_amdgcn_logf(sum * (F16 ? kUnlift : 1.f))) * kLn2;
}

template <bool F16, int D>
static void packed_launch(PackedArgs a, hipStream_t s) {
  a.side = heads_side_by_side(a.T, a.B, a.heads, D);
  attn_packed_kernel<F16, D><<<grid_of(packed_slots(a) * a.heads), 256, 0, s>>>(a);
}

hipError_t launch_attention_packed(const PackedArgs& a, bool f16, hipStream_t s) {
  if (a.D == 64)
    f16 ? packed_launch<true, 64>(a, s) : packed_launch<false, 64>(a, s);
  else
    f16 ? packed_launch<true, 128>(a, s) : packed_launch<false, 128>(a, s);
  return hipGetLastError();
}

}  // namespace fp8sm
