// Attention of ragged 16-bit queries over the paged E4M3 cache (gfx950).
//
//   out[r] = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q_r . k_t)
//
// over the cached tokens t that row r sees: all of its sequence's, up to its
// own position (causal), at most `window` of them.  One pass over the tokens
// with a running maximum m and sum l in fp32 (p = 2^((s - m) scale log2(e)), the
// exponential being the hardware's 2^x).  Maxima are held as scores, before the
// scale: differences of scores are then right however large the scale is, where
// rounding m scale would move every exponent by up to half a step of it.
//
// The query heads that share a key head are extra rows: row r of a sequence is
// token r / G and head r % G of its G query heads, so both kernels read each
// key and value once for all of them.  Scores are computed transposed,
// S^T = K Q^T: a lane then holds scores of one row at consecutive tokens, which
// is how the product O^T = V^T P^T wants its second operand, and V's cache
// layout holds consecutive tokens of one channel, which is its first: neither
// P nor V is moved between lanes.
#include "attn_common.h"

#include <algorithm>
#include <type_traits>

namespace fp8sm {

// Eight codes widened times a power of two, exactly unless the result leaves
// the type's range.
__device__ __forceinline__ bf16x8 widen_bf16(uint32_t d0, uint32_t d1, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, s, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d0, s, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, s, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d1, s, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ f16x8 widen_f16(uint32_t d0, uint32_t d1, float s) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d0, s, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d0, s, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d1, s, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(d1, s, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Byte mask of a dword whose bytes are tokens t .. t + 3: those in [lo, hi).
__device__ __forceinline__ uint32_t token_bytes(int t, int lo, int hi) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m |= (t + i >= lo && t + i < hi) ? 0xFFu << (8 * i) : 0u;
  return m;
}

// The NaN codes (0x7F, 0xFF) of four, as the top bits of their bytes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t v) {
  return ((v & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
// Their bytes, all bits.
__device__ __forceinline__ uint32_t byte_mask(uint32_t top) { return (top >> 7) * 0xFFu; }
// 1.0 for each of eight NaN codes, 0 for the others.
__device__ __forceinline__ f16x8 nan_ones(uint32_t n0, uint32_t n1) {
  f16x8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = (n0 >> (8 * i)) & 0x80u ? (_Float16)1.f : (_Float16)0.f;
    r[4 + i] = (n1 >> (8 * i)) & 0x80u ? (_Float16)1.f : (_Float16)0.f;
  }
  return r;
}

// The tokens that the rows [r0, r1) of a sequence see, [lo, hi), and the first
// token of their split 0 (a multiple of 64).
struct Span {
  int lo, hi, start;
  int chunk, splits;  // tokens of a split, splits in use
};
__device__ __forceinline__ Span row_span(const AttnArgs& a, const AttnSplit& sp, const Seq& s, int r0, int r1) {
  const int first = s.len - s.n + r0 / a.G, last = s.len - s.n + (r1 - 1) / a.G;
  Span p;
  p.hi = a.causal ? max(min(s.len, last + 1), 0) : s.len;
  p.lo = a.window ? max(first - a.window + 1, 0) : 0;
  p.start = p.lo & ~63;
  // the plan's chunk, longer where the lengths go beyond what the plan was told
  const int span = max(p.hi - p.start, 0);
  p.chunk = max(sp.chunk, ((span + sp.n - 1) / sp.n + 63) & ~63);
  p.splits = (span + p.chunk - 1) / p.chunk;
  return p;
}
// A row's place among the unjoined rows of a split.
__device__ __forceinline__ int64_t part_row(const AttnArgs& a, bool few, int b, int r, int64_t t, int head) {
  return few && a.few_by_seq ? ((int64_t)b * kFewRows + r) * a.c.heads + head / a.G : t * a.Hq + head;
}

// max over the four quarters of a wavefront
__device__ __forceinline__ float quarter_max(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return half_max(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}

// ---------------------------------------------------------------------------
// Few rows: 16 QT rows of one sequence and key head per workgroup, the cached
// tokens split over the grid and over the four wavefronts, 64 tokens a step.
// Bound by the stream of codes from memory; every code goes straight from
// memory to the registers of the lane that multiplies it, widened there.  A chip
// full of such workgroups streams 5.3 .. 5.9 TB/s (64 sequences of 500 .. 16384
// tokens, 8 key heads of 128, 1.13 GB: 195 .. 203 us with the join; two of
// 131072 tokens with 32 rows, 0.54 GB: 96 .. 105 us), above the 4.9 TB/s at
// which a large copy reads and writes.
// P is the sum of two bf16 values (2^-16 of p), so that V's widened codes stay exact in
// bf16 whatever their blocks' scales and the results are those of an fp32 softmax but
// for their own rounding.  One bf16 value in bf16 calls was 0 .. 5% faster (10.1 against
// 10.6 us for one row over 1000 tokens, 101 against 103 for the two of 131072) and
// added a tenth to their distance from the exact results.
//
// v_mfma_f32_16x16x32: lane l = 16 g + x holds row / column x and eight k
// values of quarter g of both operands; of the result column x and rows
// 4 g .. 4 g + 3.  Of a step's 64 tokens, key tile t (0..3) takes as its row m
// token 16 (m / 4) + 4 t + m % 4, so that lane quarter g ends up with the
// scores of the consecutive tokens 16 g .. 16 g + 15.
constexpr int kFewRuns = 256;  // runs of 16 tokens a gather brings

__host__ __device__ __forceinline__ int few_stride(const AttnArgs& a) { return a.c.heads * a.few.n | 1; }

template <bool F16, int D, int QT>
__global__ __launch_bounds__(256, 2) void attn_few_kernel(AttnArgs a) {
  constexpr int NI = D / 64, DT = D / 16;
  __shared__ int64_t mat[kFewRuns];  // a run's place in both code arrays, -1: no block
  __shared__ float mks[kFewRuns], mvs[kFewRuns];
  using op8 = std::conditional_t<F16, f16x8, bf16x8>;
  const int lane = threadIdx.x & 63, x = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int bs = a.c.block_shift;
  // heads, then splits, then row tiles: consecutive workgroups go to the eight
  // XCDs in turn.  An odd number of them a row tile (one idle) keeps any stride
  // of idle tiles or of short sequences from falling on the same XCDs (with an
  // even one, 154 us where 106 were due).
  const int per = few_stride(a), id = (int)(workgroup_id() % per);
  const int64_t slot = workgroup_id() / per;
  if (id >= a.c.heads * a.few.n) return;
  const int hk = id % a.c.heads, split = id / a.c.heads;
  // (where the long sequences are the other kernel's, a sequence has kFewRows rows at
  // most: tiles are counted by sequences, not by rows)
  const bool mixed = a.row_limit == kFewRows;
  const Seq s = find_seq(a.kb, bs, slot, mixed ? 0 : a.G, QT == 2 ? 5 : 4, mixed ? kFewRows / (16 * QT) : 1);
  const int b = s.b;
  const int rows = s.n * a.G;
  const int64_t r64 = (slot - s.first) * (16 * QT);
  if (r64 < 0 || r64 >= rows || rows > a.row_limit) return;  // (< 0: rows before the first sequence)
  const int r0 = (int)r64;
  const Span sp = row_span(a, a.few, s, r0, min(r0 + 16 * QT, rows));
  const int ns = sp.splits;
  if (split >= max(ns, 1)) return;
  const int t_begin = sp.start + split * sp.chunk;
  const int t_end = min(sp.hi, t_begin + sp.chunk);  // ns == 0: no step

  // rows of this lane: the query values, what they see, their running state
  // (32 rows' query values would not fit beside the rest, and reloading what
  // was spilled to memory waits for every code on its way: they stay in LDS)
  constexpr bool QLDS = QT == 2;
  __shared__ uint4 sq[QLDS ? QT : 1][QLDS ? 2 * NI : 1][64];
  const uint32_t flip = a.negate ? 0x80008000u : 0u;
  op8 qf[QT][2 * NI];
  int see_lo[QT], see_hi[QT];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    const int r = r0 + 16 * i + x;
    const bool ok = r < rows;
    const int tok = ok ? r / a.G : 0, p = s.len - s.n + tok;
    see_hi[i] = min(ok ? (a.causal ? min(p + 1, s.len) : s.len) : 0, t_end);
    see_lo[i] = ok && a.window ? max(p - a.window + 1, 0) : 0;
    const uint16_t* q = a.q + (int64_t)(s.c0 + tok) * a.ld_q + (int64_t)(hk * a.G + (ok ? r - tok * a.G : 0)) * D;
#pragma unroll
    for (int k = 0; k < 2 * NI; ++k) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (ok) v = *reinterpret_cast<const uint4*>(q + 64 * (k >> 1) + 16 * g + 8 * (k & 1));
      v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
      if constexpr (QLDS) {
        if (w == 0) sq[i][k][lane] = v;
      } else {
        qf[i][k] = __builtin_bit_cast(op8, v);
      }
    }
  }
  f32x4 o[QT][DT];
  float m[QT], l[QT];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d) o[i][d] = f32x4{0.f, 0.f, 0.f, 0.f};
  }
  // no step needs a mask between these (every row sees all of it)
  int all_lo = 0, all_hi = 0x7FFFFFFF;
  {
    const int first = s.len - s.n + r0 / a.G;
    const int last = s.len - s.n + (min(r0 + 16 * QT, rows) - 1) / a.G;
    if (a.causal) all_hi = first + 1;
    all_hi = min(min(all_hi, s.len), t_end);
    if (a.window) all_lo = last - a.window + 1;
  }

  const int32_t* table = a.kb.table + (int64_t)b * a.kb.ld_table;
  const int in_mask = (1 << (bs - 4)) - 1;
  // Keys of step i + 1 are loaded when those of step i are used up, its values
  // likewise, so one of them is always on its way.  Places and scales of the
  // runs of 16 tokens are gathered into LDS before (the plan's chunks need one
  // gather): with the block's number read just before its codes, every step waited
  // for two trips to memory (two sequences of 131072 tokens, 32 rows: 257 us, and
  // 167 with the gather; the grid's odd stride and the parallel join make it 101).
  const int last_run = max((t_end - 1) >> 4, 0);
  uint4 kc[4][NI], vc[DT];
  for (int seg = t_begin; seg < t_end; seg += 16 * kFewRuns) {
    if (seg > t_begin) __syncthreads();  // nobody reads the last segment's any more
    {
      const int run = (seg >> 4) + threadIdx.x;
      int64_t at = -1;
      float ks = 1.f, vs = 1.f;
      if (run <= last_run) {
        const int page = table[run >> (bs - 4)];
        if (page >= 0 && page < a.c.num_blocks) {
          const int64_t ph = (int64_t)page * a.c.heads + hk;
          at = ((ph << bs) + ((run & in_mask) << 4)) * D;
          ks = exp_byte_value(a.c.ke[ph]);
          vs = exp_byte_value(a.c.ve[ph]);
        }
      }
      mat[threadIdx.x] = at;
      mks[threadIdx.x] = ks;
      mvs[threadIdx.x] = vs;
    }
    __syncthreads();
    const int seg_end = min(t_end, seg + 16 * kFewRuns);
    auto fetch_k = [&](int t0) {
      const int64_t at = max(mat[((t0 - seg) >> 4) + (x >> 2)], (int64_t)0);
      const uint8_t* kb = a.c.k + at + (x & 3) * D + 16 * g;
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < NI; ++i) kc[t][i] = load_stream16(kb + 4 * t * D + 64 * i);
    };
    auto fetch_v = [&](int t0) {
      const int64_t at = max(mat[((t0 - seg) >> 4) + g], (int64_t)0);
      const uint8_t* vb = a.c.v + at + 16 * x;
#pragma unroll
      for (int d = 0; d < DT; ++d) vc[d] = load_stream16(vb + 256 * d);
    };
    int t0 = seg + 64 * w;
    if (t0 < seg_end) {
      fetch_k(t0);
      fetch_v(t0);
    }
    // (MORE at compile time: were the loads of the next step conditional, the
    // compiler would have to wait as if they had not been issued)
    auto step = [&](auto more) {
      constexpr bool MORE = decltype(more)::value;
      const int next = t0 + 256, mi = (t0 - seg) >> 4;
      const bool bad = mat[mi + g] < 0;  // the lane's value tokens have no block
      const float ks = mks[mi + (F16 ? g : x >> 2)], vs = mvs[mi + g];
      const bool partial = t0 + 64 > all_hi || t0 < all_lo || __any(bad);
      if constexpr (QLDS) {
        asm volatile("" ::: "memory");  // every step reads them anew
#pragma unroll
        for (int i = 0; i < QT; ++i)
#pragma unroll
          for (int k = 0; k < 2 * NI; ++k) qf[i][k] = __builtin_bit_cast(op8, sq[i][k][lane]);
      }
      f32x4 sc[QT][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int i = 0; i < QT; ++i) sc[i][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2 * NI; ++k) {
          const uint4 q = kc[t][k >> 1];
          const uint32_t c0 = (k & 1) ? q.z : q.x, c1 = (k & 1) ? q.w : q.y;
          if constexpr (F16) {
            const f16x8 kf = widen_f16(c0, c1, 1.0f);
#pragma unroll
            for (int i = 0; i < QT; ++i)
              sc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[i][k], sc[i][t], 0, 0, 0);
          } else {
            const bf16x8 kf = widen_bf16(c0, c1, ks);
#pragma unroll
            for (int i = 0; i < QT; ++i)
              sc[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[i][k], sc[i][t], 0, 0, 0);
          }
        }
      }
      if constexpr (MORE) fetch_k(next);
      bf16x8 ph[QT][2], pl[QT][2];
#pragma unroll
      for (int i = 0; i < QT; ++i) {
        if constexpr (F16) {
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[i][t][k] *= ks;
        }
        if (partial) {
          const int lo = bad ? 0x7FFFFFFF : see_lo[i], tok = t0 + 16 * g;
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (tok + 4 * t + k < lo || tok + 4 * t + k >= see_hi[i]) sc[i][t][k] = -INFINITY;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx = fmaxf(mx, sc[i][t][k]);
        mx = quarter_max(mx);
        if (__any((mx - m[i]) * a.scale_log2 > kSlack)) {  // (also a row's first score: m = -inf)
          const float mn = fmaxf(m[i], mx);
          const float al = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m[i] - mn) * a.scale_log2);
          m[i] = mn;
          l[i] *= al;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[i][d][k] *= al;
        }
        const float ms = m[i] == -INFINITY ? 0.f : m[i];
        float sum = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float p = __builtin_amdgcn_exp2f((sc[i][t][k] - ms) * a.scale_log2);
            sum += p;
            const __bf16 hi = (__bf16)p;
            ph[i][t >> 1][4 * (t & 1) + k] = hi;
            pl[i][t >> 1][4 * (t & 1) + k] = (__bf16)(p - (float)hi);
          }
        l[i] += sum;
      }
      if (partial) {  // what no row sees may hold anything, NaN codes too
        const int t = t0 + 16 * g, lo = bad ? 0x7FFFFFFF : sp.lo;
        uint32_t keep[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) keep[k] = token_bytes(t + 4 * k, lo, t_end);
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          vc[d].x &= keep[0];
          vc[d].y &= keep[1];
          vc[d].z &= keep[2];
          vc[d].w &= keep[3];
          // a NaN code that some rows see and others do not: see attn_many_kernel
          const uint32_t n0 = nan_codes(vc[d].x), n1 = nan_codes(vc[d].y), n2 = nan_codes(vc[d].z),
                         n3 = nan_codes(vc[d].w);
          if (!__any((n0 | n1 | n2 | n3) != 0)) continue;
#pragma unroll
          for (int i = 0; i < QT; ++i) {
            f16x8 vis[2];
            const int from = bad ? 0x7FFFFFFF : see_lo[i];
#pragma unroll
            for (int k = 0; k < 16; ++k)
              vis[k >> 3][k & 7] = t + k < from || t + k >= see_hi[i] ? (_Float16)0.f : (_Float16)1.f;
            f32x4 z = {0.f, 0.f, 0.f, 0.f};
            z = __builtin_amdgcn_mfma_f32_16x16x32_f16(nan_ones(n0, n1), vis[0], z, 0, 0, 0);
            z = __builtin_amdgcn_mfma_f32_16x16x32_f16(nan_ones(n2, n3), vis[1], z, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (z[k] > 0.f) o[i][d][k] = __builtin_nanf("");
          }
          vc[d].x &= ~byte_mask(n0);
          vc[d].y &= ~byte_mask(n1);
          vc[d].z &= ~byte_mask(n2);
          vc[d].w &= ~byte_mask(n3);
        }
      }
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t c0 = h ? vc[d].z : vc[d].x, c1 = h ? vc[d].w : vc[d].y;
          const bf16x8 vf = widen_bf16(c0, c1, vs);
#pragma unroll
          for (int i = 0; i < QT; ++i) {
            o[i][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, ph[i][h], o[i][d], 0, 0, 0);
            o[i][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, pl[i][h], o[i][d], 0, 0, 0);
          }
        }
      if constexpr (MORE) fetch_v(next);
      t0 = next;
    };
    if (t0 < seg_end) {
      while (t0 + 256 < seg_end) step(std::true_type{});
      step(std::false_type{});
    }
  }

  // join the four wavefronts
  __shared__ float so[4][16 * QT][D + 4];
  __shared__ float sm[4][16 * QT], sl[4][16 * QT];
#pragma unroll
  for (int i = 0; i < QT; ++i) {
    l[i] += __shfl_xor(l[i], 16, 64);
    l[i] += __shfl_xor(l[i], 32, 64);
    if (g == 0) {
      sm[w][16 * i + x] = m[i];
      sl[w][16 * i + x] = l[i];
    }
#pragma unroll
    for (int d = 0; d < DT; ++d)
      *reinterpret_cast<f32x4*>(&so[w][16 * i + x][16 * d + 4 * g]) = o[i][d];
  }
  __syncthreads();
  constexpr int LPR = D / 8;  // lanes a row, eight channels each
  for (int q = threadIdx.x; q < 16 * QT * LPR; q += 256) {
    const int row = q / LPR, d = q % LPR * 8, r = r0 + row;
    if (r >= rows) continue;
    float mm = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) mm = fmaxf(mm, sm[k][row]);
    const float ms = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, acc[8] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float f = __builtin_amdgcn_exp2f((sm[k][row] - ms) * a.scale_log2);
      ll = __builtin_fmaf(sl[k][row], f, ll);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = __builtin_fmaf(so[k][row][d + e], f, acc[e]);
    }
    const int tok = r / a.G, head = hk * a.G + (r - tok * a.G);
    const int64_t t = s.c0 + tok;
    if (ns <= 1) {
      const float inv = ll > 0.f || ll != ll ? 1.0f / ll : 0.f;
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        u[e] = (uint32_t)round16<F16>(acc[2 * e] * inv) | (uint32_t)round16<F16>(acc[2 * e + 1] * inv) << 16;
      *reinterpret_cast<uint4*>(a.out + t * a.ld_o + head * D + d) = make_uint4(u[0], u[1], u[2], u[3]);
      if (a.lse && d == 0) a.lse[t * a.Hq + head] = __builtin_fmaf(mm, a.scale_log2, __builtin_amdgcn_logf(ll)) * kLn2;
    } else {
      const int64_t at = split * a.few.rows + part_row(a, true, b, r, t, head);
      float* po = a.few.o + at * D + d;
      *reinterpret_cast<f32x4*>(po) = f32x4{acc[0], acc[1], acc[2], acc[3]};
      *reinterpret_cast<f32x4*>(po + 4) = f32x4{acc[4], acc[5], acc[6], acc[7]};
      if (d == 0) *reinterpret_cast<float2*>(a.few.ml + 2 * at) = make_float2(mm, ll);
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows: 128 rows of one sequence and key head per workgroup, 32 a
// wavefront, 64 tokens a step.  Wavefront w copies the step's run w of 16 tokens
// (keys and values, 2 KB each at D = 128) straight into an LDS ring of three
// steps; a run lies in one block, so its address is wavefront-uniform.  Block
// numbers and scales are gathered 128 runs at a time into LDS.
// 8320 tokens, 56 heads of 128, causal (0.99 TFLOP): 1020 .. 1080 us, 0.92 .. 0.97
// PFLOP/s, where a bf16 library product of 16384^3 reaches 1.36.  Bound by vector
// arithmetic (61% busy: widening 128 of a step's 300 instructions, the rest
// softmax), the matrix instructions beside it (43%) and the clock, which real data
// lowers by a fifth (920 us with constant operands).  Slower, measured: widening
// once per workgroup through LDS (1093 against 1033 us); eight wavefronts in
// alternating phases held apart by barriers (1273); the next step's scores
// beside this step's exponentials (no change); 64 rows a wavefront (registers
// spill, 2119); 32 tokens at a time (1180 .. 1193); reads sent off as a block before
// each product (1138 against 1077).
//
// v_mfma_f32_32x32x16: lane l = 32 h + x holds row / column x and eight k
// values of half h of both operands; of the result column x and rows
// 8 v + 4 h + i in register 4 v + i.  Of 32 tokens, row m of the key tile is
// token 16 ((m >> 2) & 1) + 4 (m >> 3) + m % 4, so lane half h has the scores
// of the consecutive tokens 16 h .. 16 h + 15 in its registers 0 .. 15.
//
// P is rounded to fp16 (half a step: 2^-11 of p, or 2^-32 of the row's largest if that
// is more, see kLift) and V is widened to fp16
// relative to the largest value scale within reach of the row tile: exact
// while the scales lie within 2^15 of each other (the smallest code's last
// bit, 2^-9, still is a fp16 value).  Wider ranges take V in bf16 and P as the
// sum of two bf16 values (WIDE).  Sums are fp32.
//
constexpr int kManyRows = 128, kManyStep = 64, kManySlots = 3;
constexpr int kMetaSteps = 32;  // steps whose runs' blocks and scales one gather brings

// 16-byte global -> LDS copy: reads base + off, lane i writes lds + 16 i.
// Inline asm, so that the compiler does not wait for it before each LDS read;
// wait_copies waits for what is needed.  m0 is used for nothing else here; a copy
// that follows its write needs one wait state, which inside inline asm nobody
// else puts in.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int OFF>
__device__ __forceinline__ void copy16(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 offset:%3"
               :
               : "s"(lds), "v"(off), "s"(base), "n"(OFF)
               : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__host__ __device__ __forceinline__ int64_t many_slots(const AttnArgs& a) {
  return (int64_t)a.kb.T * a.G / kManyRows + a.kb.B;
}

template <bool F16, int D>
__global__ __launch_bounds__(256, 2) void attn_many_kernel(AttnArgs a) {
  constexpr int DT = D / 32, NP = D / 32;  // channel tiles; 16-byte pieces of a lane's key row
  constexpr int RUN = 16 * D;              // bytes of a run's keys or values
  constexpr int TILE = 4 * RUN;
  constexpr int CPW = 2 * RUN / 1024;      // copies of a wavefront a step
  using op8 = std::conditional_t<F16, f16x8, bf16x8>;
  __shared__ __attribute__((aligned(1024))) uint8_t ring[kManySlots][2][TILE];
  __shared__ __attribute__((aligned(16))) int mpage[2][4 * kMetaSteps];  // block, -1: none
  __shared__ float mks[2][4 * kMetaSteps], mvs[2][4 * kMetaSteps];
  __shared__ int sref[12];
  const int tid = threadIdx.x, lane = tid & 63, x = lane & 31, h = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int bs = a.c.block_shift;
  // The list is head, split, row tile with the last tile (most tokens to see)
  // first.  Workgroups go to the eight XCDs in turn; where that leaves no XCD
  // with more work, each takes a contiguous part of the list, so that the tiles
  // that read the same keys share an L2 (8320 tokens, 56 heads: 1237 us in
  // list order, 1147 so; tiles in ascending order 1197).
  const int64_t slots = many_slots(a), n = slots * a.c.heads * a.many.n, id = workgroup_id();
  if (id >= n) return;
  const int pairs = a.c.heads * a.many.n;
  const int64_t part = n >> 3, rest = n & 7;
  const int64_t at = pairs % 8 == 0 || pairs >= 64 ? (id & 7) * part + min(id & 7, rest) + (id >> 3) : id;
  const int64_t pair = at / slots, k = at - pair * slots;
  const int64_t slot = slots - 1 - k;
  const int hk = (int)(pair / a.many.n), split = (int)(pair - (int64_t)hk * a.many.n);
  const Seq s = find_seq(a.kb, bs, slot, a.G, 7, 1);
  const int b = s.b;
  const int rows = s.n * a.G;
  const int64_t r64 = (slot - s.first) * kManyRows;
  if (r64 < 0 || r64 >= rows || rows <= a.row_limit) return;  // (< 0: rows before the first sequence)
  const int r0 = (int)r64;
  const Span sp = row_span(a, a.many, s, r0, min(r0 + kManyRows, rows));
  const int ns = sp.splits;
  if (split >= max(ns, 1)) return;
  const int t_begin = sp.start + split * sp.chunk;
  const int t_end = min(sp.hi, t_begin + sp.chunk);
  const int32_t* table = a.kb.table + (int64_t)b * a.kb.ld_table;
  const int in_mask = (1 << (bs - 4)) - 1;
  const int steps = t_end > t_begin ? (t_end - t_begin + kManyStep - 1) / kManyStep : 0;

  // the largest and smallest value exponents of the blocks in reach, and
  // whether one is missing
  int eref = 0, emin = 255, missing = 0;
  if (steps > 0) {
    for (int p = (t_begin >> bs) + tid; p <= (t_end - 1) >> bs; p += 256) {
      const int page = table[p];
      if (page >= 0 && page < a.c.num_blocks) {
        const int e = a.c.ve[(int64_t)page * a.c.heads + hk];
        eref = max(eref, e);
        emin = min(emin, e);
      } else {
        missing = 1;
      }
    }
    missing = __any(missing);
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) {
      eref = max(eref, __shfl_xor(eref, k, 64));
      emin = min(emin, __shfl_xor(emin, k, 64));
    }
    if (lane == 0) sref[w] = eref, sref[4 + w] = emin, sref[8 + w] = missing;
    __syncthreads();
    eref = max(max(sref[0], sref[1]), max(sref[2], sref[3]));
    emin = min(min(sref[4], sref[5]), min(sref[6], sref[7]));
    missing = __builtin_amdgcn_readfirstlane(sref[8] | sref[9] | sref[10] | sref[11]);
    eref = __builtin_amdgcn_readfirstlane(eref);
    emin = __builtin_amdgcn_readfirstlane(emin);
  }
  const bool wide = eref - emin > 15;

  // gathers the blocks and scales of steps [kMetaSteps k, kMetaSteps (k + 1))
  const int first_run = t_begin >> 4, last_run = max((t_end - 1) >> 4, 0);
  auto gather = [&](int k) {
    if (tid >= 4 * kMetaSteps) return;
    const int run = first_run + 4 * kMetaSteps * k + tid;
    int page = -1;
    float ks = 1.f, vs = 1.f;
    if (run <= last_run) {
      page = table[run >> (bs - 4)];
      if (page < 0 || page >= a.c.num_blocks) page = -1;
      if (page >= 0) {
        const int64_t ph = (int64_t)page * a.c.heads + hk;
        ks = exp_byte_value(a.c.ke[ph]);
        const int ve = a.c.ve[ph];
        vs = wide ? exp_byte_value(ve) : pow2f(ve - eref);
      }
    }
    mpage[k & 1][tid] = page;
    mks[k & 1][tid] = ks;
    mvs[k & 1][tid] = vs;
  };

  const int r = r0 + 32 * w + x;
  const bool ok = r < rows;
  const int tok = ok ? r / a.G : 0, head = hk * a.G + (ok ? r - tok * a.G : 0);
  const int pos = s.len - s.n + tok;
  const int see_hi = min(ok ? (a.causal ? min(pos + 1, s.len) : s.len) : 0, t_end);
  const int see_lo = ok && a.window ? max(pos - a.window + 1, 0) : 0;
  op8 qf[2 * NP];
  {
    const uint16_t* q = a.q + (int64_t)(s.c0 + tok) * a.ld_q + (int64_t)head * D;
    const uint32_t flip = a.negate ? 0x80008000u : 0u;
#pragma unroll
    for (int k = 0; k < 2 * NP; ++k) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (ok) v = *reinterpret_cast<const uint4*>(q + 32 * (k >> 1) + 16 * h + 8 * (k & 1));
      v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
      qf[k] = __builtin_bit_cast(op8, v);
    }
  }
  // what this wavefront's rows see: nothing outside [w_lo, w_hi), all of it
  // inside [all_lo, all_hi)
  int w_lo = 0, w_hi = 0, all_lo = 0, all_hi = 0;
  {
    const int a0 = r0 + 32 * w, a1 = min(a0 + 32, rows);
    if (a0 < a1) {
      const int first = s.len - s.n + a0 / a.G, last = s.len - s.n + (a1 - 1) / a.G;
      w_hi = a.causal ? max(min(s.len, last + 1), 0) : s.len;
      all_hi = min(a.causal ? min(s.len, first + 1) : s.len, t_end);
      w_lo = a.window ? max(first - a.window + 1, 0) : 0;
      all_lo = a.window ? last - a.window + 1 : 0;
    }
  }

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int k = 0; k < 16; ++k) o[d][k] = 0.f;
  float m = -INFINITY, l = 0.f, from = 0.f;  // from: m scale - lift, the exponents' reference
  bool far = false;                          // (of some row of the wavefront: kFarScore)

  const uint32_t lds0 = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) uint8_t*)&ring[0][0][0]);
  // a lane's place in a copy of key rows: LDS takes them in lane order, and 16-byte
  // piece c of row r belongs at c ^ key(r), so that the eight rows that eight
  // consecutive lanes read later lie in different banks
  uint32_t koff;
  if constexpr (D == 128) {
    const int row = lane >> 3, key = (row & 3) | (w & 1) << 2;
    koff = row * 128 + 16 * ((lane & 7) ^ key);
  } else {
    const int row = lane >> 2, key = ((row >> 1) & 1) | (w & 1) << 1;
    koff = row * 64 + 16 * ((lane & 3) ^ key);
  }
  auto issue = [&](int i) {
    const int run = __builtin_amdgcn_readfirstlane(first_run + 4 * i + w);
    const int page = max(__builtin_amdgcn_readfirstlane(mpage[(i / kMetaSteps) & 1][4 * (i % kMetaSteps) + w]), 0);
    const int64_t at = ((((int64_t)page * a.c.heads + hk) << bs) + ((run & in_mask) << 4)) * D;
    const uint32_t dst = lds0 + (uint32_t)(i % kManySlots) * (2 * TILE) + w * RUN;
    copy16<0>(a.c.k + at, koff, dst);
    if constexpr (D == 128) copy16<0>(a.c.k + at + 1024, koff, dst + 1024);
    copy16<0>(a.c.v + at, lane * 16, dst + TILE);
    if constexpr (D == 128) copy16<0>(a.c.v + at + 1024, lane * 16, dst + TILE + 1024);
  };

  // the lane's key row of 32 tokens, and its pieces' places
  const int krow = 16 * ((x >> 2) & 1) + 4 * (x >> 3) + (x & 3);
  const int kkey = D == 128 ? ((krow & 3) | ((krow >> 4) & 1) << 2) : (((krow >> 1) & 1) | ((krow >> 4) & 1) << 1);

  // One step.  PARTIAL: some row does not see some of its tokens.
  auto compute = [&](int i, auto wide_tag, auto partial_tag) {
    constexpr bool WIDE = decltype(wide_tag)::value, PARTIAL = decltype(partial_tag)::value;
    constexpr float lift = WIDE ? 0.f : kLift;
    const int t0 = t_begin + i * kManyStep;
    const uint8_t* lk = ring[i % kManySlots][0];
    const uint8_t* lv = ring[i % kManySlots][1];
    const int mb = (i / kMetaSteps) & 1, mi = 4 * (i % kMetaSteps);
    f32x16 sc[2];
#pragma unroll
    for (int grp = 0; grp < 2; ++grp)
#pragma unroll
      for (int k = 0; k < 16; ++k) sc[grp][k] = 0.f;
    float kr[2];
#pragma unroll
    for (int grp = 0; grp < 2; ++grp) kr[grp] = F16 ? 1.0f : mks[mb][mi + 2 * grp + (krow >> 4)];
#pragma unroll
    for (int u = 0; u < NP; ++u)
#pragma unroll
      for (int grp = 0; grp < 2; ++grp) {
        const uint4 c = *reinterpret_cast<const uint4*>(lk + (32 * grp + krow) * D + 16 * ((2 * u + h) ^ kkey));
        if constexpr (F16) {
          sc[grp] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen_f16(c.x, c.y, kr[grp]), qf[2 * u], sc[grp], 0, 0, 0);
          sc[grp] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen_f16(c.z, c.w, kr[grp]), qf[2 * u + 1], sc[grp], 0, 0, 0);
        } else {
          sc[grp] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_bf16(c.x, c.y, kr[grp]), qf[2 * u], sc[grp], 0, 0, 0);
          sc[grp] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_bf16(c.z, c.w, kr[grp]), qf[2 * u + 1], sc[grp], 0, 0, 0);
        }
      }
    uint32_t keep[2][4];
    // most masked steps hold no token that no row sees, and no NaN code: one test each
    // (1040 -> 1027 us; 41.0 -> 39.9 with a window of 1000 over ragged pieces)
    const bool edge = missing || t0 < sp.lo || t0 + kManyStep > t_end;
    float mx = -INFINITY;
#pragma unroll
    for (int grp = 0; grp < 2; ++grp) {
      if constexpr (F16) {
        const float ks = mks[mb][mi + 2 * grp + h];
#pragma unroll
        for (int k = 0; k < 16; ++k) sc[grp][k] *= ks;
      }
      if constexpr (PARTIAL) {
        const bool none = mpage[mb][mi + 2 * grp + h] < 0;
        const int t = t0 + 32 * grp + 16 * h, lo = none ? 0x7FFFFFFF : see_lo;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (t + k < lo || t + k >= see_hi) sc[grp][k] = -INFINITY;
        // what no row sees may hold anything, NaN codes too
        const int vlo = none ? 0x7FFFFFFF : sp.lo;
        if (edge)
#pragma unroll
          for (int k = 0; k < 4; ++k) keep[grp][k] = token_bytes(t + 4 * k, vlo, t_end);
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) mx = fmaxf(mx, sc[grp][k]);
    }
    mx = half_max(mx);
    if (__any((mx - m) * a.scale_log2 > kSlack)) {  // (also the first finite score of a row: m = -inf)
      const float mn = fmaxf(m, mx);
      const float al = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - mn) * a.scale_log2);
      m = mn;
      l *= al;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int k = 0; k < 16; ++k) o[d][k] *= al;
      from = __builtin_fmaf(m == -INFINITY ? 0.f : m, a.scale_log2, -lift);
      far = __any(fabsf(from) >= kFarScore);
      if (far) from = -lift;
    }
    if (far) {
      const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int grp = 0; grp < 2; ++grp)
#pragma unroll
        for (int k = 0; k < 16; ++k) sc[grp][k] -= ms;
    }
#pragma unroll
    for (int grp = 0; grp < 2; ++grp) {
      const float vs = mvs[mb][mi + 2 * grp + h];
      const uint8_t* vrow = lv + ((2 * grp + h) * D + x) * 16;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        sc[grp][k] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[grp][k], a.scale_log2, -from));
        sum += sc[grp][k];
      }
      l += sum;
      // A NaN code that some rows see and others do not: a product with the others'
      // p = 0 would give them NaN too.  Such codes become 0, and the rows that see one
      // are found by a product of their own.
      auto clear_nan = [&](uint4& c, f32x16& od) {
        const uint32_t n0 = nan_codes(c.x), n1 = nan_codes(c.y), n2 = nan_codes(c.z), n3 = nan_codes(c.w);
        const int t = t0 + 32 * grp + 16 * h;
        const int lo = mpage[mb][mi + 2 * grp + h] < 0 ? 0x7FFFFFFF : see_lo;
        f16x8 vis[2];
#pragma unroll
        for (int k = 0; k < 16; ++k) vis[k >> 3][k & 7] = t + k < lo || t + k >= see_hi ? (_Float16)0.f : (_Float16)1.f;
        f32x16 z;
#pragma unroll
        for (int k = 0; k < 16; ++k) z[k] = 0.f;
        z = __builtin_amdgcn_mfma_f32_32x32x16_f16(nan_ones(n0, n1), vis[0], z, 0, 0, 0);
        z = __builtin_amdgcn_mfma_f32_32x32x16_f16(nan_ones(n2, n3), vis[1], z, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (z[k] > 0.f) od[k] = __builtin_nanf("");
        c.x &= ~byte_mask(n0), c.y &= ~byte_mask(n1), c.z &= ~byte_mask(n2), c.w &= ~byte_mask(n3);
      };
      uint4 c[DT];
#pragma unroll
      for (int d = 0; d < DT; ++d) c[d] = *reinterpret_cast<const uint4*>(vrow + 512 * d);
      if constexpr (PARTIAL) {
        uint32_t any = 0;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          if (edge) c[d].x &= keep[grp][0], c[d].y &= keep[grp][1], c[d].z &= keep[grp][2], c[d].w &= keep[grp][3];
          any |= nan_codes(c[d].x) | nan_codes(c[d].y) | nan_codes(c[d].z) | nan_codes(c[d].w);
        }
        if (__any(any != 0)) {
#pragma unroll
          for (int d = 0; d < DT; ++d) clear_nan(c[d], o[d]);
        }
      }
      if constexpr (WIDE) {
        bf16x8 ph[2], pl[2];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const __bf16 hi = (__bf16)sc[grp][k];
          ph[k >> 3][k & 7] = hi;
          pl[k >> 3][k & 7] = (__bf16)(sc[grp][k] - (float)hi);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const bf16x8 v0 = widen_bf16(c[d].x, c[d].y, vs), v1 = widen_bf16(c[d].z, c[d].w, vs);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v0, ph[0], o[d], 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v0, pl[0], o[d], 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v1, ph[1], o[d], 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v1, pl[1], o[d], 0, 0, 0);
        }
      } else {
        f16x8 p[2];
#pragma unroll
        for (int k = 0; k < 16; ++k) p[k >> 3][k & 7] = (_Float16)sc[grp][k];
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen_f16(c[d].x, c[d].y, vs), p[0], o[d], 0, 0, 0);
          o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(widen_f16(c[d].z, c[d].w, vs), p[1], o[d], 0, 0, 0);
        }
      }
    }
  };

  // Makes step i visible, and starts the copies of step i + 2.
  auto advance = [&](int i) {
    if (i + 1 < steps)
      wait_copies<CPW>();
    else
      wait_copies<0>();
    __syncthreads();  // step i is in LDS, and nobody reads step i - 1 any more
    if (i % kMetaSteps == kMetaSteps / 2 && i + kMetaSteps / 2 < steps) gather(i / kMetaSteps + 1);
    if (i + 2 < steps) issue(i + 2);
  };
  // Steps of which this wavefront's rows see everything are a loop of their own,
  // between two that mask (one loop that picks the variant step by step moved the
  // accumulator between registers every time).  Whichever loop a wavefront is in, it
  // passes advance() once for each of the workgroup's steps, so all meet there.
  auto walk = [&](auto wide_tag) {
    auto masked = [&](int from, int to) {
      for (int i = from; i < to; ++i) {
        advance(i);
        const int t0 = t_begin + i * kManyStep;
        if (t0 < w_hi && t0 + kManyStep > w_lo) compute(i, wide_tag, std::true_type{});
      }
    };
    gather(0);
    __syncthreads();
    issue(0);
    if (steps > 1) issue(1);
    if constexpr (decltype(wide_tag)::value) {
      masked(0, steps);
    } else {
      int from = steps, to = steps;  // with missing blocks every step is masked
      if (!missing) {
        from = min(max((all_lo - t_begin + kManyStep - 1) / kManyStep, 0), steps);
        to = min(max((all_hi - t_begin) / kManyStep, from), steps);
      }
      masked(0, from);
      for (int i = from; i < to; ++i) {
        advance(i);
        compute(i, wide_tag, std::false_type{});
      }
      masked(to, steps);
    }
  };
  if (steps > 0) {
    if (wide)
      walk(std::true_type{});
    else
      walk(std::false_type{});
  }
  {
    const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = (__uint_as_float(sw[0]) + __uint_as_float(sw[1])) * (wide ? 1.f : kUnlift);
  }
  if (!ok) return;
  const int64_t t = s.c0 + tok;
  const float vref = wide ? 1.f : exp_byte_value(eref) * kUnlift;
  if (ns <= 1) {
    const float inv = l > 0.f || l != l ? 1.0f / l : 0.f;
    uint16_t* dst = a.out + t * a.ld_o + head * D;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        uint32_t u[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          u[e] = (uint32_t)round16<F16>(o[d][4 * v + 2 * e] * inv * vref) |
                 (uint32_t)round16<F16>(o[d][4 * v + 2 * e + 1] * inv * vref) << 16;
        *reinterpret_cast<uint2*>(dst + 32 * d + 8 * v + 4 * h) = make_uint2(u[0], u[1]);
      }
    if (a.lse && h == 0) a.lse[t * a.Hq + head] = __builtin_fmaf(m, a.scale_log2, __builtin_amdgcn_logf(l)) * kLn2;
  } else {
    const int64_t at = split * a.many.rows + part_row(a, false, b, r, t, head);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        *reinterpret_cast<f32x4*>(a.many.o + at * D + 32 * d + 8 * v + 4 * h) =
            f32x4{o[d][4 * v] * vref, o[d][4 * v + 1] * vref, o[d][4 * v + 2] * vref, o[d][4 * v + 3] * vref};
    if (h == 0) *reinterpret_cast<float2*>(a.many.ml + 2 * at) = make_float2(m, l);
  }
}

// ---------------------------------------------------------------------------
// Joins the splits of a row, WPR wavefronts per row: four for many splits, one
// for few.  D / 4 lanes take the row's channels, four each, of every NG-th split,
// keeping a running maximum as the attention itself does; the groups are joined
// in ascending order.  Four splits are read at a time: with one, the join of 64
// splits took longer than the attention (the loads' latency, one after the
// other).
template <bool F16, int D, int WPR>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a, int few_rows) {
  constexpr int TPG = D / 4, NG = WPR * 64 / TPG, U = 4;
  __shared__ f32x4 so[256 / TPG][TPG];
  __shared__ float sm[256 / TPG], sl[256 / TPG];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = workgroup_id() * (4 / WPR) + wave / WPR;
  const bool there = id < (int64_t)a.kb.T * a.Hq;
  const int t = there ? (int)(id / a.Hq) : 0, head = there ? (int)(id - (int64_t)t * a.Hq) : 0;
  const Seq s = find_seq(a.kb, a.c.block_shift, t, 1, 0, 0);
  const int b = s.b;
  const int rows = s.n * a.G;
  const bool few = rows <= a.row_limit;
  const AttnSplit& sp = few ? a.few : a.many;
  const int tile = few ? few_rows : kManyRows;
  const int r = (t - s.c0) * a.G + head % a.G, r0 = r / tile * tile;
  int ns = 0;
  if (there && t >= s.c0 && t < s.c0 + s.n)  // some sequence's row
    ns = row_span(a, sp, s, r0, min(r0 + tile, rows)).splits;
  const int gw = threadIdx.x / TPG, g = gw % NG, c = threadIdx.x % TPG;
  const int64_t part = part_row(a, few, b, r, t, head);
  float m = -INFINITY, l = 0.f;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (ns > 1) {  // (with one split the row is written already)
    for (int i0 = g; i0 < ns; i0 += NG * U) {
      float2 ml[U];
      f32x4 o[U];
      float mn = m;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * NG;
        const int64_t at = part + min(i, ns - 1) * sp.rows;
        ml[u] = *reinterpret_cast<const float2*>(sp.ml + 2 * at);
        o[u] = *reinterpret_cast<const f32x4*>(sp.o + at * D + 4 * c);
        if (i >= ns) ml[u] = make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) mn = fmaxf(mn, ml[u].x);
      const float ms = mn == -INFINITY ? 0.f : mn;
      const float al = __builtin_amdgcn_exp2f((m - ms) * a.scale_log2);
      m = mn;
      l *= al;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= al;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = __builtin_amdgcn_exp2f((ml[u].x - ms) * a.scale_log2);
        if (i0 + u * NG >= ns) continue;
        l = __builtin_fmaf(ml[u].y, f, l);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(o[u][e], f, acc[e]);
      }
    }
  }
  so[gw][c] = acc;
  if (c == 0) sm[gw] = m, sl[gw] = l;
  __syncthreads();
  if (ns <= 1 || g > 0) return;
  float mm = -INFINITY;
#pragma unroll
  for (int k = 0; k < NG; ++k) mm = fmaxf(mm, sm[gw + k]);
  const float ms = mm == -INFINITY ? 0.f : mm;
  float ll = 0.f;
  acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    const float f = __builtin_amdgcn_exp2f((sm[gw + k] - ms) * a.scale_log2);
    ll = __builtin_fmaf(sl[gw + k], f, ll);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(so[gw + k][c][e], f, acc[e]);
  }
  const float inv = ll > 0.f || ll != ll ? 1.0f / ll : 0.f;
  const uint32_t u0 = (uint32_t)round16<F16>(acc[0] * inv) | (uint32_t)round16<F16>(acc[1] * inv) << 16;
  const uint32_t u1 = (uint32_t)round16<F16>(acc[2] * inv) | (uint32_t)round16<F16>(acc[3] * inv) << 16;
  *reinterpret_cast<uint2*>(a.out + (int64_t)t * a.ld_o + head * D + 4 * c) = make_uint2(u0, u1);
  if (a.lse && c == 0) a.lse[id] = __builtin_fmaf(mm, a.scale_log2, __builtin_amdgcn_logf(ll)) * kLn2;
}

// ---------------------------------------------------------------------------
// The plan, from sizes alone (the lengths are on the device).

// Most bytes of unjoined results of one kernel.  512 sequences of one token, 64 heads
// of 128, may have 15 splits then, of 2048 tokens or more; without a bound a reach of
// 131072 tokens took 1 GiB, and 2^20 tokens of 1024 sequences 16.
constexpr int64_t kMostWorkspace = (int64_t)1 << 28;

AttnPlan plan_attention(int64_t T, int64_t B, int Hq, int Hkv, int D, int64_t max_q, int64_t max_kv,
                        int64_t window) {
  const int64_t G = Hq / Hkv;
  AttnPlan p;
  p.D = D;
  max_q = std::min(max_q, T);
  max_kv = std::min<int64_t>(max_kv, 1 << 30);
  const int64_t max_rows = max_q * G;
  // tokens that a tile of rows sees at most
  const auto reach = [&](int64_t rows) {
    return window ? std::min(max_kv, window + 64 + rows / G) : max_kv;
  };
  // tokens a split: `most`, or less to make 512 workgroups (two a CU), but not
  // below `least`
  const auto split = [&](int64_t tiles, int64_t kv, int64_t least, int64_t most, int64_t rows) {
    const int64_t ns = std::max<int64_t>(1, 512 / std::max<int64_t>(tiles, 1));
    int64_t chunk = std::min((kv + ns - 1) / ns, most);
    chunk = std::max(least, (chunk + 255) / 256 * 256);
    AttnSplit s{};
    s.chunk = (int)chunk;
    // (the grid stays within bounds whatever the hints say, also with more sequences
    // than rows, each of which has a slot: the chunks grow)
    int64_t cap = std::max<int64_t>(1, ((int64_t)1 << 22) / std::max(tiles, B * Hkv));
    // (and so does the workspace: a large batch of long contexts fills the chip with
    // fewer splits)
    cap = std::min(cap, std::max<int64_t>(1, kMostWorkspace / (rows * (D + 2) * (int64_t)sizeof(float))));
    s.n = (int)std::min(std::max<int64_t>(1, (kv + chunk - 1) / chunk), cap);
    s.rows = rows;
    return s;
  };
  p.few_split = p.many_split = AttnSplit{1, 256, T * Hq, nullptr, nullptr};
  p.few_by_seq = false;
  // One tile of 32 rows streams every code once; for more rows the tiles of the other
  // kernel are wide enough (64 sequences of 8192 tokens, 8 heads: 40 rows 270 us
  // there, 414 in two tiles here; 64 rows 335 and 442; one sequence of 4096: 23 and 19).
  p.many = max_rows > kFewRows;
  p.few_tiles = 0;
  p.row_limit = 0;
  if (p.many) {
    const int64_t tiles = std::max(T * G / kManyRows, std::min(B, T)) * Hkv;
    p.many_split = split(tiles, reach(kManyRows), 512, 1 << 30, T * Hq);
  }
  // The short sequences of a mixed batch: the kernel for many rows computes them
  // in passing where they see few tokens; with more, one workgroup of it would be
  // busy with each long after the others (and sequences that are all long, by what
  // we are told, leave nothing to do).
  const bool short_ones = !p.many || (B * max_q != T && reach(kFewRows) > 2048);
  if (short_ones) {
    // Chunks: long enough that a workgroup's start (about 4 us of dependent reads)
    // is small beside its stream, short enough that ragged lengths spread over the
    // chip.  64 sequences of 500 .. 16384 tokens, 8 heads: 203 us with 2048, 209
    // with 4096, 240 with 8192; 2 of 131072 with 32 rows: 99 us with 4096, 114 with
    // 2048, 132 with 1024.  One workgroup streams 1024 tokens in about the time that
    // the join takes.
    p.few_tiles = std::min<int64_t>(max_rows, kFewRows) <= 16 ? 1 : 2;
    p.row_limit = p.many ? kFewRows : 0x7FFFFFFF;
    const int64_t few_T = p.many ? std::min(B, T) : T;
    const int64_t tiles = std::max(few_T * G / (16 * p.few_tiles), std::min(B, T)) * Hkv;
    p.few_by_seq = p.many && B * kFewRows * Hkv < T * Hq;
    p.few_split = split(tiles, reach(16 * p.few_tiles), 1024, p.few_tiles == 1 ? 2048 : 4096,
                        p.few_by_seq ? B * kFewRows * Hkv : T * Hq);
  }
  return p;
}

template <bool F16, int D>
static void attn_launch(const AttnArgs& a, const AttnPlan& p, hipStream_t s) {
  const int64_t R = (int64_t)a.kb.T * a.G;
  if (p.many)
    attn_many_kernel<F16, D><<<grid_of(many_slots(a) * a.c.heads * a.many.n), 256, 0, s>>>(a);
  const auto few_slots = [&](int rows) {
    return p.many ? (int64_t)a.kb.B * (kFewRows / rows) : R / rows + a.kb.B;
  };
  if (p.few_tiles == 1)
    attn_few_kernel<F16, D, 1><<<grid_of(few_slots(16) * few_stride(a)), 256, 0, s>>>(a);
  else if (p.few_tiles == 2)
    attn_few_kernel<F16, D, 2><<<grid_of(few_slots(32) * few_stride(a)), 256, 0, s>>>(a);
  const int64_t out_rows = (int64_t)a.kb.T * a.Hq;
  const int n = std::max(p.few_split.n, p.many_split.n), few_rows = 16 * std::max(p.few_tiles, 1);
  if (n > 8)
    attn_join_kernel<F16, D, 4><<<grid_of(out_rows), 256, 0, s>>>(a, few_rows);
  else if (n > 1)
    attn_join_kernel<F16, D, 1><<<grid_of((out_rows + 3) / 4), 256, 0, s>>>(a, few_rows);
}

hipError_t launch_attention(const AttnArgs& a, bool f16, const AttnPlan& p, hipStream_t s) {
  if (a.c.D == 64)
    f16 ? attn_launch<true, 64>(a, p, s) : attn_launch<false, 64>(a, p, s);
  else
    f16 ? attn_launch<true, 128>(a, p, s) : attn_launch<false, 128>(a, p, s);
  return hipGetLastError();
}

}  // namespace fp8sm
