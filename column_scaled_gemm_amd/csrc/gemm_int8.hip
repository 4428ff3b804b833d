// Scaled int8 GEMM for gfx950: C[m,n] = rnd(RN32(RN32(f32(acc) * sa[m]) * sb[n]) + bias[n]),
// acc = sum_k A[m,k] B[n,k] in int32 on the int8 matrix instructions.
//
// The sum is exact (K <= 65536 products of at most 2^14 fit 31 bits), so K may be
// walked in any order and split over wavefronts: every variant gives the same bits.
#include "gemm_common.h"
#include "lds_copy.h"

#include <algorithm>
#include <type_traits>

namespace fp8sm {

// Scales and bias of NC (4 or a multiple of 8) consecutive columns, and a row's outputs
// there: NC / 4 tiles of four sums.  Columns come in eights inside N or outside.
template <int EPI, int NC>
struct Columns {
  float sb[NC], bias[(EPI & EPI_BIAS) != 0 ? NC : 1];
  __device__ __forceinline__ void load(const float* __restrict__ scales, int vec, const uint16_t* __restrict__ b, int c0, int N) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const int c = min(c0 + (k & ~3), N - 4) + (k & 3);
      sb[k] = scales[vec ? c : 0];
      if constexpr ((EPI & EPI_BIAS) != 0)
        bias[k] = (EPI & EPI_F16) != 0 ? (float)__builtin_bit_cast(_Float16, b[c]) : __uint_as_float((uint32_t)b[c] << 16);
    }
  }
  __device__ __forceinline__ uint32_t pair(int a0, int a1, float sa, int k) const {
    uint16_t u[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float y = (float)(e ? a1 : a0) * sa;
      y = y * sb[k + e];
      if constexpr ((EPI & EPI_BIAS) != 0) y = y + bias[k + e];
      // Keeps the fp32 value before its rounding: the compiler would join the last
      // product and the conversion to fp16 into one instruction that rounds once
      // (v_fma_mixlo_f16), which differs in 1 of some thousand outputs.
      if constexpr ((EPI & EPI_F16) != 0) asm("" : "+v"(y));
      u[e] = epi_round<EPI>(y);
    }
    return (uint32_t)u[0] | (uint32_t)u[1] << 16;
  }
  // `left`: columns from here to N
  __device__ __forceinline__ void store(uint16_t* __restrict__ C, const i32x4 (&t)[NC / 4], float sa, int left) const {
    if constexpr (NC == 4) {
      if (left > 0) *reinterpret_cast<uint2*>(C) = make_uint2(pair(t[0][0], t[0][1], sa, 0), pair(t[0][2], t[0][3], sa, 2));
    } else {
#pragma unroll
      for (int j = 0; j < NC / 4; j += 2)
        if (4 * j < left)
          *reinterpret_cast<uint4*>(C + 4 * j) =
              make_uint4(pair(t[j][0], t[j][1], sa, 4 * j), pair(t[j][2], t[j][3], sa, 4 * j + 2),
                         pair(t[j + 1][0], t[j + 1][1], sa, 4 * j + 4), pair(t[j + 1][2], t[j + 1][3], sa, 4 * j + 6));
    }
  }
};

// ---------------------------------------------------------------------------
// Tile kernel.  A workgroup computes BM x BN outputs with WM x WN wavefronts.  K is
// walked in steps of 128, whole 128-byte lines of every row, that copies bring into an
// LDS ring of NSLOT slots (BM rows of A, then BN rows of B), one barrier a step.  A step
// is two chunks of 64, each in a register set of its own: one is multiplied while the
// next is read, and reads and copies are placed between the rows of products.
//
// 8320 x 21504 x 5376, 256 x 256 tiles: 778 .. 790 us, 2.44 .. 2.47 POPS, where a
// library int8 product takes 850 .. 865 on the same box.  The same tile measured 1000 us with
// v_mfma_i32_32x32x32_i8 and steps of 64, 974 with scales read ahead of the stores, 872
// with 16x16x64 (half the accumulator traffic of an operation), 833 with reads and
// copies between the products, 812 with a ring walk of 4 tile rows instead of 8, 788
// with steps of 128 (half the lines that copies touch).  Bound by the chip's power and
// the copies beside the products: without copies 744 us in the first form, with all
// codes 0 825 against 972.  Small tiles are bound by the copies' rate, about 30 bytes a
// clock and CU, which more wavefronts raise (333 x 5376 x 14336 in tiles of 128 x 128: 63
// us with 4 wavefronts, 44 with 8; of 64 x 128 39, of 128 x 64 38).  Slower, measured:
// wavefronts of 128 x 128 (895 against 833), rings of 3 and 5 slots of 64 (the same,
// 847), splitting a step's K over two sets of wavefronts (the same), six slots for the
// tiles of 64 and 128 (39.9 against 39.2).
//
// Outputs: B is the first operand of v_mfma_i32_16x16x64_i8, so lane l gets row l % 16
// and four columns of a 16 x 16 result.  The TN column tiles of a wavefront interleave:
// operand row 4 g + i of tile j is column 4 TN g + 4 j + i, and lane group g = l / 16
// ends up with 4 TN consecutive columns, written 16 bytes at a time.
//
// LDS: 16-byte piece c of a row lies at c ^ key, a key that differs between the eight
// rows that eight consecutive lanes read.
constexpr int kTileK = 128;

// Waits until at most min(ahead, MOST) chunks of CPW copies are on their way.
template <int CPW, int MOST>
__device__ __forceinline__ void wait_ahead(int ahead) {
  if constexpr (MOST > 0) {
    if (ahead < MOST) return wait_ahead<CPW, MOST - 1>(ahead);
  }
  wait_copies_but<MOST * CPW>();
}

template <int BM, int BN, int WM, int WN, int NSLOT, int OCC, int EPI>
__global__ __launch_bounds__(64 * WM * WN, OCC * WM * WN / 4) void gemm_int8_tile_kernel(
    const uint8_t* __restrict__ A, int64_t lda, const uint8_t* __restrict__ B, int64_t ldb,
    uint16_t* __restrict__ C, int64_t ldc, int M, int N, int K, const float* __restrict__ sa,
    int sa_vec, const float* __restrict__ sb, int sb_vec, const uint16_t* __restrict__ bias,
    int tiles_m, int tiles_n, GemmBatch gb) {
  constexpr int NW = WM * WN, TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int SLOT = (BM + BN) * kTileK;
  constexpr int CPW = SLOT / 1024 / NW;  // copies of a wavefront a step: 8 rows of 128 bytes each
  static_assert(TM * 16 * WM == BM && TN * 16 * WN == BN && CPW * NW * 1024 == SLOT && TM >= 2, "tile shape");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NSLOT * SLOT];

  int tm, tn;
  tile_coords<4>(blockIdx.x, gridDim.x, tiles_m, tiles_n, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;
  {
    const int64_t bi = blockIdx.y;
    A += bi * gb.a;
    B += bi * gb.b;
    C += bi * gb.c;
    sa += bi * gb.sa;
    sb += bi * gb.sb;
    M = (int)batch_rows(gb.rows, M);
    if (m0 >= M) return;  // the whole workgroup, before any barrier
  }
  const int lane = threadIdx.x & 63, x = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / WN, wn = w % WN;
  const uint32_t lds0 = lds_address(lds);
  auto key_a = [](int r) { return r & 7; };
  auto key_b = [](int r) { return (r & 3) | (r / (4 * TN) & 1) << 2; };

  // Copy i of wavefront w brings 8 rows from row 8 (NW i + w) of the slot on; lane l
  // row l / 8, piece l % 8 of its slot.  Rows past M / N repeat the last one.  A
  // buffer ends at K of its last row: pieces past K of that row come as zeros, those
  // of the others as what follows in memory, and `read` drops both.
  i32x4 rs[CPW];
  uint32_t vo[CPW];
#pragma unroll
  for (int i = 0; i < CPW; ++i) {
    const int seg = i * NW + w, r = lane >> 3;
    const bool isa = seg * 8 < BM;
    const int64_t ld = isa ? lda : ldb;
    const int first = isa ? m0 + seg * 8 : n0 + seg * 8 - BM, last = (isa ? M : N) - 1;
    const int r0 = min(first, last), rr = min(first + r, last);
    const int key = isa ? key_a(r) : key_b(seg * 8 - BM + r);
    // (8 rows of at most 2^24 bytes: below 2^31)
    rs[i] = raw_buffer((isa ? A : B) + (int64_t)r0 * ld, (uint32_t)((min(first + 7, last) - r0) * ld) + (uint32_t)K);
    vo[i] = (uint32_t)((rr - r0) * ld) + (uint32_t)(((lane & 7) ^ key) * 16);
  }
  const int nk = (K + kTileK - 1) / kTileK;
  auto issue = [&](int k) {
    const uint32_t slot = lds0 + (uint32_t)((k % NSLOT) * SLOT);
    // (only the lane's own offset is sure to be held against the buffer's end)
    const bool tail = (k + 1) * kTileK > K;
    const int soff = tail ? 0 : k * kTileK;
    const uint32_t more = tail ? k * kTileK : 0;
#pragma unroll
    for (int i = 0; i < CPW; ++i) lds_copy16_buf(vo[i] + more, rs[i], soff, slot + (uint32_t)((i * NW + w) * 1024));
  };
  // Makes step k visible, `ahead` younger ones may be on their way.
  auto arrive = [&](int ahead) {
    wait_ahead<CPW, NSLOT - 2>(ahead);
    __syncthreads();
  };

  // A step is two chunks of 64: a lane reads piece 4 half + g of its rows
  const int a_at = (wm * (BM / WM) + x) * kTileK + 16 * (g ^ key_a(x));
  const int b_row = wn * (BN / WN) + 4 * TN * (x >> 2) + (x & 3);  // of column tile 0; tile j is 4 j further
  const int b_at = (BM + b_row) * kTileK + 16 * (g ^ key_b(b_row));
  auto read_a = [&](int k, int half, int i) {
    return *reinterpret_cast<const i32x4*>(lds + (k % NSLOT) * SLOT + (a_at ^ (64 * half)) + i * 16 * kTileK);
  };
  auto read_b = [&](int k, int half, int j) {
    return *reinterpret_cast<const i32x4*>(lds + (k % NSLOT) * SLOT + (b_at ^ (64 * half)) + j * 4 * kTileK);
  };
  auto read = [&](int k, int half, i32x4(&fa)[TM], i32x4(&fb)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j) fb[j] = read_b(k, half, j);
#pragma unroll
    for (int i = 0; i < TM; ++i) fa[i] = read_a(k, half, i);
    if (k * kTileK + 64 * half + 16 * g >= K) {  // past K: counts nothing (zeros on one side)
#pragma unroll
      for (int j = 0; j < TN; ++j) fb[j] = i32x4{0, 0, 0, 0};
    }
  };
  i32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto row = [&](int i, const i32x4(&fa)[TM], const i32x4(&fb)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
  };
  auto multiply = [&](const i32x4(&fa)[TM], const i32x4(&fb)[TN]) {
#pragma unroll
    for (int i = 0; i < TM; ++i) row(i, fa, fb);
  };
  // The same with the reads of another chunk, and copies, beside the rows of products.
  auto beside = [&](const i32x4(&fa)[TM], const i32x4(&fb)[TN], int k, int half, i32x4(&na)[TM], i32x4(&nb)[TN], int copy, auto with_copies) {
    const uint32_t to = lds0 + (uint32_t)((copy % NSLOT) * SLOT);
#pragma unroll
    for (int i = 0; i < TM; ++i) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        if (j * TM / TN / 2 == i) nb[j] = read_b(k, half, j);
#pragma unroll
      for (int q = 0; q < TM; ++q)
        if (q * (TM - 2) / TM + 1 == i) na[q] = read_a(k, half, q);
      if constexpr (decltype(with_copies)::value) {
#pragma unroll
        for (int q = 0; q < CPW; ++q)
          if (q * TM / CPW == i) lds_copy16_buf(vo[q], rs[q], copy * kTileK, to + (uint32_t)((q * NW + w) * 1024));
      }
      row(i, fa, fb);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  i32x4 fa0[TM], fb0[TN], fa1[TM], fb1[TN];
  for (int k = 0; k < NSLOT - 1 && k < nk; ++k) issue(k);
  arrive(min(NSLOT - 2, nk - 1));
  if (NSLOT - 1 < nk) issue(NSLOT - 1);
  read(0, 0, fa0, fb0);
  int k = 0;
  for (; k + NSLOT < nk - 1; ++k) {  // neither step k + 1 nor step k + NSLOT is the last
    beside(fa0, fb0, k, 1, fa1, fb1, 0, std::false_type{});
    wait_copies_but<(NSLOT - 2) * CPW>();
    __syncthreads();  // step k + 1 is there, and everybody has read step k
    beside(fa1, fb1, k + 1, 0, fa0, fb0, k + NSLOT, std::true_type{});
  }
  for (; k < nk; ++k) {
    read(k, 1, fa1, fb1);
    multiply(fa0, fb0);
    if (k + 1 < nk) {
      arrive(min(NSLOT - 2, nk - 2 - k));
      if (k + NSLOT < nk) issue(k + NSLOT);
      read(k + 1, 0, fa0, fb0);
    }
    multiply(fa1, fb1);
  }

  // Scales and bias are read before any store (they were not, in the first form: 21 us of 77 at 333 x 5376 x
  // 14336), from columns held inside N.
  const int c0 = n0 + wn * (BN / WN) + 4 * TN * g;
  Columns<EPI, 4 * TN> col;
  col.load(sb, sb_vec, bias, c0, N);
  float sar[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) sar[i] = sa[sa_vec ? min(m0 + wm * (BM / WM) + 16 * i + x, M - 1) : 0];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = m0 + wm * (BM / WM) + 16 * i + x;
    if (r < M) col.store(C + (int64_t)r * ldc + c0, acc[i], sar[i], N - c0);
  }
}

// ---------------------------------------------------------------------------
// Few rows: 16 MT rows x 16 NT columns a workgroup.  The weights are streamed once
// and that stream is the bound, so operands go straight from memory to registers and
// the NW wavefronts split K, 256 at a time, each with the next 256 on their way; the
// partial sums are added in LDS.  v_mfma_i32_16x16x64_i8: lane l holds 16 bytes
// from k = 16 (l / 16) on of row l % 16.  16 rows, weights from HBM: 4096 x 4096 7.3
// us, 14336 x 4096 15.6 .. 16.3 us (3.7 TB/s, some 3 us of it the launch; 14.4 where the
// last-level cache holds the 59 MB).  Streaming
// (nontemporal) loads of B took 9.1 and 16.7 us: each 128-byte line is read by two of them.
template <int MT, int NT, int NW, bool TAIL, int EPI>
__global__ __launch_bounds__(64 * NW) void gemm_int8_few_kernel(
    const uint8_t* __restrict__ A, int64_t lda, const uint8_t* __restrict__ B, int64_t ldb,
    uint16_t* __restrict__ C, int64_t ldc, int M, int N, int K, const float* __restrict__ sa,
    int sa_vec, const float* __restrict__ sb, int sb_vec, const uint16_t* __restrict__ bias,
    GemmBatch gb) {
  constexpr int U = 4, STEP = 64 * U;  // instructions and bytes of k a step
  __shared__ i32x4 part[NW][MT * NT][64];
  const int m0 = blockIdx.z * (16 * MT), n0 = blockIdx.x * (16 * NT);
  {
    const int64_t bi = blockIdx.y;
    A += bi * gb.a;
    B += bi * gb.b;
    C += bi * gb.c;
    sa += bi * gb.sa;
    sb += bi * gb.sb;
    M = (int)batch_rows(gb.rows, M);
    if (m0 >= M) return;  // the whole workgroup, before any barrier
  }
  const int lane = threadIdx.x & 63, x = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint8_t *pa[MT], *pb[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) pa[i] = A + (int64_t)min(m0 + 16 * i + x, M - 1) * lda;
#pragma unroll
  for (int j = 0; j < NT; ++j) pb[j] = B + (int64_t)min(n0 + 16 * j + x, N - 1) * ldb;
  i32x4 acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  struct Set {
    i32x4 a[U][MT], b[U][NT];
  };
  const int steps = (K + STEP - 1) / STEP;
  auto load = [&](int k, Set& s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int at = k * STEP + 64 * u + 16 * g;
      if constexpr (TAIL) at = min(at, K - 16);  // no branch around a load
#pragma unroll
      for (int j = 0; j < NT; ++j) s.b[u][j] = *reinterpret_cast<const i32x4*>(pb[j] + at);
#pragma unroll
      for (int i = 0; i < MT; ++i) s.a[u][i] = *reinterpret_cast<const i32x4*>(pa[i] + at);
    }
  };
  auto multiply = [&](int k, Set& s) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (TAIL) {
        if (k * STEP + 64 * u + 16 * g >= K)
#pragma unroll
          for (int i = 0; i < MT; ++i) s.a[u][i] = i32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(s.b[u][j], s.a[u][i], acc[i][j], 0, 0, 0);
    }
  };
  Set s0, s1;
  int k = w;
  if (k < steps) {
    load(k, s0);
    while (true) {
      if (k + NW >= steps) {
        multiply(k, s0);
        break;
      }
      load(k + NW, s1);
      multiply(k, s0);
      k += NW;
      if (k + NW >= steps) {
        multiply(k, s1);
        break;
      }
      load(k + NW, s0);
      multiply(k, s1);
      k += NW;
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[w][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  for (int at = threadIdx.x; at < MT * NT * 64; at += 64 * NW) {
    const int tile = at >> 6, l = at & 63;
    // lane l: row l % 16, columns 4 (l / 16) .. + 3
    const int r = m0 + 16 * (tile / NT) + (l & 15), c = n0 + 16 * (tile % NT) + 4 * (l >> 4);
    Columns<EPI, 4> col;
    col.load(sb, sb_vec, bias, c, N);
    const float sar = sa[sa_vec ? min(r, M - 1) : 0];
    i32x4 sum[1] = {part[0][tile][l]};
#pragma unroll
    for (int v = 1; v < NW; ++v) sum[0] += part[v][tile][l];
    if (r < M) col.store(C + (int64_t)r * ldc + c, sum, sar, N - c);
  }
}

// ---------------------------------------------------------------------------
// host launchers

template <int BM, int BN, int WM, int WN, int NSLOT, int OCC>
static hipError_t launch_tile(const GemmArgs& g, hipStream_t s) {
  const int tiles_m = (int)((g.M + BM - 1) / BM), tiles_n = (int)((g.N + BN - 1) / BN);
  return with_epi(g, [&](auto e) {
    hipLaunchKernelGGL((gemm_int8_tile_kernel<BM, BN, WM, WN, NSLOT, OCC, decltype(e)::value>),
                       grid2((int64_t)tiles_m * tiles_n, g), dim3(64 * WM * WN), 0, s, g.A, g.lda, g.B, g.ldb, g.C,
                       g.ldc, (int)g.M, (int)g.N, (int)g.K, static_cast<const float*>(g.sa), (int)(g.sa_kind == 1),
                       static_cast<const float*>(g.sb), (int)(g.sb_kind == 2), static_cast<const uint16_t*>(g.bias),
                       tiles_m, tiles_n, g.batch);
  });
}

template <int MT, int NT, int NW>
static hipError_t launch_few(const GemmArgs& g, hipStream_t s) {
  const dim3 grid((unsigned)((g.N + 16 * NT - 1) / (16 * NT)), (unsigned)g.batch.count,
                  (unsigned)((g.M + 16 * MT - 1) / (16 * MT)));
  auto go = [&](auto tail) {
    return with_epi(g, [&](auto e) {
      hipLaunchKernelGGL((gemm_int8_few_kernel<MT, NT, NW, decltype(tail)::value, decltype(e)::value>), grid,
                         dim3(64 * NW), 0, s, g.A, g.lda, g.B, g.ldb, g.C, g.ldc, (int)g.M, (int)g.N, (int)g.K,
                         static_cast<const float*>(g.sa), (int)(g.sa_kind == 1), static_cast<const float*>(g.sb),
                         (int)(g.sb_kind == 2), static_cast<const uint16_t*>(g.bias), g.batch);
    });
  };
  return g.K % 256 ? go(std::true_type{}) : go(std::false_type{});
}

// Few rows go to the streaming kernel, in panels of 16 columns while the whole batch has
// one for each CU at most; then up to 16 rows in panels of 32 columns, 17 .. 32 rows in
// tiles.  Weights from HBM, us in panels of 16 and in what follows: 16 rows x 4096 x 7168
// 10.6 and 12.8, 16 x 4352 x 4096 10.6 and 8.8 (1 row 8.3 and 7.5), 16 x 8192 x 8192 19.0
// and 16.9 (1 row 15.4 and 16.6), 32 experts of 16 x 7168 x 2048 137 and 110 (1 row 105
// and 87); 32 x 4096 x 7168 13.7 and 14.7, two of them 23.6 and 16.1, 32 experts of 32 x
// 4096 x 2048 106 and 55.  Tiles for up to 16 rows lie between 20% faster than panels of
// 32 columns (16 rows, K of 2048, more than 1800 panels) and 19% slower (1 row, K of 4096).
//
// The others go to the tile whose turns cost least: a workgroup per CU and turn, times
// what a step of 128 measured (in 10 ns, alone in its turn and with others behind it).
// Over 17 .. 8320 rows of six weights of 1 .. 116 MB this picks within 1% of the fastest tile on
// average, 15% at worst.  Of the two tiles of 128 and 64, the one with 128 rows has half as
// many workgroups read each weight (300 x 5376 x 14336: 42.0 us against 38.0), the other
// wastes less of a few rows (150 rows: 26.1 and 34.4).
enum { INT8_FEW_16X16, INT8_FEW_16X32, INT8_FEW_32X16, INT8_64X32, INT8_64X64, INT8_64X128, INT8_128X64,
       INT8_128X128_ALONE, INT8_128X128, INT8_256X256 };

int pick_int8_kernel(int64_t batches, int64_t M, int64_t N) {
  const bool one_each = (N + 15) / 16 * batches <= 256;  // panels of 16 columns, CUs
  if (M <= 16 && one_each) return INT8_FEW_16X16;
  if (M <= 16 && N <= (1 << 26)) return INT8_FEW_16X32;
  if (M <= 32 && one_each) return INT8_FEW_32X16;
  struct Tile {
    int id, bm, bn, alone, turn;
  };
  constexpr Tile tiles[] = {{INT8_64X32, 64, 32, 17, 19},     {INT8_64X64, 64, 64, 22, 22},
                            {INT8_64X128, 64, 128, 31, 33},   {INT8_128X64, 128, 64, 29, 31},
                            {INT8_128X128, 128, 128, 37, 46}, {INT8_256X256, 256, 256, 125, 150}};
  int best = INT8_256X256;
  int64_t least = INT64_MAX;
  for (int i = 5; i >= 0; --i) {
    const Tile& t = tiles[i];
    const int64_t n = ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
    const int64_t turns = (n * batches + 255) / 256;
    const int64_t cost = turns == 1 ? t.alone : turns * t.turn;
    // (a launch holds less than 2^32 threads, a workgroup up to 512; 256 x 256 always fits)
    if (n < (1 << 23) && cost < least) {
      least = cost;
      // two workgroups a CU hide each other's waits; a single one takes a deeper ring
      best = t.id == INT8_128X128 && turns == 1 ? INT8_128X128_ALONE : t.id;
    }
  }
  return best;
}

const char* int8_kernel_name(int id) {
  switch (id) {
    case INT8_FEW_16X16: return "few 16x16";
    case INT8_FEW_16X32: return "few 16x32";
    case INT8_FEW_32X16: return "few 32x16";
    case INT8_64X32: return "64x32";
    case INT8_64X64: return "64x64";
    case INT8_64X128: return "64x128";
    case INT8_128X64: return "128x64";
    case INT8_128X128_ALONE: return "128x128 alone";
    case INT8_128X128: return "128x128";
    default: return "256x256";
  }
}

hipError_t launch_gemm_int8(const GemmArgs& g, hipStream_t s) {
  switch (pick_int8_kernel(g.batch.count, g.M, g.N)) {
    case INT8_FEW_16X16: return launch_few<1, 1, 8>(g, s);
    case INT8_FEW_16X32: return launch_few<1, 2, 8>(g, s);
    case INT8_FEW_32X16: return launch_few<2, 1, 8>(g, s);
    case INT8_64X32: return launch_tile<64, 32, 2, 2, 6, 2>(g, s);
    case INT8_64X64: return launch_tile<64, 64, 2, 4, 4, 2>(g, s);
    case INT8_64X128: return launch_tile<64, 128, 2, 4, 4, 1>(g, s);
    case INT8_128X64: return launch_tile<128, 64, 4, 2, 4, 1>(g, s);
    case INT8_128X128_ALONE: return launch_tile<128, 128, 2, 4, 4, 1>(g, s);
    case INT8_128X128: return launch_tile<128, 128, 2, 4, 2, 2>(g, s);
    default: return launch_tile<256, 256, 2, 4, 2, 1>(g, s);
  }
}

}  // namespace fp8sm
