// Scaled int8 GEMM for gfx950: C[m,n] = rnd(RN32(RN32(f32(acc) * sa[m]) * sb[n]) + bias[n]),
// acc = sum_k A[m,k] B[n,k] in int32 on the int8 matrix instructions.
//
// The sum is exact (K <= 65536 products of at most 2^14 fit 31 bits), so K may be
// walked in any order and split over wavefronts: every variant gives the same
// bits.  A lane's operand of v_mfma_i32_32x32x32_i8 is 16 bytes of a row; which k
// they are does not matter as long as both operands agree.
#include "gemm_common.h"
#include "lds_copy.h"

#include <algorithm>
#include <type_traits>

namespace fp8sm {

typedef int i32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x4 to_f32(int a, int b, int c, int d) {
  return f32x4{(float)a, (float)b, (float)c, (float)d};
}

// ---------------------------------------------------------------------------
// Tile kernel.  A workgroup computes BM x BN outputs with WM x WN wavefronts; K is
// walked in chunks of 64 that copies bring into an LDS ring of NSLOT slots (BM rows
// of A, then BN rows of B), one barrier a chunk.  The barrier that makes chunk k + 1
// visible comes before chunk k's matrix work; its fragments are read into a second
// register set while chunk k is multiplied.
//
// LDS: 16-byte piece c of row r lies at c ^ swizzle(r mod 16), so that consecutive
// lanes, which read the same piece of consecutive rows, hit distinct banks.
constexpr int kTileK = 64;

__device__ __forceinline__ int swizzle64(int r) { return ((r >> 1) ^ (r >> 3)) & 3; }

template <int BM, int BN, int WM, int WN, int NSLOT, int OCC, int EPI>
__global__ __launch_bounds__(64 * WM * WN, OCC * WM * WN / 4) void gemm_int8_tile_kernel(
    const uint8_t* __restrict__ A, int64_t lda, const uint8_t* __restrict__ B, int64_t ldb,
    uint16_t* __restrict__ C, int64_t ldc, int M, int N, int K, const float* __restrict__ sa,
    int sa_vec, const float* __restrict__ sb, int sb_vec, const uint16_t* __restrict__ bias,
    int tiles_m, int tiles_n, GemmBatch gb) {
  constexpr int NW = WM * WN, TM = BM / WM / 32, TN = BN / WN / 32;
  constexpr int SLOT = (BM + BN) * kTileK;
  constexpr int CPW = SLOT / 1024 / NW;  // copies of a wavefront a chunk: 16 rows of 64 bytes each
  static_assert(TM * 32 * WM == BM && TN * 32 * WN == BN && CPW * NW * 1024 == SLOT, "tile shape");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NSLOT * SLOT];

  int tm, tn;
  tile_coords(blockIdx.x, gridDim.x, tiles_m, tiles_n, tm, tn);
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
  const int lane = threadIdx.x & 63, x = lane & 31, h = lane >> 5;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / WN, wn = w % WN;
  const uint32_t lds0 = lds_address(lds);

  // Copy i of wavefront w brings 16 rows from row 16 (NW i + w) of the slot on; lane l
  // row l / 4, piece l % 4 of its slot.  Rows past M / N repeat the last one.  A
  // buffer ends at K of its last row: pieces past K of that row come as zeros, those
  // of the others as what follows in memory, and `read` drops both.
  i32x4 rs[CPW];
  uint32_t vo[CPW];
#pragma unroll
  for (int i = 0; i < CPW; ++i) {
    const int seg = i * NW + w, r = lane >> 2;
    const bool isa = seg * 16 < BM;
    const int64_t ld = isa ? lda : ldb;
    const int first = isa ? m0 + seg * 16 : n0 + seg * 16 - BM, last = (isa ? M : N) - 1;
    const int r0 = min(first, last), rr = min(first + r, last);
    // (16 rows of at most 2^24 bytes: below 2^31)
    rs[i] = raw_buffer((isa ? A : B) + (int64_t)r0 * ld, (uint32_t)((min(first + 15, last) - r0) * ld) + (uint32_t)K);
    vo[i] = (uint32_t)((rr - r0) * ld) + (uint32_t)(((lane & 3) ^ swizzle64(r)) * 16);
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
  // waits for the copies of chunk k, `ahead` younger ones may be on their way
  auto arrive = [&](int ahead) {
    if (NSLOT > 3 && ahead >= 2)
      wait_copies_but<2 * CPW>();
    else if (NSLOT > 2 && ahead >= 1)
      wait_copies_but<CPW>();
    else
      wait_copies_but<0>();
    __syncthreads();
  };

  const int piece0 = ((2 * h) ^ swizzle64(x & 15)) * 16, piece1 = ((2 * h + 1) ^ swizzle64(x & 15)) * 16;
  const int a_row = (wm * (BM / WM) + x) * kTileK, b_row = (BM + wn * (BN / WN) + x) * kTileK;
  struct Frag {
    i32x4 q[2];
  };
  auto read = [&](int k, Frag(&fa)[TM], Frag(&fb)[TN]) {
    const uint8_t* slot = lds + (k % NSLOT) * SLOT;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      fa[i].q[0] = *reinterpret_cast<const i32x4*>(slot + a_row + i * 32 * kTileK + piece0);
      fa[i].q[1] = *reinterpret_cast<const i32x4*>(slot + a_row + i * 32 * kTileK + piece1);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      fb[j].q[0] = *reinterpret_cast<const i32x4*>(slot + b_row + j * 32 * kTileK + piece0);
      fb[j].q[1] = *reinterpret_cast<const i32x4*>(slot + b_row + j * 32 * kTileK + piece1);
    }
    if ((k + 1) * kTileK > K) {  // K % 64 != 0: k past K counts nothing (zeros on one side)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (k * kTileK + 32 * h + 16 * p >= K)
#pragma unroll
          for (int i = 0; i < TM; ++i) fa[i].q[p] = i32x4{0, 0, 0, 0};
    }
  };
  i32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  // B first: a lane gets four consecutive columns of its output row
  auto multiply = [&](const Frag(&fa)[TM], const Frag(&fb)[TN]) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j].q[p], fa[i].q[p], acc[i][j], 0, 0, 0);
  };

  Frag fa0[TM], fb0[TN], fa1[TM], fb1[TN];
  for (int k = 0; k < NSLOT - 1 && k < nk; ++k) issue(k);
  arrive(min(NSLOT - 2, nk - 1));
  if (NSLOT - 1 < nk) issue(NSLOT - 1);
  read(0, fa0, fb0);
  auto step = [&](int k, const Frag(&fa)[TM], const Frag(&fb)[TN], Frag(&na)[TM], Frag(&nb)[TN]) {
    if (k + 1 < nk) {
      arrive(min(NSLOT - 2, nk - 2 - k));
      if (k + NSLOT < nk) issue(k + NSLOT);  // into chunk k's slot: everybody has read it
      read(k + 1, na, nb);
    }
    multiply(fa, fb);
  };
  int k = 0;
  for (; k + 1 < nk; k += 2) {
    step(k, fa0, fb0, fa1, fb1);
    step(k + 1, fa1, fb1, fa0, fb0);
  }
  if (k < nk) step(k, fa0, fb0, fa1, fb1);

  // lane (x, h): row x of each row subtile, columns 8v + 4h .. + 3 of each column
  // subtile in registers 4v .. 4v + 3
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const int r = m0 + wm * (BM / WM) + 32 * i + x;
    if (r >= M) continue;
    const float sar = sa[sa_vec ? r : 0];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int c = n0 + wn * (BN / WN) + 32 * j + 8 * v + 4 * h;
        if (c >= N) continue;
        const i32x16& t = acc[i][j];
        store_row4<EPI>(C, ldc, r, c, to_f32(t[4 * v], t[4 * v + 1], t[4 * v + 2], t[4 * v + 3]), sar, sb, sb_vec, bias);
      }
  }
}

// ---------------------------------------------------------------------------
// Few rows: 16 MT rows x 16 NT columns a workgroup.  The weights are streamed once
// and that stream is the bound, so operands go straight from memory to registers and
// the NW wavefronts split K, 256 at a time, each with the next 256 on their way; the
// partial sums are added in LDS.  v_mfma_i32_16x16x64_i8: lane l holds 16 bytes
// from k = 16 (l / 16) on of row l % 16.
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
      for (int j = 0; j < NT; ++j) s.b[u][j] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(pb[j] + at));
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
    i32x4 sum = part[0][tile][l];
#pragma unroll
    for (int v = 1; v < NW; ++v) sum += part[v][tile][l];
    // lane l: row l % 16, columns 4 (l / 16) .. + 3
    const int r = m0 + 16 * (tile / NT) + (l & 15), c = n0 + 16 * (tile % NT) + 4 * (l >> 4);
    if (r < M && c < N)
      store_row4<EPI>(C, ldc, r, c, to_f32(sum[0], sum[1], sum[2], sum[3]), sa[sa_vec ? r : 0], sb, sb_vec, bias);
  }
}

// ---------------------------------------------------------------------------
// host launchers

template <int BM, int BN, int WM, int WN, int NSLOT, int OCC>
static hipError_t launch_tile(const GemmArgs& g, hipStream_t s) {
  const int tiles_m = (int)((g.M + BM - 1) / BM), tiles_n = (int)((g.N + BN - 1) / BN);
  return with_epi(g, [&](auto e) {
    hipLaunchKernelGGL((gemm_int8_tile_kernel<BM, BN, WM, WN, NSLOT, OCC, decltype(e)::value | EPI_STEPS>),
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
      hipLaunchKernelGGL((gemm_int8_few_kernel<MT, NT, NW, decltype(tail)::value, decltype(e)::value | EPI_STEPS>), grid,
                         dim3(64 * NW), 0, s, g.A, g.lda, g.B, g.ldb, g.C, g.ldc, (int)g.M, (int)g.N, (int)g.K,
                         static_cast<const float*>(g.sa), (int)(g.sa_kind == 1), static_cast<const float*>(g.sb),
                         (int)(g.sb_kind == 2), static_cast<const uint16_t*>(g.bias), g.batch);
    });
  };
  return g.K % 256 ? go(std::true_type{}) : go(std::false_type{});
}

hipError_t launch_gemm_int8(const GemmArgs& g, hipStream_t s) {
  // (a launch holds less than 2^32 threads)
  if (g.M <= 64 && g.N <= (1 << 26)) {
    if (g.M <= 16) return launch_few<1, 2, 8>(g, s);
    if (g.M <= 32) return launch_few<2, 2, 8>(g, s);
    return launch_few<4, 2, 8>(g, s);
  }
  if (g.M * g.N >= (int64_t)256 * 256 * 256) return launch_tile<256, 256, 2, 4, 4, 1>(g, s);
  return launch_tile<128, 128, 2, 2, 4, 2>(g, s);
}

}  // namespace fp8sm
