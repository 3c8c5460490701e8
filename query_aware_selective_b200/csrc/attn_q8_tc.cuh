// attn_q8_tc.cuh - exact attention of few queries over an 8-bit cache of head dim 128 on
// the fifth-generation tensor cores (sm_100a tcgen05), codes fed to them as they are.
//
// The formulas are those of attn_q8.cuh. Both products take the codes as the M = 128 side
// of an 8-bit MMA straight from shared memory, without any conversion:
//   S^T [128 keys x N] = K [128 x 128] Q^T    (A: K rows, K-major)
//   O^T [128 dims x N] = V^T [128 x 128] W^T  (A: V rows read M-major; B: W N-major, so a
//                                              thread stores its key's pieces side by side)
// kind::f8f6f4 for e4m3 (fp32 sums), kind::i8 for int8 (exact 32-bit sums). Queries and
// weights go in as P pieces of 8 bits, each its own column:
//   e4m3: piece p = e4m3(16^p (x - pieces before)), 4 significant bits each: two for a bf16
//         query, three for a weight (relative 2^-13), four with up to 8 query rows (2^-17: the
//         columns are there anyway, N is a multiple of 16, and the rows are few; 16 sequences
//         of 4 rows 38.9 -> 39.1 us. With 20 rows the fourth took 40.4 -> 42.2 us, with 400
//         71 -> 75)
//   int8: digits of 7 bits of an integer: three for a query (its row's largest is 2^19 to
//         2^20), four for a weight (its tile's largest is 2^27)
// (a query's element to 2^-21 or 2^-20 of its row's largest: bf16's 8 bits are whole down to
// 2^-12 of that, and one more piece would be a column to load and to add for each key and row)
// and a row's value is the sum of its columns times 2^(-4 p) or 2^(-7 p). Column (rg NW + p)
// WR + r is piece p of row r of row group rg.
// Weights are taken relative to their key tile's own maximum (of 128 keys), and a tile's O
// is drained from TMEM into fp32 registers and scaled there: the range of 8-bit pieces
// then only has to span one tile (a weight is rounded to 2^-26 or 2^-30 (e4m3) or 2^-28 (int8)
// of its tile's largest at worst; three int8 digits, 2^-21, showed in dims where the largest
// weight's value is next to zero), and nothing in TMEM is ever rescaled. The maximum is
// that of x_j + log2 b_j, and a weight e_j b_j with e_j = 2^(x_j - maximum); l sums the e_j (as in
// attn_q8.cuh: b_j spans 2^198, which a weight does not hold).
//
// Roles: one to three softmax warpgroups (thread = key for S and W, thread = dim for O; up to
// 8 query rows each, and with few rows two that take turns at the key tiles), one warp that
// issues the MMAs, two that copy keys, values and scales (16-byte cp.async, 8 lanes a row,
// into 128-byte-swizzled tiles). TMEM: four buffers of S (two where N leaves no room), two of
// O. A CTA takes a share of one (sequence, KV head)'s key list; at the end each CTA of a
// cluster sends every other its part of their dims and merges its own.
//
// Bound by HBM with up to 8 rows: 16 sequences x 6.3K keys x 8 heads (206 MB, a CTA per
// sequence and head) take 39.2 us (int8 38.8), 5.3 TB/s; the loop alone streams at 6.4 TB/s, 2.7 us go
// to the launch, the queries and the first keys, 1.8 us to the last tile and the merge, and
// 128 units leave 20 of 148 SMs idle. One CTA of six stages an SM beat two of three, 39.7
// against 42 us. With more rows bound by the softmax warps' issue slots: 20 rows x 24 units
// (39 MB) take 20.7 us, a tile of 128 keys 2400 cycles (12 warps in step: 340 waiting for
// barriers that are complete, 850 to the tile's maxima, 800 for weights and pieces, 450 each
// to store them and to read O). (Converted to f16 for mma.sync, as
// attn_q8.cuh does, the same keys took 70 and 77 us: the conversions cost more issue slots
// than the softmax.)
#pragma once
#include "attn_q8.cuh"
#include "common.cuh"
#include "keylist.cuh"

namespace esa {

constexpr int kQtKeys = 128;
constexpr uint32_t kQtTile = 128 * 128;                       // bytes of a key or value tile
constexpr uint32_t kQtStage = 2 * kQtTile + 2 * kQtKeys * 4;  // keys, values, their scales
constexpr int kQtMaxCluster = 8;

// RG row groups of WR query rows (RT rows of a tile) times TG tile groups: the warpgroup of
// row group rg and tile group tg takes those rows of the key tiles j with j % TG == tg.
template <int FMT, int WR, int RG, int TG>
struct QtShape {
  static constexpr int RT = WR * RG;
  static constexpr int NQ = FMT == kQ8E4M3 ? 2 : 3, NW = FMT == kQ8E4M3 && RT > 8 ? 3 : 4;   // pieces of a query, of a weight
  static constexpr int N = (NW * RT + 15) / 16 * 16;          // MMA columns (M = 128: a multiple of 16)
  static constexpr int kThreads = (4 * RG * TG + 3) * 32;
  static constexpr int kStages = RT <= 8 ? 6 : 5;
  static constexpr int NS = 6 * N <= 512 ? 4 : 2;             // score buffers in TMEM (O: two behind them)
  static constexpr uint32_t kCols = (NS + 2) * N <= 128 ? 128 : (NS + 2) * N <= 256 ? 256 : 512;   // TMEM columns
  static constexpr uint32_t kQ = kStages * kQtStage, kW = kQ + N * 128, kCtrl = kW + 2 * N * 128;
  // behind the control block, in floats: tile maxima [TG][2][4][RT], logit factors [RT], l of
  // each warp [TG][4][RT], and what the warpgroups of the cluster's CTAs send: (m, l)
  // [8 TG][RT][2], o [RT][csize TG][dims of this CTA]
  static constexpr int kMax = 0, kXs = 8 * TG * RT, kL = kXs + RT, kMl = kL + 4 * TG * RT + (RT & 4 ? 4 : 0);
  static constexpr int kO = kMl + 2 * kQtMaxCluster * TG * RT, kOFloats = 160 * TG * RT;   // csize * q8_dims_per <= 160
  static constexpr uint32_t kRing = kCtrl + 256 + (kO + kOFloats) * 4;                     // list entries [stage][128]
  static constexpr uint32_t kSmem = kRing + kStages * 512;
  // a warpgroup sees every phase of the barriers it waits for
  static_assert(kStages % TG == 0 && NS % TG == 0 && 2 % TG == 0, "stages and buffers that the tile groups share");
  static_assert((WR == 4 && RG == 1 && NW == 4) || (WR == 8 && N - NW * RT <= 8), "columns of a weight's stores");
  static_assert(kSmem <= 232448 && (NS + 2) * N <= 512 && (kMl * 4) % 16 == 0 && (kO * 4) % 16 == 0, "does not fit an SM");
};

struct QtCtrl {
  uint64_t full[6], empty[6], s_full[4], w_full[2], o_full[2], q_full, mma_done;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(QtCtrl) <= 256, "control block overflows its reservation");

// D[tmem] (+)= A[smem] * B[smem]^T on 8-bit codes, issued by one elected lane of a converged
// warp (descriptors as low and high words: only the low one moves).
template <int FMT>
__device__ __forceinline__ void umma_q8_elect(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo,
                                              uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
  if constexpr (FMT == kQ8E4M3) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "mov.b64 da, {%1, %2};\n\t"
        "mov.b64 db, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate));
  } else {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "mov.b64 da, {%1, %2};\n\t"
        "mov.b64 db, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::i8 [%0], da, db, %5, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate));
  }
}
// Instruction descriptor: e4m3 x e4m3 -> fp32, or s8 x s8 -> s32.
template <int FMT>
__host__ __device__ constexpr uint32_t q8_idesc(uint32_t n, uint32_t mn_major) {
  return FMT == kQ8E4M3 ? umma_idesc(0, 128, n, mn_major, mn_major)
                        : (2u << 4) | (1u << 7) | (1u << 10) | (mn_major << 15) | (mn_major << 16) | ((n >> 3) << 17) |
                              (8u << 24);
}
// Descriptor of an operand without swizzle: 8 x 16-byte core matrices, here MN-major (a row
// of 16 bytes is 16 columns of one k): next 8 k at k_bytes, next 16 columns at mn_bytes.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t saddr, uint32_t k_bytes, uint32_t mn_bytes) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((k_bytes >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((mn_bytes >> 4) & 0x3FFFu) << 32) | ((uint64_t)1 << 46);
}

__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Whether both phases have completed, in the time of one test.
__device__ __forceinline__ bool mbar_test_both(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 q, [%3], %4;\n\t"
      "and.pred p, p, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// NC columns (a multiple of 4) of a TMEM buffer, this thread's lane
template <int NC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t (&v)[NC]) {
#pragma unroll
  for (int c = 0; c + 8 <= NC; c += 8) tmem_ld8(addr + c, v + c);
  if constexpr (NC % 8 == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[NC - 4]), "=r"(v[NC - 3]), "=r"(v[NC - 2]), "=r"(v[NC - 1])
                 : "r"(addr + NC - 4));
  tmem_wait_ld();
}
__device__ __forceinline__ void st_dsmem_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// A row's value from its pieces (v[p * WR + r]): in units of piece 0, or of piece 1 for four
// digits. Digits are joined in pairs as integers (sums of 128 products: 2^21, 2^28 joined).
template <int FMT, int WR, int NP>
__device__ __forceinline__ float q8_join(const uint32_t* v, int r) {
  if constexpr (FMT == kQ8E4M3) {
    float x = __uint_as_float(v[(NP - 1) * WR + r]);
#pragma unroll
    for (int p = NP - 2; p >= 0; --p) x = fmaf(x, 0.0625f, __uint_as_float(v[p * WR + r]));
    return x;
  } else {
    static_assert(NP == 3 || NP == 4);
    const int lo = (int)v[(NP - 2) * WR + r] * 128 + (int)v[(NP - 1) * WR + r];
    const int hi = NP == 3 ? (int)v[r] : (int)v[r] * 128 + (int)v[WR + r];
    return fmaf((float)lo, 0x1p-14f, (float)hi);
  }
}
// Two values as pieces: byte 0 of pc[p] is piece p of x0, byte 1 of x1. e4m3: |x| <= 448;
// int8: |x| < 2^(7 NP), in digits of 7 bits (the first signed, the others 0 .. 127).
template <int FMT, int NP>
__device__ __forceinline__ void q8_split2(float x0, float x1, uint32_t* pc) {
  if constexpr (FMT == kQ8E4M3) {
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      uint16_t c;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x1), "f"(x0));
      pc[p] = c;
      if (p + 1 < NP) {
        const float2 f = f16x2_to_float2(e4m3x2_to_f16x2(c));
        x0 = (x0 - f.x) * 16.f;
        x1 = (x1 - f.y) * 16.f;
      }
    }
  } else {
    const int i0 = __float2int_rn(x0), i1 = __float2int_rn(x1);
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const int sh = 7 * (NP - 1 - p);
      const uint32_t d0 = p ? (i0 >> sh) & 127 : (i0 >> sh) & 255, d1 = p ? (i1 >> sh) & 127 : (i1 >> sh) & 255;
      pc[p] = d0 | (d1 << 8);
    }
  }
}
// Four weights >= 0 (a row each) as pieces: byte r of pc[p] is piece p of x[r].
template <int FMT, int NP>
__device__ __forceinline__ void q8_split4(const float* x, uint32_t* pc) {
  if constexpr (FMT == kQ8E4M3) {
    uint32_t lo[NP], hi[NP];
    q8_split2<FMT, NP>(x[0], x[1], lo);
    q8_split2<FMT, NP>(x[2], x[3], hi);
#pragma unroll
    for (int p = 0; p < NP; ++p) pc[p] = __byte_perm(lo[p], hi[p], 0x5410);
  } else {
    // 28 bits spread to four bytes of 7: the halves first, then the digits of both (sums of
    // bits that do not meet), and the 4 x 4 bytes transposed
    static_assert(NP == 4);
    uint32_t y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t i = (uint32_t)__float2int_rn(x[r]);
      const uint32_t t = (i & 0x0fffc000u) * 3u + i;
      y[r] = t + (t & 0x3f803f80u);
    }
    const uint32_t a = __byte_perm(y[0], y[1], 0x5140), b = __byte_perm(y[2], y[3], 0x5140);
    const uint32_t c = __byte_perm(y[0], y[1], 0x7362), d = __byte_perm(y[2], y[3], 0x7362);
    pc[0] = __byte_perm(c, d, 0x7632);
    pc[1] = __byte_perm(c, d, 0x5410);
    pc[2] = __byte_perm(a, b, 0x7632);
    pc[3] = __byte_perm(a, b, 0x5410);
  }
}

// Dims that each CTA of a cluster merges, a multiple of 4 (the last CTA the rest, if any).
__device__ __forceinline__ int q8_dims_per(int csize) { return ((128 + csize - 1) / csize + 3) & ~3; }

// grid (cluster size, Hkv * tiles, B), cluster (cluster size, 1, 1).
template <int FMT, int WR, int RG, int TG>
__global__ void __launch_bounds__((QtShape<FMT, WR, RG, TG>::kThreads), 1) attn_q8_tc_kernel(const AttnQ8Args a) {
  using Sh = QtShape<FMT, WR, RG, TG>;
  constexpr int RT = Sh::RT, N = Sh::N, NST = Sh::kStages, NS = Sh::NS, NQ = Sh::NQ, NW = Sh::NW;
  constexpr int kMmaWarp = 4 * RG * TG, kProdWarp = kMmaWarp + 1, kSoftThreads = 128 * RG * TG;
  constexpr int kBarTmem = RG * TG + 1, kBarQ = RG * TG + 2;      // named barriers (1 .. RG * TG: the warpgroups)
  // a tile's largest weight goes in as 2^8 (e4m3, <= 448), 2^27 (int8, <= 127 * 2^21)
  constexpr float kTop = FMT == kQ8E4M3 ? 0x1p8f : 0x1p27f;
  // units of q8_join for a query and for a weight
  constexpr float kUnitQ = FMT == kQ8E4M3 ? 1.f : 0x1p14f, kUnitW = FMT == kQ8E4M3 ? 1.f : 0x1p14f;
  extern __shared__ __align__(1024) uint8_t qtsm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(qtsm);
  QtCtrl& sm = *reinterpret_cast<QtCtrl*>(qtsm + Sh::kCtrl);
  float* const smf = reinterpret_cast<float*>(qtsm + Sh::kCtrl + 256);
  float* const sm_l = smf + Sh::kL;
  float* const sm_xs = smf + Sh::kXs;

  const int g = blockIdx.y / a.tiles, tile = blockIdx.y - g * a.tiles, b = blockIdx.z;
  const int rank = blockIdx.x, csize = gridDim.x;
  const int list = a.lists > 1 ? b * a.lists + g : b;
  KeyList kl = a.keys;
  pdl_wait();
  const int64_t c0 = kl.vl.len ? kl.resolve(b, 706) : a.c0;
  const int ni = (int)kl.ni;
  // Key slot `row` of tile j of this CTA (tiles rank, rank + csize, ...: every CTA gets its
  // share of the scattered keys, which load slower than the consecutive ones: with
  // consecutive shares the CTA of the local tokens waited 11 of 45 us for its peer), and the
  // place of its list entry, if it has one. Entries (loads that may miss all the way to HBM)
  // do not wait for the list's length.
  auto slot_t = [&](int j, int row) { return (j * csize + rank) * kQtKeys + row; };
  auto entry = [&](int j, int row) {
    return kl.idx + (int64_t)list * kl.idx_stride + min(max(slot_t(j, row) - ni, 0), (int)kl.idx_stride - 1);
  };
  const int prow = (warp - kProdWarp) * 64 + lane;  // producer lanes: rows prow and prow + 32 of a tile
  int32_t raw[NST][2];
  if (warp >= kProdWarp) {
#pragma unroll
    for (int u = 0; u < NST; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) raw[u][h] = *entry(u, prow + 32 * h);
  }
  // queries: thread (r, part) of the first tile group takes DPT dims of row r, loaded now for
  // the time that the list's length and the setup take
  constexpr int TPR = 128 / WR, DPT = 128 / TPR;
  const int q_row = (warp >> 2) % RG * WR + (threadIdx.x & 127) / TPR, q_part = (threadIdx.x & 127) % TPR;
  uint2 q_raw[DPT / 4];
  if (warp < 4 * RG) {
    const int rr = min(tile * RT + q_row, a.lq * a.G - 1), i = rr / a.G, hl = rr - i * a.G;
    const uint2* qp = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) +
        (((int64_t)b * a.lq + i) * a.hq + g * a.G + hl) * 128 + q_part * DPT);
#pragma unroll
    for (int e = 0; e < DPT / 4; ++e) q_raw[e] = qp[e];
  }
  const int32_t n_listed = kl.count[list];
  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 64);                   // every producer thread, when its copies have landed
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < NS; ++s) mbar_init(&sm.s_full[s], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.w_full[s], 4 * RG);
      mbar_init(&sm.o_full[s], 1);
    }
    mbar_init(&sm.q_full, 4 * RG);
    mbar_init(&sm.mma_done, 1);
    sm.abort_flag = base & 1023u ? 1 : 0;
    if (base & 1023u) record_status(5u, 710);
    fence_barrier_init();
  }
  __syncthreads();
  if (csize > 1) cluster_arrive();                  // this CTA runs: its shared memory may be written to
  const int cnt = min(max(n_listed, 0), (int)kl.idx_stride);
  const int n_prior = (int)(kl.ni + cnt + (c0 - kl.lo));
  const int r0 = tile * RT, nrow = min(RT, a.lq * a.G - r0);
  const int n_keys = n_prior + (r0 + nrow - 1) / a.G + 1;      // that the tile's last row attends
  const int n_all = n_prior + r0 / a.G + 1;                    // that every row of the tile attends
  const int tiles_all = (n_keys + kQtKeys - 1) / kQtKeys;
  const int nt = rank < tiles_all ? (tiles_all - rank - 1) / csize + 1 : 0;   // this CTA's key tiles
  volatile int* abort_flag = &sm.abort_flag;
  // TMEM is the softmax and MMA warps' business: the producers are off already
  uint32_t tmem = 0;
  if (warp <= kMmaWarp) {
    if (warp == kMmaWarp) {
      tmem_alloc(&sm.tmem_base, Sh::kCols);
      tmem_relinquish();
    }
    tc_fence_before();
    asm volatile("bar.sync %0, %1;" ::"n"(kBarTmem), "n"(kSoftThreads + 32) : "memory");
    tc_fence_after();
    tmem = sm.tmem_base;
  }

  float o[WR], l[WR];
  float m = -INFINITY;                              // of row lane % WR
#pragma unroll
  for (int r = 0; r < WR; ++r) {
    o[r] = 0.f;
    l[r] = 0.f;
  }

  if (base & 1023u) {
    // misaligned shared memory: reported, nothing done
    if (csize > 1 && warp < kMmaWarp) cluster_wait();
  } else if (warp >= kProdWarp) {
    // ------------------------------------------------------------------- producers
    const uint32_t row_bytes = (uint32_t)a.hkv * 128;
    const int pw = warp - kProdWarp, c = lane & 7, lr = lane >> 3;
    const uint8_t* kb = a.k + (int64_t)b * a.n_cap * row_bytes + g * 128 + c * 16;
    const uint8_t* vb = a.v + (int64_t)b * a.n_cap * row_bytes + g * 128 + c * 16;
    const float* ksb = a.ks + (int64_t)b * a.nblk * a.hkv + g;
    const float* vsb = a.vs + (int64_t)b * a.nblk * a.hkv + g;
    const int jump = (int)(kl.lo - kl.ni) - cnt;
    // Later entries are copied a ring ahead, with tile j - NST, into shared memory, where each
    // lane reads back its own: the stage of tile j is free only after those copies have landed.
    const uint32_t ring = base + Sh::kRing + prow * 4;
#pragma unroll
    for (int u = 0; u < NST; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(ring + u * 512 + h * 128), "r"(raw[u][h]) : "memory");
    const uint32_t sw0 = (uint32_t)(pw * 64 + lr) * 128 + ((c ^ lr) << 4);            // rows 8 i + lr
    const uint32_t sw1 = (uint32_t)(pw * 64 + 4 + lr) * 128 + ((c ^ (4 + lr)) << 4);  // rows 8 i + 4 + lr
    int s = 0;
    for (int j = 0; j < nt; ++j, s = s + 1 == NST ? 0 : s + 1) {
      if (!mbar_wait_warp(&sm.empty[s], ((j / NST) & 1) ^ 1, abort_flag, 707)) break;
      const uint32_t kd = base + s * kQtStage, vd = kd + kQtTile;
      int pos[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = min(slot_t(j, prow + 32 * h), n_keys - 1);             // behind the list: its last key
        const int e = (int)lds32(ring + s * 512 + h * 128);
        const int p = t < ni ? t : (t < ni + cnt ? e : t + jump);
        pos[h] = min(max(p, 0), (int)a.n_cap - 1);
        cp_async4(ring + s * 512 + h * 128, entry(j + NST, prow + 32 * h));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint64_t off = (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, pos[h], 4 * i + lr) * row_bytes;
          const uint32_t d = (i & 1 ? sw1 : sw0) + (h * 4 + (i >> 1)) * 1024;
          cp_async16(kd + d, kb + off, 16u);
          cp_async16(vd + d, vb + off, 16u);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint64_t so = (uint64_t)(uint32_t)(pos[h] >> a.bshift) * (uint32_t)a.hkv;
        const uint32_t d = vd + kQtTile + (pw * 64 + h * 32 + lane) * 4;
        cp_async4(d, ksb + so);
        cp_async4(d + kQtKeys * 4, vsb + so);
      }
      cp_async_arrive(&sm.full[s]);
    }
    cp_async_wait_all();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------- MMA issuer
    // The warp runs converged and one elected lane issues (by lane 0 alone, in a branch, the
    // four MMAs and two commits of a product took 800 cycles: the pace of the whole kernel).
    constexpr uint32_t idesc_s = q8_idesc<FMT>(N, 0), idesc_o = q8_idesc<FMT>(N, 1);        // (A, and with it B, MN-major)
    const uint64_t dsc = sdesc_sw128(base, 16, 1024);
    const uint32_t d_lo = (uint32_t)dsc, d_hi = (uint32_t)(dsc >> 32);     // of the start of shared memory
    const uint64_t wsc = sdesc_plain(base + Sh::kW, 128, 2048);            // 8 keys: 128 bytes; 16 columns: 2 KB
    const uint32_t w_lo0 = (uint32_t)wsc, w_hi = (uint32_t)(wsc >> 32);
    bool ok = nt == 0 || mbar_wait_warp(&sm.q_full, 0, abort_flag, 709);
    // Whichever is ready next: O of tile jp (its weights are written), or S of tile js (its
    // codes have landed, and js < jp + NS: the scores that were in its buffer have been read,
    // as the weights of tile js - NS say). Waiting for the two in a fixed order held O_j, and
    // with it the release of a stage, until tile j + 1 had landed; with NS of 2 a warpgroup
    // waited for its own O before it got new scores.
    int js = 0, jp = 0, ss = 0, sp = 0;                                    // tiles and their stages
    uint32_t fs = 0;                                                       // phase of full[ss]
    uint64_t since = globaltimer_ns();
    for (uint32_t spin = 0; ok && jp < nt;) {
      if (jp < js && __all_sync(0xffffffffu, mbar_test_wait(&sm.w_full[jp & 1], (jp >> 1) & 1))) {
        tc_fence_after();
        const uint32_t v_lo = d_lo + ((sp * kQtStage + kQtTile) >> 4), w_lo = w_lo0 + (((jp & 1) * N * 128) >> 4);
        const uint32_t d = tmem + (NS + (jp & 1)) * N;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)              // 32 keys: four 8-row groups of V and of W
          umma_q8_elect<FMT>(d, v_lo + kk * 256, d_hi, w_lo + kk * 32, w_hi, idesc_o, kk > 0);
        umma_commit_elect(&sm.o_full[jp & 1]);
        umma_commit_elect(&sm.empty[sp]);
        ++jp;
        sp = sp + 1 == NST ? 0 : sp + 1;
        spin = 0;
      } else if (js < nt && js < jp + NS && __all_sync(0xffffffffu, mbar_test_wait(&sm.full[ss], fs))) {
        fence_proxy_async();                        // cp.async wrote through the generic proxy
        tc_fence_after();
        const uint32_t k_lo = d_lo + ((ss * kQtStage) >> 4), q_lo = d_lo + (Sh::kQ >> 4);
        const uint32_t d = tmem + (js % NS) * N;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_q8_elect<FMT>(d, k_lo + kk * 2, d_hi, q_lo + kk * 2, d_hi, idesc_s, kk > 0);
        umma_commit_elect(&sm.s_full[js % NS]);
        ++js;
        if (++ss == NST) {
          ss = 0;
          fs ^= 1;
        }
        spin = 0;
      } else if (spin++ == 0) {
        since = globaltimer_ns();
      } else if ((spin & 255u) == 0) {
        bool stop = *abort_flag;
        if (!stop && globaltimer_ns() - since > ESA_WAIT_LIMIT_NS) {
          *abort_flag = 1;
          if (lane == 0) record_status(4u, 708);
          stop = true;
        }
        ok = !__any_sync(0xffffffffu, stop);
      }
    }
    // every MMA issued so far has completed before TMEM and shared memory are reused
    umma_commit_elect(&sm.mma_done);
    mbar_wait(&sm.mma_done, 0, abort_flag, 714, /*respect_abort=*/false);
    __syncwarp();
  } else {
    // ------------------------------------------------------------------- softmax warps
    const int rg = (warp >> 2) % RG, tg = (warp >> 2) / RG;
    const int key = threadIdx.x & 127;                    // key of a tile, for S and W; the dim, for O
    const uint32_t bar_wg = 1 + (warp >> 2);              // named barrier of the warpgroup
    const int row_wg = rg * WR;                           // its first row of the tile
    float xs[WR];                                   // logit factor of each row
    if (tg == 0) {
      // queries as pieces
      const int r = q_row, part = q_part;
      float f[DPT];
      uint32_t mx = 0;                              // largest magnitude, as bits (in the order of the values)
#pragma unroll
      for (int e = 0; e < DPT; e += 4) {
        const float2 f01 = bf16x2_to_float2(q_raw[e / 4].x), f23 = bf16x2_to_float2(q_raw[e / 4].y);
        f[e] = f01.x; f[e + 1] = f01.y; f[e + 2] = f23.x; f[e + 3] = f23.y;
#pragma unroll
        for (int u = 0; u < 4; ++u) mx = max(mx, __float_as_uint(f[e + u]) & 0x7fffffffu);
      }
#pragma unroll
      for (int w = TPR < 32 ? TPR / 2 : 16; w > 0; w >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      // 2^qe brings the row's largest to [2^7, 2^8) (e4m3) or [2^19, 2^20) (int8). Pieces hold no
      // infinity (nor, as digits, NaN): a row with one gets a factor of NaN.
      const int qe = min((FMT == kQ8E4M3 ? 7 : 19) - ((int)(mx >> 23) - 127), 100);
      const float up = __uint_as_float((uint32_t)(qe + 127) << 23);
      if (part == 0)
        sm_xs[r] = mx >= 0x7f800000u ? NAN : a.scale_log2 * kUnitQ * __uint_as_float((uint32_t)(127 - qe) << 23);
      const uint32_t q0 = base + Sh::kQ;
#pragma unroll
      for (int e = 0; e < DPT; e += 4) {
        uint32_t pc[2][NQ];
        q8_split2<FMT, NQ>(f[e] * up, f[e + 1] * up, pc[0]);
        q8_split2<FMT, NQ>(f[e + 2] * up, f[e + 3] * up, pc[1]);
        const int d = part * DPT + e;
#pragma unroll
        for (int p = 0; p < NW; ++p) {
          const uint32_t n = (rg * NW + p) * WR + (r - row_wg);
          const uint32_t v = p < NQ ? pc[0][p < NQ ? p : 0] | (pc[1][p < NQ ? p : 0] << 16) : 0u;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(q0 + n * 128 + (((d >> 4) ^ (n & 7)) << 4) + (d & 15)), "r"(v)
                       : "memory");
        }
      }
      // columns that belong to no piece are zero
      if constexpr (N > NW * RT)
        for (int z = threadIdx.x; z < (N - NW * RT) * 8; z += 128 * RG)
          st_shared_v4(q0 + NW * RT * 128 + z * 16, 0u, 0u, 0u, 0u);
      fence_proxy_async();
      mbar_arrive_warp(&sm.q_full);
    }
    asm volatile("bar.sync %0, %1;" ::"n"(kBarQ), "n"(kSoftThreads) : "memory");
#pragma unroll
    for (int q = 0; q < WR; ++q) xs[q] = sm_xs[row_wg + q];
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16) + rg * NW * WR;
    float al[WR], be[WR];                           // the tile's factors on o and on its own O
    const int row_own = lane % WR;                  // this lane finds them for one row
    auto spin_warp = [&](uint64_t* bar, uint32_t parity, unsigned site) -> bool {
      return __all_sync(0xffffffffu, mbar_wait_spin(bar, parity, abort_flag, site));
    };
    auto drain = [&](int j) -> bool {               // o = o al + O_j be
      if (!spin_warp(&sm.o_full[j & 1], (j >> 1) & 1, 712)) return false;
      tc_fence_after();
      uint32_t v[NW * WR];
      tmem_ld_cols(lane_base + (NS + (j & 1)) * N, v);
#pragma unroll
      for (int r = 0; r < WR; ++r) o[r] = fmaf(o[r], al[r], q8_join<FMT, WR, NW>(v, r) * be[r]);
      return true;
    };
    bool ok = true;
    for (int j = tg; j < nt; j += TG) {
      // (full: the scales, which this warp reads itself)
      ok = ok && (__all_sync(0xffffffffu, mbar_test_both(&sm.s_full[j % NS], (j / NS) & 1, &sm.full[j % NST], (j / NST) & 1)) ||
                  (spin_warp(&sm.s_full[j % NS], (j / NS) & 1, 713) && spin_warp(&sm.full[j % NST], (j / NST) & 1, 715)));
      tc_fence_after();
      float x[WR];
      const float* sc = reinterpret_cast<const float*>(qtsm + (j % NST) * kQtStage + 2 * kQtTile);
      float ka = sc[key], vb = sc[kQtKeys + key];
      q8_scales(ka, vb);
      {
        uint32_t v[NQ * WR];
        tmem_ld_cols(lane_base + (j % NS) * N, v);
#pragma unroll
        for (int r = 0; r < WR; ++r) x[r] = q8_join<FMT, WR, NQ>(v, r) * (ka * xs[r]);
      }
      const int t0 = slot_t(j, 0);
      if (t0 + kQtKeys > n_all) {
#pragma unroll
        for (int r = 0; r < WR; ++r)
          if (t0 + key >= n_prior + min(r0 + row_wg + r, a.lq * a.G - 1) / a.G + 1) x[r] = -INFINITY;
      }
      // the tile's maximum of each row, of logit and value scale together
      // [warp][RT]; two buffers in turn: a warp that writes one has passed the barrier of the
      // tile in between, and with it every warp's reads of the maxima before that
      float* mx = smf + Sh::kMax + (2 * tg + ((j / TG) & 1)) * 4 * RT + row_wg;
      {
        float mw[WR];
        const float lv = fast_log2(vb);
#pragma unroll
        for (int r = 0; r < WR; ++r) mw[r] = redux_max(x[r] + lv);
        if (lane == 0) {
#pragma unroll
          for (int r = 0; r < WR; r += 4)
            *reinterpret_cast<float4*>(mx + (warp & 3) * RT + r) = make_float4(mw[r], mw[r + 1], mw[r + 2], mw[r + 3]);
        }
      }
      // With two tile groups, now the O of this warpgroup's tile before: PV_j will overwrite it,
      // and the W buffer below was its own. (With one, both are those of tile j - 2, which was
      // drained; its O_{j - 1} can wait until W_j is out.)
      if (TG == 2 && j >= TG) ok = ok && drain(j - TG);
      // a named barrier has no time limit: the four warps leave together if a wait ran out
      if (!(ok = bar_all(bar_wg, 128, ok))) break;
      const float mt = fmaxf(fmaxf(mx[row_own], mx[RT + row_own]), fmaxf(mx[2 * RT + row_own], mx[3 * RT + row_own]));
      const float top = mt == -INFINITY ? 0.f : mt;
      const float mn = fmaxf(m, mt), mr = mn == -INFINITY ? 0.f : mn;
      const float al_own = fast_exp2(m - mr), be_own = fast_exp2(mt - mr);                       // (one of them is 1)
      const bool far = __any_sync(0xffffffffu, al_own * be_own < 0x1p-120f && m > -INFINITY);
      // weights, as pieces, to this key's row of the W buffer: [16 columns][128 keys][16 bytes]
      const float unit = vb * kTop;
      uint32_t ww[NW + 1][WR / 4];
#pragma unroll
      for (int r = 0; r < WR; r += 4) {
        uint32_t pc[NW];
        float w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x[r + u] = fast_exp2(x[r + u] - __shfl_sync(0xffffffffu, top, r + u));
          w[u] = x[r + u] * unit;
        }
        q8_split4<FMT, NW>(w, pc);
#pragma unroll
        for (int p = 0; p < NW; ++p) ww[p][r / 4] = pc[p];
        ww[NW][r / 4] = 0u;
      }
      const uint32_t wb = base + Sh::kW + (j & 1) * N * 128 + key * 16;
      if constexpr (WR == 4) {
        st_shared_v4(wb, ww[0][0], ww[1][0], ww[2][0], ww[3][0]);
      } else {
        // (the last row group's pieces are followed by the columns that belong to none)
#pragma unroll
        for (int p = 0; p < NW + (N > NW * RT ? 1 : 0); ++p) {
          const int col = (rg * NW + p) * WR;
          if (p < NW || rg == RG - 1) st_shared_v2(wb + (col >> 4) * 2048 + (col & 15), ww[p][0], ww[p][WR / 4 - 1]);
        }
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive_warp(&sm.w_full[j & 1]);
      if (TG == 1 && j >= TG) ok = ok && drain(j - TG);
#pragma unroll
      for (int r = 0; r < WR; ++r) {
        al[r] = __shfl_sync(0xffffffffu, al_own, r);
        be[r] = __shfl_sync(0xffffffffu, be_own, r);
      }
      if (__builtin_expect(far, 0)) {
        // a factor that an exponential does not hold, though its product with the sum may be
        // any number: as two halves
        const float ah = fast_exp2(0.5f * (m - mr)), bh = fast_exp2(0.5f * (mt - mr));
#pragma unroll
        for (int r = 0; r < WR; ++r) {
          const float a = __shfl_sync(0xffffffffu, ah, r), c = __shfl_sync(0xffffffffu, bh, r);
          l[r] = fmaf(l[r] * a, a, x[r] * c * c);
        }
      } else {
#pragma unroll
        for (int r = 0; r < WR; ++r) l[r] = fmaf(l[r], al[r], x[r] * be[r]);
      }
      m = mn;
    }
    const int last = (nt - 1 - tg) / TG * TG + tg;  // the warpgroup's last tile, if it had one
    if (tg < nt && ok) ok = drain(last);

    // ---- the CTA's row sums, then every CTA of the cluster gets its share of the dims (dim
    // d belongs to CTA d / per) and all (m, l)
#pragma unroll
    for (int r = 0; r < WR; ++r) {
      const float s = warp_sum(l[r]);
      if (lane == 0) sm_l[(tg * 4 + (warp & 3)) * RT + row_wg + r] = s;
    }
    if (csize > 1) cluster_wait();
    const int per = q8_dims_per(csize), owner = key / per, slot = key - owner * per;
    const uint32_t my_o = smem_u32(smf + Sh::kO), my_ml = smem_u32(smf + Sh::kMl);
    const int part = rank * TG + tg, parts = csize * TG;
    const uint32_t dst = dsmem_map(my_o, owner) + (part * per + slot) * 4;
#pragma unroll
    for (int r = 0; r < WR; ++r) st_dsmem_f32(dst + (row_wg + r) * per * parts * 4, o[r]);
    asm volatile("bar.sync %0, 128;" ::"r"(bar_wg) : "memory");
    for (int it = key; it < WR * csize; it += 128) {
      const int to = it / WR, r = row_wg + it % WR;
      const float* lw = sm_l + tg * 4 * RT + r;
      const float L = (lw[0] + lw[RT]) + (lw[2 * RT] + lw[3 * RT]);
      const uint32_t p = dsmem_map(my_ml, to) + (part * RT + r) * 8;
      st_dsmem_f32(p, m);                           // (it % WR is lane % WR)
      st_dsmem_f32(p + 4, L);
    }
  }
  if (csize > 1 && warp >= kMmaWarp) cluster_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, Sh::kCols);
  if (csize > 1) cluster_sync_all();                // every CTA's rows are here
  if (*abort_flag) return;
  const int per = q8_dims_per(csize), d0 = rank * per, d_items = min(per, 128 - d0) / 4;
  for (int it = threadIdx.x; it < nrow * d_items; it += Sh::kThreads) {      // four dims of a row
    const int r = it / d_items, d = (it - r * d_items) * 4;
    const int parts = csize * TG;
    const float* ml = smf + Sh::kMl + r * 2;        // [parts][RT][2]
    const float* po = smf + Sh::kO + r * per * parts + d;
    float M = -INFINITY;
#pragma unroll 4
    for (int u = 0; u < parts; ++u) M = fmaxf(M, ml[u * RT * 2]);
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int u = 0; u < parts; ++u) {
      const float2 z = *reinterpret_cast<const float2*>(ml + u * RT * 2);
      const float4 x = *reinterpret_cast<const float4*>(po + u * per);
      const float half = fast_exp2(0.5f * (z.x - (M == -INFINITY ? 0.f : M))), c = half * half;
      L += z.y * half * half;
      O.x += x.x * c; O.y += x.y * c; O.z += x.z * c; O.w += x.w * c;
    }
    const int i = a.lq == 1 ? 0 : (r0 + r) / a.G, hl = (r0 + r) - i * a.G;
    const int64_t row = ((int64_t)b * a.lq + i) * a.hq + g * a.G + hl;
    const float inv = kUnitW / kTop / L;
    uint2 w;
    w.x = bf16x2_rn(O.x * inv, O.y * inv);
    w.y = bf16x2_rn(O.z * inv, O.w * inv);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + row * 128 + d0 + d) = w;
    if (d0 + d == 0 && a.lse) a.lse[row] = (M + __log2f(L)) * 0.69314718055994531f;
  }
}

}  // namespace esa
