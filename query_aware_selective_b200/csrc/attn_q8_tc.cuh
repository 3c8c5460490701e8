// attn_q8_tc.cuh - exact attention of few queries over an 8-bit cache of head dim 128 on
// the fifth-generation tensor cores (sm_100a tcgen05), codes fed to them as they are.
//
// The formulas are those of attn_q8.cuh. Both products take the codes as the M = 128 side
// of an 8-bit MMA straight from shared memory, without any conversion:
//   S^T [128 keys x N] = K [128 x 128] Q^T    (A: K rows, K-major)
//   O^T [128 dims x N] = V^T [128 x 128] W^T  (A: V rows read M-major)
// kind::f8f6f4 for e4m3 (fp32 sums), kind::i8 for int8 (exact 32-bit sums). Queries and
// weights go in as P pieces of 8 bits, each its own column:
//   e4m3: piece p = e4m3(16^p (x - pieces before)), 4 significant bits each: two for a bf16
//         query, three for a weight (relative 2^-13)
//   int8: digits of 7 bits of an integer: three for a query (its row's largest is 2^19 to
//         2^20), four for a weight (its tile's largest is 2^27)
// so column p * RT + r is piece p of query row r, and a row's value is the sum of its
// columns times 2^(-4 p) or 2^(-7 p).
// Weights are taken relative to their key tile's own maximum (of 128 keys), and a tile's O
// is drained from TMEM into fp32 registers and scaled there: the range of 8-bit pieces
// then only has to span one tile (a weight is rounded to 2^-26 (e4m3) or 2^-28 (int8) of its
// tile's largest at worst; three int8 digits, 2^-21, showed in dims where the largest
// weight's value is next to zero), and nothing in TMEM is ever rescaled.
//
// Roles (7 warps): warps 0-3 softmax (thread = key for S and W, thread = dim for O), warp 4
// issues the MMAs, warps 5-6 copy keys, values and scales (16-byte cp.async, 8 lanes a
// row, into 128-byte-swizzled tiles). TMEM: S and O, two buffers each. A CTA takes a share
// of one (sequence, KV head)'s key list; the CTAs of a cluster meet in distributed shared
// memory at the end.
#pragma once
#include "attn_q8.cuh"
#include "common.cuh"
#include "keylist.cuh"

namespace esa {

constexpr int kQtThreads = 7 * 32;
constexpr int kQtKeys = 128;
constexpr uint32_t kQtTile = 128 * 128;                       // bytes of a key or value tile
constexpr uint32_t kQtStage = 2 * kQtTile + 2 * kQtKeys * 4;  // keys, values, their scales

template <int FMT, int RT>
struct QtShape {
  static constexpr int NQ = FMT == kQ8E4M3 ? 2 : 3, NW = FMT == kQ8E4M3 ? 3 : 4;   // pieces of a query, of a weight
  static constexpr int N = (NW * RT + 15) / 16 * 16;          // MMA columns (M = 128: a multiple of 16)
  static constexpr int kCtas = RT <= 4 ? 2 : 1;               // per SM
  static constexpr int kStages = kCtas == 2 ? 3 : 5;
  static constexpr uint32_t kCols = 4 * N <= 64 ? 64 : 4 * N <= 128 ? 128 : 256;   // TMEM columns
  static constexpr uint32_t kQ = kStages * kQtStage, kW = kQ + N * 128, kCtrl = kW + 2 * N * 128;
  static constexpr uint32_t kSmem = kCtrl + 1024 + (2 * 4 * RT + 2 * RT + 4 * RT) * 4;
};

struct QtCtrl {
  uint64_t full[5], empty[5], s_full[2], w_full[2], o_full[2], q_full, mma_done;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(QtCtrl) <= 1024, "control block overflows its reservation");

template <int FMT>
__device__ __forceinline__ void umma_q8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  if constexpr (FMT == kQ8E4M3) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
  }
}
// Instruction descriptor: e4m3 x e4m3 -> fp32, or s8 x s8 -> s32.
template <int FMT>
__host__ __device__ constexpr uint32_t q8_idesc(uint32_t n, uint32_t a_mn_major) {
  return FMT == kQ8E4M3 ? umma_idesc(0, 128, n, a_mn_major, 0)
                        : (2u << 4) | (1u << 7) | (1u << 10) | (a_mn_major << 15) | ((n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ float redux_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// N columns of a TMEM buffer, this thread's lane
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t addr, uint32_t* v) {
#pragma unroll
  for (int c = 0; c < N; c += 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[c]), "=r"(v[c + 1]), "=r"(v[c + 2]), "=r"(v[c + 3]), "=r"(v[c + 4]), "=r"(v[c + 5]), "=r"(v[c + 6]),
          "=r"(v[c + 7]), "=r"(v[c + 8]), "=r"(v[c + 9]), "=r"(v[c + 10]), "=r"(v[c + 11]), "=r"(v[c + 12]),
          "=r"(v[c + 13]), "=r"(v[c + 14]), "=r"(v[c + 15])
        : "r"(addr + c));
  tmem_wait_ld();
}
// a row's value from its columns (NP pieces RT columns apart)
template <int FMT, int RT, int NP>
__device__ __forceinline__ float q8_join(const uint32_t* v, int r) {
  if constexpr (FMT == kQ8E4M3) {
    float x = __uint_as_float(v[(NP - 1) * RT + r]);
#pragma unroll
    for (int p = NP - 2; p >= 0; --p) x = fmaf(x, 0.0625f, __uint_as_float(v[p * RT + r]));
    return x;
  } else {
    float x = (float)(int)v[(NP - 1) * RT + r];
#pragma unroll
    for (int p = NP - 2; p >= 0; --p) x = fmaf(x, 0.0078125f, (float)(int)v[p * RT + r]);
    return x;
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

// The CTAs of a cluster hold partial rows o [nrow][RF] with (m, l) pairs ml [nrow][2] at the
// same shared-memory offsets; CTA `rank` writes its share of the merged rows. o carries a
// factor 1 / o_scale; row r belongs to query (r0 + r) / G, head g * G + (r0 + r) % G.
template <typename T, int RF, int D>
__device__ __forceinline__ void q8_cluster_merge(const AttnQ8Args& a, const float* sm_o, const float* sm_ml, int b,
                                                 int g, int r0, int nrow, int rank, int csize, float o_scale,
                                                 int threads) {
  constexpr int Q = D / 4;
  for (int it = threadIdx.x + threads * rank; it < nrow * Q; it += threads * csize) {
    const int d4 = it % Q, r = it / Q;
    const uint32_t ml = smem_u32(sm_ml + r * 2), oo = smem_u32(sm_o + r * RF + d4 * 4);
    float M = -INFINITY;
    for (int u = 0; u < csize; ++u) M = fmaxf(M, __uint_as_float(ld_dsmem_u32(dsmem_map(ml, u))));
    const float mr = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int u = 0; u < csize; ++u) {
      const uint2 z = ld_dsmem_u2(dsmem_map(ml, u));
      const float4 o = ld_dsmem_f4(dsmem_map(oo, u));
      const float c = fast_exp2(__uint_as_float(z.x) - mr);
      L += __uint_as_float(z.y) * c;
      O.x += o.x * c; O.y += o.y * c; O.z += o.z * c; O.w += o.w * c;
    }
    const int i = (r0 + r) / a.G, hl = (r0 + r) - i * a.G;
    const int64_t row = ((int64_t)b * a.lq + i) * a.hq + g * a.G + hl;
    const float inv = o_scale / L;
    T* dst = static_cast<T*>(a.o) + row * D + d4 * 4;
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(dst) = make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
    } else {
      uint2 w;
      w.x = bf16x2_rn(O.x * inv, O.y * inv);
      w.y = bf16x2_rn(O.z * inv, O.w * inv);
      *reinterpret_cast<uint2*>(dst) = w;
    }
    if (d4 == 0 && a.lse) a.lse[row] = (M + __log2f(L)) * 0.69314718055994531f;
  }
}

// grid (cluster size, Hkv * tiles, B), cluster (cluster size, 1, 1); a.hc = 1. RT: query
// rows of a tile.
template <int FMT, int RT>
__global__ void __launch_bounds__(kQtThreads, (QtShape<FMT, RT>::kCtas)) attn_q8_tc_kernel(const AttnQ8Args a) {
  using Sh = QtShape<FMT, RT>;
  constexpr int N = Sh::N, NST = Sh::kStages, NQ = Sh::NQ, NW = Sh::NW;
  // a weight of 1 (its tile's largest) goes in as 2^8 (e4m3, <= 448), 2^27 (int8, <= 127 * 2^21)
  constexpr float kTop = FMT == kQ8E4M3 ? 8.f : 27.f;
  // units of the first piece of a query and of a weight
  constexpr float kUnitQ = FMT == kQ8E4M3 ? 1.f : 0x1p14f, kUnitW = FMT == kQ8E4M3 ? 1.f : 0x1p21f;
  constexpr int RF = 132;
  extern __shared__ __align__(1024) uint8_t qtsm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = smem_u32(qtsm);
  QtCtrl& sm = *reinterpret_cast<QtCtrl*>(qtsm + Sh::kCtrl);
  float* const sm_max = reinterpret_cast<float*>(qtsm + Sh::kCtrl + 1024);   // [2][4 warps][RT] tile maxima
  float* const sm_ml = sm_max + 8 * RT;                                      // [RT][2]
  float* const sm_l = sm_ml + 2 * RT;                                        // [4 warps][RT]
  float* const sm_o = reinterpret_cast<float*>(qtsm);                        // [RT][RF], over the stages at the end

  const int g = blockIdx.y / a.tiles, tile = blockIdx.y - g * a.tiles, b = blockIdx.z;
  const int rank = blockIdx.x, csize = gridDim.x;
  const int list = a.lists > 1 ? b * a.lists + g : b;
  KeyList kl = a.keys;
  const int64_t c0 = kl.vl.len ? kl.resolve(b, 706) : a.c0;
  const int cnt = min(max(kl.count[list], 0), (int)kl.idx_stride);
  const int n_prior = (int)(kl.ni + cnt + (c0 - kl.lo));
  const int r0 = tile * RT, nrow = min(RT, a.lq * a.G - r0);
  const int n_keys = n_prior + (r0 + nrow - 1) / a.G + 1;      // that the tile's last row attends
  const int n_all = n_prior + r0 / a.G + 1;                    // that every row of the tile attends
  const int tiles_all = (n_keys + kQtKeys - 1) / kQtKeys;
  const int j0 = (int)((int64_t)tiles_all * rank / csize);
  const int nt = (int)((int64_t)tiles_all * (rank + 1) / csize) - j0;   // this CTA's key tiles

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 64);                   // every producer thread, when its copies have landed
      mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.w_full[s], 4);
      mbar_init(&sm.o_full[s], 1);
    }
    mbar_init(&sm.q_full, 4);
    mbar_init(&sm.mma_done, 1);
    sm.abort_flag = base & 1023u ? 1 : 0;
    if (base & 1023u) record_status(5u, 710);
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(&sm.tmem_base, Sh::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;

  float o[RT], m[RT], l[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    o[r] = 0.f;
    m[r] = -INFINITY;
    l[r] = 0.f;
  }

  if (*abort_flag) {
    // misaligned shared memory: reported, nothing done
  } else if (warp >= 5) {
    // ------------------------------------------------------------------- producers
    const uint32_t row_bytes = (uint32_t)a.hkv * 128;
    const int pw = warp - 5, c = lane & 7, lr = lane >> 3;
    const uint8_t* kb = a.k + (int64_t)b * a.n_cap * row_bytes + g * 128 + c * 16;
    const uint8_t* vb = a.v + (int64_t)b * a.n_cap * row_bytes + g * 128 + c * 16;
    const float* ksb = a.ks + (int64_t)b * a.nblk * a.hkv + g;
    const float* vsb = a.vs + (int64_t)b * a.nblk * a.hkv + g;
    const int32_t* ib = kl.idx + (int64_t)list * kl.idx_stride;
    const int ni = (int)kl.ni, jump = (int)(kl.lo - kl.ni) - cnt;
    auto position = [&](int j, int h) -> int {      // of row 64 pw + 32 h + lane (behind the list: its last key)
      const int t = min((j0 + j) * kQtKeys + pw * 64 + h * 32 + lane, n_keys - 1);
      const int p = t < ni ? t : (t < ni + cnt ? __ldg(ib + t - ni) : t + jump);
      return min(max(p, 0), (int)a.n_cap - 1);
    };
    int pos[2] = {0, 0};
    if (nt > 0) { pos[0] = position(0, 0); pos[1] = position(0, 1); }
    const uint32_t sw0 = (uint32_t)(pw * 64 + lr) * 128 + ((c ^ lr) << 4);            // rows 8 i + lr
    const uint32_t sw1 = (uint32_t)(pw * 64 + 4 + lr) * 128 + ((c ^ (4 + lr)) << 4);  // rows 8 i + 4 + lr
    for (int j = 0; j < nt; ++j) {
      const int s = j % NST;
      if (!mbar_wait_warp(&sm.empty[s], ((j / NST) & 1) ^ 1, abort_flag, 707)) break;
      const uint32_t kd = base + s * kQtStage, vd = kd + kQtTile;
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
      if (j + 1 < nt) { pos[0] = position(j + 1, 0); pos[1] = position(j + 1, 1); }
    }
    cp_async_wait_all();
  } else if (warp == 4) {
    // ------------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = q8_idesc<FMT>(N, 0), idesc_o = q8_idesc<FMT>(N, 1);
      const uint64_t dq = sdesc_sw128(base + Sh::kQ, 16, 1024);
      // S_j into buffer j & 1: its previous scores S_{j-2} were read before w_full[j - 2]
      auto issue_s = [&](int j) -> bool {
        const int s = j % NST;
        if (!mbar_wait(&sm.full[s], (j / NST) & 1, abort_flag, 708)) return false;
        fence_proxy_async();                        // cp.async wrote through the generic proxy
        tc_fence_after();
        const uint64_t dk = sdesc_sw128(base + s * kQtStage, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_q8<FMT>(tmem + (j & 1) * N, dk + kk * 2, dq + kk * 2, idesc_s, kk > 0);
        umma_commit(&sm.s_full[j & 1]);
        return true;
      };
      bool ok = nt == 0 || mbar_wait(&sm.q_full, 0, abort_flag, 709);
      for (int j = 0; j < 2 && j < nt && ok; ++j) ok = issue_s(j);
      for (int j = 0; j < nt && ok; ++j) {
        if (!(ok = mbar_wait(&sm.w_full[j & 1], (j >> 1) & 1, abort_flag, 711))) break;
        tc_fence_after();
        const uint64_t dv = sdesc_sw128(base + (j % NST) * kQtStage + kQtTile, 16, 1024);
        const uint64_t dw = sdesc_sw128(base + Sh::kW + (j & 1) * N * 128, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)              // 32 keys: four 8-row groups of V, 32 bytes of a W row
          umma_q8<FMT>(tmem + (2 + (j & 1)) * N, dv + kk * 256, dw + kk * 2, idesc_o, kk > 0);
        umma_commit(&sm.o_full[j & 1]);
        umma_commit(&sm.empty[j % NST]);
        if (j + 2 < nt) ok = issue_s(j + 2);
      }
      // every MMA issued so far has completed before TMEM and shared memory are reused
      umma_commit(&sm.mma_done);
      mbar_wait(&sm.mma_done, 0, abort_flag, 714, /*respect_abort=*/false);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------- softmax warps
    // queries as pieces: thread (r, part) takes 128 / (128 / RT) dims of row r
    constexpr int TPR = 128 / RT, DPT = 128 / TPR;  // threads of a row, dims of a thread
    float xs[RT];                                   // logit factor of each row
    {
      const int r = threadIdx.x / TPR, part = threadIdx.x % TPR;
      const int rr = min(r0 + r, a.lq * a.G - 1), i = rr / a.G, hl = rr - i * a.G;
      const __nv_bfloat16* qp =
          static_cast<const __nv_bfloat16*>(a.q) + (((int64_t)b * a.lq + i) * a.hq + g * a.G + hl) * 128 + part * DPT;
      float f[DPT];
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < DPT; e += 4) {
        load4(qp + e, f + e);
#pragma unroll
        for (int u = 0; u < 4; ++u) mx = fmaxf(mx, fabsf(f[e + u]));
      }
#pragma unroll
      for (int w = TPR < 32 ? TPR / 2 : 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      // 2^qe brings the row's largest to [2^7, 2^8) (e4m3) or [2^19, 2^20) (int8)
      const int qe = min((FMT == kQ8E4M3 ? 7 : 19) - ((int)((__float_as_uint(mx) >> 23) & 0xffu) - 127), 100);
      const float up = __uint_as_float((uint32_t)(qe + 127) << 23);
      if (part == 0) sm_l[r] = a.scale_log2 * kUnitQ * __uint_as_float((uint32_t)(127 - qe) << 23);
      const uint32_t q0 = base + Sh::kQ;
#pragma unroll
      for (int e = 0; e < DPT; e += 4) {
        uint32_t pc[2][NQ];
        q8_split2<FMT, NQ>(f[e] * up, f[e + 1] * up, pc[0]);
        q8_split2<FMT, NQ>(f[e + 2] * up, f[e + 3] * up, pc[1]);
        const int d = part * DPT + e;
#pragma unroll
        for (int p = 0; p < NW; ++p) {
          const uint32_t n = p * RT + r;
          const uint32_t v = p < NQ ? pc[0][p < NQ ? p : 0] | (pc[1][p < NQ ? p : 0] << 16) : 0u;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(q0 + n * 128 + (((d >> 4) ^ (n & 7)) << 4) + (d & 15)), "r"(v)
                       : "memory");
        }
      }
      // columns that belong to no piece: zero in the queries and in both weight buffers
      if constexpr (N > NW * RT) {
        constexpr int pad = (N - NW * RT) * 8;          // 16-byte pieces of a buffer (W follows Q)
        for (int z = threadIdx.x; z < 3 * pad; z += 128)
          st_shared_v4(base + Sh::kQ + ((z / pad) * N + NW * RT) * 128 + (z % pad) * 16, 0u, 0u, 0u, 0u);
      }
      fence_proxy_async();
      mbar_arrive_warp(&sm.q_full);
      asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
      for (int q = 0; q < RT; ++q) xs[q] = sm_l[q];
    }
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const int key = threadIdx.x;                    // of a tile, for S and W; the dim, for O
    float al[RT], be[RT];                           // the tile's factors on o and on its own O
    auto drain = [&](int j) -> bool {               // o = o al + O_j be
      if (!mbar_wait_warp(&sm.o_full[j & 1], (j >> 1) & 1, abort_flag, 712)) return false;
      tc_fence_after();
      uint32_t v[N];
      tmem_ld_n<N>(lane_base + (2 + (j & 1)) * N, v);
#pragma unroll
      for (int r = 0; r < RT; ++r) o[r] = fmaf(o[r], al[r], q8_join<FMT, RT, NW>(v, r) * be[r]);
      return true;
    };
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      // (full: the scales, which this warp reads itself)
      ok = ok && mbar_wait_warp(&sm.full[j % NST], (j / NST) & 1, abort_flag, 715) &&
           mbar_wait_warp(&sm.s_full[j & 1], (j >> 1) & 1, abort_flag, 713);
      // a named barrier has no time limit: all four warps leave together
      if (!(ok = bar_all(1, 128, ok))) break;
      tc_fence_after();
      float x[RT];
      const float* sc = reinterpret_cast<const float*>(qtsm + (j % NST) * kQtStage + 2 * kQtTile);
      const float ka = sc[key];
      const float lv = __log2f(fmaxf(sc[kQtKeys + key], 0x1p-120f));
      {
        uint32_t v[N];
        tmem_ld_n<N>(lane_base + (j & 1) * N, v);
#pragma unroll
        for (int r = 0; r < RT; ++r) x[r] = fmaf(q8_join<FMT, RT, NQ>(v, r), ka * xs[r], lv);
      }
      const int t0 = (j0 + j) * kQtKeys;
      if (t0 + kQtKeys > n_all) {
#pragma unroll
        for (int r = 0; r < RT; ++r)
          if (t0 + key >= n_prior + min(r0 + r, a.lq * a.G - 1) / a.G + 1) x[r] = -INFINITY;
      }
      // the tile's maximum of each row
      float mt[RT];
      float* mx = sm_max + (j & 1) * 4 * RT;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        mt[r] = redux_max(x[r]);
        if (lane == 0) mx[warp * RT + r] = mt[r];
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
      for (int r = 0; r < RT; ++r)
        mt[r] = fmaxf(fmaxf(mx[r], mx[RT + r]), fmaxf(mx[2 * RT + r], mx[3 * RT + r]));
      // weights, as pieces, to row p * RT + r of the W buffer, byte `key`
      const uint32_t wb = base + Sh::kW + (j & 1) * N * 128;
      const float iv = fast_exp2(-lv - kTop);
#pragma unroll
      for (int r = 0; r < RT; r += 2) {
        uint32_t pc[NW];
        x[r] = fast_exp2(x[r] - (mt[r] == -INFINITY ? 0.f : mt[r]) + kTop);
        x[r + 1] = fast_exp2(x[r + 1] - (mt[r + 1] == -INFINITY ? 0.f : mt[r + 1]) + kTop);
        q8_split2<FMT, NW>(x[r], x[r + 1], pc);
#pragma unroll
        for (int p = 0; p < NW; ++p) {
          const uint32_t n0 = p * RT + r, n1 = n0 + 1;
          st_shared_u8(wb + n0 * 128 + (((key >> 4) ^ (n0 & 7)) << 4) + (key & 15), pc[p]);
          st_shared_u8(wb + n1 * 128 + (((key >> 4) ^ (n1 & 7)) << 4) + (key & 15), pc[p] >> 8);
        }
      }
      fence_proxy_async();
      tc_fence_before();
      mbar_arrive_warp(&sm.w_full[j & 1]);
      if (j > 0) ok = drain(j - 1);                 // (a wait that ran out: the next bar_all)
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float mn = fmaxf(m[r], mt[r]);
        const float mr = mn == -INFINITY ? 0.f : mn;
        al[r] = fast_exp2(m[r] - mr);
        const float bt = fast_exp2(mt[r] - mr);
        l[r] = fmaf(l[r], al[r], x[r] * iv * bt);
        be[r] = bt * kUnitW;
        m[r] = mn;
      }
    }
    if (nt > 0 && ok) ok = drain(nt - 1);
  }
  tc_fence_before();
  __syncthreads();                                  // every MMA and copy is done: the stages are free
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tmem, Sh::kCols);
  if (warp < 4) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      sm_o[r * RF + threadIdx.x] = o[r];
      const float s = warp_sum(l[r]);
      if (lane == 0) sm_l[warp * RT + r] = s;
      if (threadIdx.x == 0) sm_ml[2 * r] = m[r];
    }
  }
  __syncthreads();
  if (threadIdx.x < RT)
    sm_ml[2 * threadIdx.x + 1] = (sm_l[threadIdx.x] + sm_l[RT + threadIdx.x]) +
                                 (sm_l[2 * RT + threadIdx.x] + sm_l[3 * RT + threadIdx.x]);
  if (csize > 1) cluster_sync_all();
  else __syncthreads();
  if (!*abort_flag)
    q8_cluster_merge<__nv_bfloat16, RF, 128>(a, sm_o, sm_ml, b, g, r0, nrow, rank, csize,
                                             FMT == kQ8E4M3 ? 0x1p-8f : 0x1p-27f, kQtThreads);
  if (csize > 1) cluster_sync_all();                // no CTA leaves while it is read
}

}  // namespace esa
