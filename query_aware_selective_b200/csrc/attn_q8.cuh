// attn_q8.cuh - exact attention over the initial + selected + local tokens of an 8-bit cache
// for fp32 queries and for heads of 64 (ESA write-up: implementation and final-attention
// paragraphs - global part = initial + selected tokens, window part = local tokens, one
// softmax). bf16 queries on heads of 128 run attn_q8_tc.cuh.
//
// With codes kc, vc and block scales a, b the logits and the output of a query row are
//   x_j = c (q . kc_j) a_j,    l = sum_j 2^(x_j - m),    o = sum_j 2^(x_j + log2 b_j - m) vc_j / l
// (c = softmax scale * log2 e), so the scales never touch the codes: they multiply one
// logit and add to one exponent per key. Both products run on the tensor cores as
// m16n8k16 f16 MMAs with fp32 accumulation, and an e4m3 or int8 code is an exact f16:
//   S^T [16 keys x 8 rows]  = Kc [16 x D] . Q^T       (A = codes, B = queries)
//   O^T [D x 8 rows]       += Vc^T [D x 16 keys] . W^T (A = codes transposed, B = weights)
// Keys and dims are the M dimension and the query rows N = 8, because a decode step has
// only the G heads of a KV head as rows. A dot product does not mind the order of its
// terms, so the fragments take their dims (K) and keys (V) in the order in which 16-byte
// shared-memory loads deliver them: no transposition but byte pairs of two keys brought
// side by side (prmt), and one conversion per two codes. S^T becomes the B operand of the
// second product by movmatrix.
// m is a reference, not the maximum: it is raised to max_j (x_j + log2 b_j) when that
// exceeds it by 5, and W = e_j b_j 2^10 <= 2^15, e_j = 2^(x_j - m), is rounded to f16 (relative
// 2^-11; a weight under 2^-35 of the largest is lost, which 2^20 of them do not make
// visible). l sums the e_j, which hold no b_j: from W it would lose the keys whose values are
// zero (b_j 2^-100) beside loud ones. e_j spans 2^105 (those keys) down to 2^-98 for the row's
// largest x_j (under values of 2^97), and a step of m the sum of the two, more than one
// exponential holds: l takes it as two halves. fp32 queries go in as two f16 (q = hi +
// lo), and so do the weights, for 22 bits of each: more bits than 8-bit pieces give in a
// narrow MMA, which is why fp32 stays here; a head of 64 is half the M = 128 that the
// 8-bit MMAs of attn_q8_tc.cuh take.
//
// Bound by the latency of a warp's own chain (copy, products, exponentials, products), of which
// the SM holds too few to hide it: bf16 on heads of 64, 16 sequences x 6.3K keys x 8 heads
// (103 MB), 28 us, 3.7 TB/s, with 14 warps an SM and 44% of the issue slots used, a warp waiting
// for loads, fixed latencies and shared memory in about equal parts; fp32 on heads of 128
// (206 MB) 46 us, 4.5 TB/s, with the 8 warps that its registers allow and 39%; 512 fp32 queries
// at 40% of the issue slots and of the mma.sync pipe each. One short sequence (4 heads of 64,
// 400 keys) takes 5 us, of which 2 are the launch. A warp streams 16 keys a step through its own ring of
// three steps in shared memory (16-byte cp.async). The key list of a (sequence, KV head) is
// split over the 8 warps of a CTA and over the CTAs of a cluster; the parts meet in
// (distributed) shared memory, so there is no workspace, no counter to clear and no second
// kernel. (A CTA per KV head; several heads in one, for longer consecutive reads, measured
// the same or slower: 32.0, 32.5, 33.3 us for 1, 2, 4 heads at 256 CTAs.)
#pragma once
#include "attn_tc.cuh"
#include "cache_q8.cuh"
#include "common.cuh"
#include "keylist.cuh"

namespace esa {

constexpr int kQ8Warps = 8, kQ8Threads = kQ8Warps * 32;
constexpr int kQ8Keys = 16;                     // keys of a warp's step
constexpr int kQ8Stages = 3;                    // steps of a warp's ring
// weights: 2^10 at the reference, at most 2^15 (f16: 2^16)
constexpr float kQ8Head = 10.f, kQ8Unit = 0x1p10f;
constexpr uint32_t kQ8Most = 0x78007800u;       // 2^15 twice, as f16

struct AttnQ8Args {
  const void* q;            // [B, Lq, Hq, D]
  const uint8_t* k;         // [B, n_cap, Hkv, D]
  const uint8_t* v;
  const float* ks;          // [B, nblk, Hkv]
  const float* vs;
  void* o;                  // [B, Lq, Hq, D]
  float* lse;               // [B, Lq, Hq] or null
  KeyList keys;
  int64_t n_cap, nblk, c0;
  int lq, hq, hkv, G;
  int lists, bshift;
  int tiles;                // row tiles of a KV head
  float scale_log2;
};

template <int NT, int D>
__host__ __device__ constexpr int q8_row_floats() { return D + 4; }     // o, then padding
// A step in a warp's ring: 16 key rows, 16 value rows, their 32 scales.
template <int D>
__host__ __device__ constexpr int q8_stage_bytes() { return 2 * kQ8Keys * D + 128; }
template <int NT, int D>
__host__ __device__ constexpr int q8_smem_bytes() {
  // the rings; after the loop the warps' partial rows, (m, l) of every warp row, (m, l) of
  // every merged row
  constexpr int rings = kQ8Warps * kQ8Stages * q8_stage_bytes<D>();
  constexpr int merge = (kQ8Warps * 8 * NT * q8_row_floats<NT, D>() + 4 * kQ8Warps * 8 * NT) * 4;
  return rings > merge ? rings : merge;
}
// Byte offset of 16-byte piece c of row r of a step's keys / values. The pieces are placed
// so that the eight lanes of a shared-memory phase hit all 32 banks: keys are read as rows
// (gid, all tig), values as pieces gid, gid + 1 of rows 2 tig.
template <int D>
__device__ __forceinline__ uint32_t q8_k_off(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ ((r & 1) << 2)) << 4);
  else return r * 64 + (c << 4);
}
template <int D>
__device__ __forceinline__ uint32_t q8_v_off(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (((r >> 1) & 3) << 1)) << 4);
  else return (r ^ ((r >> 2) & 1)) * 64 + ((c ^ (r & 2)) << 4);
}
__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(p) : "memory");
  return v;
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void mma_f16(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The four codes of word w as two f16 pairs. K: word = 4 dims of one key; the pairs are
// the dims (0, 1), (2, 3) for e4m3 and (0, 2), (1, 3) for int8 (q8_pair_dim).
template <int FMT>
__device__ __forceinline__ void q8_pairs(uint32_t w, uint32_t& p0, uint32_t& p1) {
  if constexpr (FMT == kQ8E4M3) {
    p0 = e4m3x2_to_f16x2((uint16_t)w);
    p1 = e4m3x2_to_f16x2((uint16_t)(w >> 16));
  } else {
    // 0x6400 | (c + 128) is the f16 1024 + 128 + c: exact, and so is the difference
    const uint32_t t0 = (w & 0x00ff00ffu) ^ 0x64806480u, t1 = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(p0) : "r"(t0), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(p1) : "r"(t1), "r"(0x64806480u));
  }
}
// dim (0..3 of a word) that element e (0, 1) of pair p holds
template <int FMT>
__host__ __device__ constexpr int q8_pair_dim(int p, int e) { return FMT == kQ8E4M3 ? 2 * p + e : p + 2 * e; }

// Words wa, wb: the same 4 dims of two keys. dims[d] = (key a, key b) of dim d as f16.
template <int FMT>
__device__ __forceinline__ void q8_transpose(uint32_t wa, uint32_t wb, uint32_t* dims) {
  if constexpr (FMT == kQ8E4M3) {
    q8_pairs<FMT>(__byte_perm(wa, wb, 0x5140), dims[0], dims[1]);
    q8_pairs<FMT>(__byte_perm(wa, wb, 0x7362), dims[2], dims[3]);
  } else {
    q8_pairs<FMT>(__byte_perm(wa, wb, 0x5410), dims[0], dims[1]);
    q8_pairs<FMT>(__byte_perm(wa, wb, 0x7632), dims[2], dims[3]);
  }
}

// log2 of a normal number
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The scales of a key as the softmax takes them. Scales of values under the least that is
// written, zero among them, count as that: 2^100 times 2^22 tokens still fit a row sum behind
// an m that is 5 low. One that is no finite number makes NaN of the rows that attend the key
// (through its logit), and of no others (their weight is a finite number times 0).
__device__ __forceinline__ void q8_scales(float& k, float& v) {
  k = fmaf(v, 0.f, k);
  v = fminf(fmaxf(v, 0x1p-100f), 0x1p100f);
}

// The exponent of a power of two that brings amax to [2^13, 2^14): queries of any range
// fit f16, and the elements that matter stay normal there.
__device__ __forceinline__ int q8_query_exp(float amax) {
  const int e = (int)((__float_as_uint(amax) >> 23) & 0xffu) - 127;
  return min(13 - e, 100);
}

template <typename T>
__device__ __forceinline__ void load4(const T* p, float* f) {
  if constexpr (sizeof(T) == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 a = bf16x2_to_float2(v.x), b = bf16x2_to_float2(v.y);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  } else {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
}

// grid (cluster size, Hkv * tiles, B), cluster (cluster size, 1, 1).
template <typename T, int D, int FMT, int NT>
__global__ void __launch_bounds__(kQ8Threads, NT == 1 && D == 64 ? 2 : 1) attn_q8_kernel(const AttnQ8Args a) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int ROWS = 8 * NT;
  constexpr int KC = D / 64;             // 16-byte pieces of a key row a lane takes (K)
  constexpr int VW = D / 32;             // words of a value row a lane takes (V)
  constexpr int RF = q8_row_floats<NT, D>();
  extern __shared__ __align__(128) float q8sm[];
  float* const sm_o = q8sm;                                    // [warp][ROWS][RF]
  float* const sm_ml = sm_o + kQ8Warps * ROWS * RF;            // [warp][ROWS][2]
  float* const sm_fin = sm_ml + 2 * kQ8Warps * ROWS;           // [ROWS][2]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gid = lane >> 2, tig = lane & 3;
  const int g = blockIdx.y / a.tiles, tile = blockIdx.y - g * a.tiles, b = blockIdx.z;
  const int rank = blockIdx.x, csize = gridDim.x;

  const int list = a.lists > 1 ? b * a.lists + g : b;
  KeyList kl = a.keys;
  pdl_wait();
  const int64_t c0 = kl.vl.len ? kl.resolve(b, 704) : a.c0;
  const int cnt = min(max(kl.count[list], 0), (int)kl.idx_stride);
  const int n_prior = (int)(kl.ni + cnt + (c0 - kl.lo));       // keys before the first query's own
  const int r0 = tile * ROWS, nrow = min(ROWS, a.lq * a.G - r0);
  const int i_first = r0 / a.G;
  const int n_keys = n_prior + (r0 + nrow - 1) / a.G + 1;      // that the tile's last row attends
  const int n_all = n_prior + i_first + 1;                     // that every row of the tile attends
  const int steps = (n_keys + kQ8Keys - 1) / kQ8Keys;
  // the warps' shares of the steps interleave: each gets its part of the scattered keys
  const int s_beg = rank * kQ8Warps + warp, s_end = steps, s_inc = csize * kQ8Warps;

  // ---- the stream: the warp's own ring of kQ8Stages steps in shared memory, filled by
  // 16-byte cp.async (8 or 4 lanes a row), positions looked up one step before that
  constexpr int CPR = D / 16;                      // 16-byte pieces of a row
  const uint32_t row_bytes = (uint32_t)a.hkv * D;
  const int cpc = lane % CPR, cpr = lane / CPR;    // this lane's piece of a row, and which rows it copies
  const uint8_t* kb = a.k + (int64_t)b * a.n_cap * row_bytes + g * D + cpc * 16;
  const uint8_t* vb = a.v + (int64_t)b * a.n_cap * row_bytes + g * D + cpc * 16;
  const float* sb = (lane < 16 ? a.ks : a.vs) + (int64_t)b * a.nblk * a.hkv + g;
  const int32_t* ib = kl.idx + (int64_t)list * kl.idx_stride;
  const int ni = (int)kl.ni, jump = (int)(kl.lo - kl.ni) - cnt;
  // Key slot lane % 16 of step s (a key behind the list: its last). Its list entry is fetched
  // kAhead steps before the step is copied and only looked at then: selecting or clamping it
  // at once would wait for a load that may miss all the way to HBM.
  constexpr int kAhead = 2;
  auto at = [&](int s) { return min(s * kQ8Keys + (lane & 15), n_keys - 1); };
  auto entry = [&](int s) -> int32_t { return ib[min(max(at(s) - ni, 0), (int)kl.idx_stride - 1)]; };
  const uint32_t ring = smem_u32(q8sm) + warp * (kQ8Stages * q8_stage_bytes<D>());
  auto issue = [&](int pos, uint32_t st) {
#pragma unroll
    for (int i = 0; i < kQ8Keys * CPR / 32; ++i) {
      // rows whose bits that place a value's pieces (q8_v_off) are the same for every i
      const int row = D == 128 ? 2 * cpr + (i & 1) + 8 * (i >> 1) : cpr + 8 * i;
      const uint64_t off = (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, pos, row) * row_bytes;
      cp_async16(st + q8_k_off<D>(row, cpc), kb + off, 16u);
      cp_async16(st + kQ8Keys * D + q8_v_off<D>(row, cpc), vb + off, 16u);
    }
    cp_async4(st + 2 * kQ8Keys * D + lane * 4, sb + (int64_t)(pos >> a.bshift) * a.hkv);
  };

  float acc[2 * VW][NT][4];              // O^T tiles: dims (2 t, 2 t + 1) of the lane's D / 8, rows 2 tig, 2 tig + 1
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m[nt][j] = -INFINITY;
      l[nt][j] = 0.f;
    }
#pragma unroll
  for (int t = 0; t < 2 * VW; ++t)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][nt][e] = 0.f;

  int s_n = s_beg;                       // the next step to issue
  int32_t raw[kAhead];                   // list entries of steps s_n, s_n + s_inc, ...
#pragma unroll
  for (int u = 0; u < kAhead; ++u) raw[u] = entry(s_n + u * s_inc);
  uint32_t st_n = ring;                  // and the ring slot it goes to
  const uint32_t ring_end = ring + kQ8Stages * q8_stage_bytes<D>();
  auto advance = [&](uint32_t st) { return st + q8_stage_bytes<D>() == ring_end ? ring : st + q8_stage_bytes<D>(); };
  auto issue_next = [&]() {
    if (s_n < s_end) {
      const int t = at(s_n), p = t < ni ? t : (t < ni + cnt ? raw[0] : t + jump);
      issue(min(max(p, 0), (int)a.n_cap - 1), st_n);
    }
    cp_async_commit();                   // one group per step, empty past the end
#pragma unroll
    for (int u = 0; u + 1 < kAhead; ++u) raw[u] = raw[u + 1];
    raw[kAhead - 1] = entry(s_n + kAhead * s_inc);
    s_n += s_inc;
    st_n = advance(st_n);
  };
#pragma unroll
  for (int i = 0; i < kQ8Stages - 1; ++i) issue_next();

  // ---- queries: B fragments, row gid of each group of 8, dims in the order of K's words
  uint32_t qf[NT][KC][4][2], ql[F32 ? NT : 1][KC][4][2];
  float xs[NT][2];                                             // logit factors of rows 2 tig, 2 tig + 1
  int lim[NT][2];                                              // first key they do not attend
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = min(r0 + nt * 8 + gid, a.lq * a.G - 1);
    const int i = r / a.G, hl = r - i * a.G;
    const T* qp = static_cast<const T*>(a.q) + (((int64_t)b * a.lq + i) * a.hq + g * a.G + hl) * D;
    float f[KC][4][4];
    float mx = 0.f;
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        load4(qp + c * 64 + tig * 16 + w * 4, f[c][w]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(f[c][w][e]));
      }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int qe = q8_query_exp(mx);
    const float up = __uint_as_float((uint32_t)(qe + 127) << 23);
    const float down = a.scale_log2 * __uint_as_float((uint32_t)(127 - qe) << 23);
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int w = 0; w < 4; ++w)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float x0 = f[c][w][q8_pair_dim<FMT>(p, 0)] * up, x1 = f[c][w][q8_pair_dim<FMT>(p, 1)] * up;
          qf[nt][c][w][p] = f16x2_rn(x0, x1);
          if constexpr (F32) {
            const float2 h = f16x2_to_float2(qf[nt][c][w][p]);
            ql[nt][c][w][p] = f16x2_rn(x0 - h.x, x1 - h.y);
          }
        }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      xs[nt][j] = __shfl_sync(0xffffffffu, down, 4 * (2 * tig + j));
      lim[nt][j] = n_prior + min(r0 + nt * 8 + 2 * tig + j, a.lq * a.G - 1) / a.G + 1;
    }
  }

  uint32_t st = ring;
  for (int s = s_beg; s < s_end; s += s_inc, st = advance(st)) {
    cp_async_wait<kQ8Stages - 2>();      // this lane's pieces of step s are here
    __syncwarp();                        // every lane's are, and every lane has left the slot filled next
    issue_next();
    uint4 kr[2][KC];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < KC; ++c) kr[u][c] = lds128(st + q8_k_off<D>(gid + 8 * u, tig + 4 * c));
    float sc_k[2], sc_v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      sc_k[u] = __uint_as_float(lds32(st + 2 * kQ8Keys * D + (gid + 8 * u) * 4));
      sc_v[u] = __uint_as_float(lds32(st + 2 * kQ8Keys * D + (16 + gid + 8 * u) * 4));
    }

    // S^T = Kc Q^T, two chains of half the dims
    float sx[NT][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) sx[nt][h][0] = sx[nt][h][1] = sx[nt][h][2] = sx[nt][h][3] = 0.f;
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t a0, a1, a2, a3;
        const uint4 &ka = kr[0][c], &kbb = kr[1][c];
        q8_pairs<FMT>(w == 0 ? ka.x : w == 1 ? ka.y : w == 2 ? ka.z : ka.w, a0, a2);
        q8_pairs<FMT>(w == 0 ? kbb.x : w == 1 ? kbb.y : w == 2 ? kbb.z : kbb.w, a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(sx[nt][w & 1], a0, a1, a2, a3, qf[nt][c][w][0], qf[nt][c][w][1]);
          if constexpr (F32) mma_f16(sx[nt][w & 1], a0, a1, a2, a3, ql[nt][c][w][0], ql[nt][c][w][1]);
        }
      }

    // softmax: keys gid and gid + 8 (u), rows 2 tig and 2 tig + 1 (j). The weights come
    // first, against m as it is; the row maxima (a reduction over 8 lanes) only when one of
    // them says that m has to rise (at once on the first step: m is -inf).
    float ka[2], vb[2];                  // scales of the two keys, the values' times 2^10
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      q8_scales(ka[u] = sc_k[u], vb[u] = sc_v[u]);
      vb[u] *= kQ8Unit;
    }
    const int t0 = s * kQ8Keys;
    const bool cut = t0 + kQ8Keys > n_all;                     // some row does not see some key
    float ex[NT][2][2], wt[NT][2][2];
    uint32_t wh[NT][2];                                        // the weights as f16, rows 2 tig, 2 tig + 1
    auto weights = [&]() -> bool {                             // whether one is above kQ8Most
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int u = 0; u < 2; ++u)
            ex[nt][u][j] = fast_exp2(fmaf(sx[nt][0][2 * u + j] + sx[nt][1][2 * u + j], ka[u] * xs[nt][j], -m[nt][j]));
      if (cut) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (t0 + gid + 8 * u >= lim[nt][j]) ex[nt][u][j] = 0.f;
      }
      uint32_t top = 0u;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          wt[nt][u][0] = ex[nt][u][0] * vb[u];
          wt[nt][u][1] = ex[nt][u][1] * vb[u];
          wh[nt][u] = f16x2_rn(wt[nt][u][0], wt[nt][u][1]);
          asm("max.f16x2 %0, %0, %1;" : "+r"(top) : "r"(wh[nt][u]));       // (not NaN, where one of the two is not)
        }
      return ((top + 0x80008000u - kQ8Most - 0x00010001u) & 0x80008000u) != 0u;
    };
    if (__any_sync(0xffffffffu, weights())) {
      const float lv[2] = {fast_log2(vb[0]) - kQ8Head, fast_log2(vb[1]) - kQ8Head};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float al[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = -INFINITY;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float x = fmaf(sx[nt][0][2 * u + j] + sx[nt][1][2 * u + j], ka[u] * xs[nt][j], lv[u]);
            if (t0 + gid + 8 * u < lim[nt][j]) mx = fmaxf(mx, x);
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[nt][j], mx);
          const float half = mn == -INFINITY ? 1.f : fast_exp2(0.5f * (m[nt][j] - mn));
          al[j] = half * half;
          m[nt][j] = mn;
          l[nt][j] = l[nt][j] * half * half;
        }
#pragma unroll
        for (int t = 0; t < 2 * VW; ++t) {
          acc[t][nt][0] *= al[0];
          acc[t][nt][1] *= al[1];
          acc[t][nt][2] *= al[0];
          acc[t][nt][3] *= al[1];
        }
      }
      weights();
    }
    uint32_t wf[NT][2], wl[F32 ? NT : 1][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int j = 0; j < 2; ++j) l[nt][j] += ex[nt][u][j];
        wf[nt][u] = movmatrix_t(wh[nt][u]);
        if constexpr (F32) {
          const float2 hf = f16x2_to_float2(wh[nt][u]);
          wl[nt][u] = movmatrix_t(f16x2_rn(wt[nt][u][0] - hf.x, wt[nt][u][1] - hf.y));
        }
      }

    // O^T += Vc^T W^T
    uint32_t vr[4][VW];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int row = 2 * tig + (u & 1) + 8 * (u >> 1);
      if constexpr (VW == 4) {
        const uint4 x4 = lds128(st + kQ8Keys * D + q8_v_off<D>(row, gid));
        vr[u][0] = x4.x; vr[u][1] = x4.y; vr[u][2] = x4.z; vr[u][3] = x4.w;
      } else {
        const uint2 x2 = lds64(st + kQ8Keys * D + q8_v_off<D>(row, gid >> 1) + (gid & 1) * 8);
        vr[u][0] = x2.x; vr[u][1] = x2.y;
      }
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      uint32_t da[4], db[4];
      q8_transpose<FMT>(vr[0][w], vr[1][w], da);       // keys 2 tig, 2 tig + 1
      q8_transpose<FMT>(vr[2][w], vr[3][w], db);       // keys 2 tig + 8, 2 tig + 9
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_f16(acc[2 * w + p][nt], da[2 * p], da[2 * p + 1], db[2 * p], db[2 * p + 1], wf[nt][0], wf[nt][1]);
          if constexpr (F32)
            mma_f16(acc[2 * w + p][nt], da[2 * p], da[2 * p + 1], db[2 * p], db[2 * p + 1], wl[nt][0], wl[nt][1]);
        }
    }
  }
  cp_async_wait_all();
  __syncthreads();                       // the rings are free: the merge reuses them

  // ---- the warp's rows to shared memory
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 4);
      l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 8);
      l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], 16);
      const int r = nt * 8 + 2 * tig + j;
      if (r >= nrow) continue;
      float* p = sm_o + (warp * ROWS + r) * RF + gid * (D / 8);
#pragma unroll
      for (int t = 0; t < 2 * VW; ++t)
        *reinterpret_cast<float2*>(p + 2 * t) = make_float2(acc[t][nt][j], acc[t][nt][2 + j]);
      if (gid == 0) *reinterpret_cast<float2*>(sm_ml + (warp * ROWS + r) * 2) = make_float2(m[nt][j], l[nt][j]);
    }
  __syncthreads();
  // merge the warps of the CTA, into the first one's rows
  constexpr int Q = D / 4;
  for (int it = threadIdx.x; it < nrow * Q; it += kQ8Threads) {
    const int d4 = it % Q, r = it / Q;
    float M = -INFINITY;
#pragma unroll
    for (int u = 0; u < kQ8Warps; ++u) M = fmaxf(M, sm_ml[(u * ROWS + r) * 2]);
    const float mr = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kQ8Warps; ++u) {
      const int wr = u * ROWS + r;
      const float half = fast_exp2(0.5f * (sm_ml[wr * 2] - mr)), c = half * half;
      const float4 o = *reinterpret_cast<const float4*>(sm_o + wr * RF + d4 * 4);
      L += sm_ml[wr * 2 + 1] * half * half;
      O.x += o.x * c; O.y += o.y * c; O.z += o.z * c; O.w += o.w * c;
    }
    *reinterpret_cast<float4*>(sm_o + r * RF + d4 * 4) = O;                  // read by this thread only
    if (d4 == 0) *reinterpret_cast<float2*>(sm_fin + r * 2) = make_float2(M, L);
  }
  if (csize > 1) cluster_sync_all();
  else __syncthreads();
  // merge the CTAs of the cluster: CTA `rank` writes every csize-th group of 256 items
  for (int it = threadIdx.x + kQ8Threads * rank; it < nrow * Q; it += kQ8Threads * csize) {
    const int d4 = it % Q, r = it / Q;
    const uint32_t ml = smem_u32(sm_fin + r * 2), oo = smem_u32(sm_o + r * RF + d4 * 4);
    float M = -INFINITY;
    for (int u = 0; u < csize; ++u) M = fmaxf(M, __uint_as_float(ld_dsmem_u32(dsmem_map(ml, u))));
    const float mr = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int u = 0; u < csize; ++u) {
      const uint2 z = ld_dsmem_u2(dsmem_map(ml, u));
      const float4 o = ld_dsmem_f4(dsmem_map(oo, u));
      const float half = fast_exp2(0.5f * (__uint_as_float(z.x) - mr)), c = half * half;
      L += __uint_as_float(z.y) * half * half;
      O.x += o.x * c; O.y += o.y * c; O.z += o.z * c; O.w += o.w * c;
    }
    const int i = a.lq == 1 ? 0 : (r0 + r) / a.G, hl = (r0 + r) - i * a.G;
    const int64_t row = ((int64_t)b * a.lq + i) * a.hq + g * a.G + hl;
    const float inv = 1.f / kQ8Unit / L;
    T* dst = static_cast<T*>(a.o) + row * D + d4 * 4;
    if constexpr (F32) {
      *reinterpret_cast<float4*>(dst) = make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
    } else {
      uint2 w;
      w.x = bf16x2_rn(O.x * inv, O.y * inv);
      w.y = bf16x2_rn(O.z * inv, O.w * inv);
      *reinterpret_cast<uint2*>(dst) = w;
    }
    if (d4 == 0 && a.lse) a.lse[row] = (M + __log2f(L)) * 0.69314718055994531f;
  }
  if (csize > 1) cluster_sync_all();                                         // no CTA leaves while it is read
}

// Chunks: the tensor-core attention over the staged rows [B, t_pad, Hkv, D] of the whole key
// list (cache_stage_q8_kernel), so every key tile is one box. Heads of 64 fill the first half
// of the 128 columns: the maps' rows end there, and a load behind them brings zeros. A group
// that does not divide 128 rows gathers its queries (heads of 128), or goes in `parts` parts
// that do, each a head of its own here (heads of 64, whose rows a gather would overrun).
struct Q8TcProblem : EsaTcProblem {
  int64_t t_pad;
  int d;
  int parts;             // G is that of a part, blockIdx.y counts parts
  bool boxed;            // Q tiles are boxes
  int kvh;               // per CTA: the KV head
  __device__ bool setup() {
    tile = blockIdx.x;
    g = blockIdx.y;
    b = blockIdx.z;
    if (tile * kTcRows >= lq * G) return false;
    kvh = g / parts;
    list = lists > 1 ? b * lists + kvh : b;
    cnt = min(max(keys.count[list], 0), (int)keys.idx_stride);
    n_prior = keys.ni + cnt + (c0 - keys.lo);
    nk = n_prior + min(lq - 1, (tile * kTcRows + kTcRows - 1) / G) + 1;
    return true;
  }
  __device__ bool q_box(int* y, int* z) const { return boxed && EsaTcProblem::q_box(y, z); }
  __device__ int32_t kv_row(int64_t t) const { return (int32_t)(((int64_t)b * t_pad + t) * hkv + kvh); }
  __device__ int kv_box(int j, int* y, int* z) const {
    *y = kvh;
    *z = (int)((int64_t)b * t_pad + (int64_t)j * kTcKeys);
    return 1;
  }
  __device__ void store(int r, int col0, const float* acc, float m2, float l) {
    if (d == kTcD) return EsaTcProblem::store(r, col0, acc, m2, l);
    const int R = tile * kTcRows + r;
    if (R >= lq * G || col0 >= d) return;
    const int i = R / G, hl = R % G;
    const int64_t row = ((int64_t)b * lq + i) * hq + g * G + hl;
    const float inv = 1.f / l;
    uint4* dst = reinterpret_cast<uint4*>(o + row * d + col0);
#pragma unroll
    for (int c = 0; c < kTcD / kTcSplit / 8; ++c)
      dst[c] = make_uint4(pack_bf16x2(acc[8 * c] * inv, acc[8 * c + 1] * inv),
                          pack_bf16x2(acc[8 * c + 2] * inv, acc[8 * c + 3] * inv),
                          pack_bf16x2(acc[8 * c + 4] * inv, acc[8 * c + 5] * inv),
                          pack_bf16x2(acc[8 * c + 6] * inv, acc[8 * c + 7] * inv));
    if (lse && col0 == 0) lse[row] = (m2 + __log2f(l)) * 0.69314718055994531f;
  }
};

}  // namespace esa
