// cache_q8.cuh - the 8-bit key/value cache: rows quantised as they are written, and read
// back.
//
// A cache operand holds codes [B, n_cap, Hkv, D] (e4m3 or int8) and one fp32 scale for
// each block of 2^bshift tokens and head, [B, ceil(n_cap / block), Hkv]; the value of a
// code is code * scale. Writing rows into a block gives it
//   s' = max(s of the rows already in the block, 2^E),
//   E  = the smallest integer with  max |new x| <= qmax 2^E  (qmax 448 / 127; E >= -100),
// stores the new rows as round(x / s') and, where s' > s, the older rows as
// round(code s / s'). The scale is a power of two on purpose: x / s' and code * s' are then
// exact in fp32 (and code * s' in bf16, whose 8 significant bits hold every code), so a
// code is the correctly rounded one whatever the order of the arithmetic, reading a row
// back rounds nothing, and a growing scale costs the older rows one rounding of a halving
// (e4m3: none, above its subnormals). An e4m3 code keeps its 3 mantissa bits under any
// scale; an int8 code gives up to one of its 7 bits for it.
#pragma once
#include "common.cuh"
#include "keylist.cuh"

namespace esa {

// Programmatic dependent launch: a kernel launched with the attribute may be set up while
// the one before it in the stream still drains; nothing of global memory may be touched
// before this wait, which returns once that kernel is complete and its writes are visible.
// What a kernel before may have written (rows, codes, scales, lists, queries) is then read by
// plain loads: the read-only path (ld.global.nc, __ldg) is for data that nothing writes in the
// kernel's whole lifetime, which begins under the writer, and the compiler may lift such a
// load above the wait.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

constexpr int kQ8E4M3 = 0, kQ8Int8 = 1;
constexpr int kQ8LeastExp = -100;          // scales stay normal, and so do their reciprocals

// ------------------------------------------------------------------ codes <-> values --
// two e4m3 codes (the low 16 bits of a register) as f16, exact
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return h;
}
__device__ __forceinline__ float2 f16x2_to_float2(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// four codes of a word as fp32
template <int FMT>
__device__ __forceinline__ void q8_widen4(uint32_t w, float* f) {
  if constexpr (FMT == kQ8E4M3) {
    const float2 a = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)w));
    const float2 b = f16x2_to_float2(e4m3x2_to_f16x2((uint16_t)(w >> 16)));
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  } else {
    // 0x4b000000 | (c + 128) is the float 2^23 + 128 + c
    w ^= 0x80808080u;
    f[0] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)) - 8388736.f;
    f[1] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441)) - 8388736.f;
    f[2] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)) - 8388736.f;
    f[3] = __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443)) - 8388736.f;
  }
}
// Four values times inv (a power of two) as codes: nearest, ties to even. The products fit
// the format (|f inv| <= qmax); e4m3 saturates besides.
template <int FMT>
__device__ __forceinline__ uint32_t q8_narrow4(const float* f, float inv) {
  if constexpr (FMT == kQ8E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1] * inv), "f"(f[0] * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3] * inv), "f"(f[2] * inv));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  } else {
    // 1.5 * 2^23 + c holds c's two's complement in its low bits; the product is exact, so
    // the sum's rounding is the one to the nearest integer
    uint32_t g[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = __float_as_uint(fmaf(f[e], inv, 12582912.f));
    return __byte_perm(__byte_perm(g[0], g[1], 0x0040), __byte_perm(g[2], g[3], 0x0040), 0x5410);
  }
}

// The smallest power of two s >= 2^kQ8LeastExp with amax <= qmax * s, from the bits of a
// finite amax >= 0. qmax is 1.75 * 2^8 (e4m3) or 1.984375 * 2^6 (int8): the exponent goes
// up by one when amax's mantissa is above that of qmax.
template <int FMT>
__device__ __forceinline__ float q8_scale_of(uint32_t amax_bits) {
  constexpr int top_exp = FMT == kQ8E4M3 ? 8 : 6;
  constexpr uint32_t top_mant = FMT == kQ8E4M3 ? 0x600000u : 0x7e0000u;
  int e = (int)(amax_bits >> 23) - 127 - top_exp + ((amax_bits & 0x7fffffu) > top_mant ? 1 : 0);
  e = max(e, kQ8LeastExp);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// ------------------------------------------------------------------------- write --
struct CacheWriteArgs {
  const void* x[2];        // new keys, new values: row (b, r) at x + b * bs + r * rs, [Hkv, D] contiguous
  int64_t bs[2], rs[2];    // elements
  uint8_t* codes[2];       // [B, n_cap, Hkv, D]
  float* scale[2];         // [B, nblk, Hkv]
  int64_t n_cap, nblk;
  int64_t start;           // first position (no device lengths)
  int64_t rows;            // new rows of a sequence (the most, with new_len)
  const int64_t* seq_len;  // null, or [B]: rows end at seq_len[b]
  const int64_t* new_len;  // null, or [B]: new rows of sequence b
  int hkv, bshift;
  bool wide;               // rows of x are 32-byte aligned
};

// Positions [start, end) that sequence b writes. False: nothing (an empty write, or
// lengths that do not fit the cache: recorded, the sequence is left as it was).
__device__ __forceinline__ bool q8_write_range(const CacheWriteArgs& a, int b, int64_t& start, int64_t& end) {
  if (!a.seq_len) {
    start = a.start;
    end = a.start + a.rows;
    return true;
  }
  const int64_t t = a.new_len ? a.new_len[b] : a.rows;
  end = a.seq_len[b];
  if (t == 0) return false;
  if (t < 0 || t > a.rows || end < t || end > a.n_cap) {
    if (threadIdx.x == 0) record_status(8u, 705);
    return false;
  }
  start = end - t;
  return true;
}

// 16 bytes that are read once
__device__ __forceinline__ uint4 ld_once16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// 32 bytes of global memory in one load (they are 32-byte aligned), or in two
__device__ __forceinline__ void ld_global_32(const void* p, bool wide, uint32_t* w) {
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = ld_once16(p), b = ld_once16(static_cast<const uint8_t*>(p) + 16);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}

// One CTA per (block of tokens, head, operand) of a sequence: block * D / 64 threads, so
// that a thread holds 16 elements of each of 4 rows in registers and the block is read
// once: load everything, take the maximum, scale, round, store. Bound by HBM (and by
// launch and one memory latency for a single token). grid (blocks * 2 Hkv, B), heads
// fastest: the CTAs that share rows run together, so DRAM pages are read whole.
// 32768 tokens of 8 heads of 128 (201 MB): 31.2 us, 6.4 TB/s, of fp32 rows (336 MB) 50.2 us,
// 6.7 TB/s. (16-byte loads of 8 elements a row and thread: 39.1 us where these 32-byte loads
// took 33.7.)
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(256) cache_write_q8_kernel(const CacheWriteArgs a) {
  constexpr int TPR = D / 16;                      // threads of a row
  constexpr int W = 16 * sizeof(T) / 4;            // 32-bit words of 16 elements: 8 or 16
  constexpr int NP = 4;                            // rows of a thread
  const uint32_t width = 2u * a.hkv, yb = blockIdx.x / width, col = blockIdx.x - yb * width;
  const int op = col >= (uint32_t)a.hkv, h = col - (op ? a.hkv : 0), b = blockIdx.y;
  pdl_wait();
  int64_t start, end;
  if (!q8_write_range(a, b, start, end)) return;
  const int64_t blk = (start >> a.bshift) + yb;
  const int64_t base = blk << a.bshift;
  if (base >= end) return;
  const int block = 1 << a.bshift;
  const int row0 = threadIdx.x / TPR, piece = threadIdx.x % TPR, rpp = blockDim.x / TPR;
  const T* src = static_cast<const T*>(op ? a.x[1] : a.x[0]) + (int64_t)b * a.bs[op] + (int64_t)h * D + piece * 16;
  const int64_t rs = a.rs[op];
  float* sc = a.scale[op] + ((int64_t)b * a.nblk + blk) * a.hkv + h;
  uint8_t* codes = a.codes[op] + ((int64_t)b * a.n_cap * a.hkv + h) * D;     // + position * Hkv * D
  const int64_t cs = (int64_t)a.hkv * D;

  uint32_t x[NP][W];
  bool mine[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = row0 + p * rpp;
    const int64_t pos = base + r;
    mine[p] = r < block && pos >= start && pos < end;
#pragma unroll
    for (int w = 0; w < W; ++w) x[p][w] = 0u;
    if (mine[p]) {
#pragma unroll
      for (int q = 0; q < W / 8; ++q) ld_global_32(src + (pos - start) * rs + q * 8, a.wide, x[p] + q * 8);
    }
  }
  float old = start > base ? *sc : 0.f;            // rows before the write hold their values under it
  old = old > 0.f && old < INFINITY ? old : 0.f;

  // maximum magnitude as bits: of floats >= 0 the order of the bits is the order of the
  // values, and infinities and NaN come out on top
  auto block_max = [&](uint32_t mx) -> uint32_t {
    __shared__ uint32_t part[8];
    mx = __reduce_max_sync(0xffffffffu, mx);
    if (blockDim.x > 32) {
      __syncthreads();
      if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = mx;
      __syncthreads();
      for (int w = 0; w < (int)blockDim.x >> 5; ++w) mx = max(mx, part[w]);
    }
    return mx;
  };
  uint32_t mx = 0;
#pragma unroll
  for (int p = 0; p < NP; ++p)
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if constexpr (sizeof(T) == 2) mx = __vmaxu2(mx, x[p][w] & 0x7fff7fffu);
      else mx = max(mx, x[p][w] & 0x7fffffffu);
    }
  if constexpr (sizeof(T) == 2) mx = max(mx & 0xffff0000u, mx << 16);
  mx = block_max(mx);
  const bool finite = mx < 0x7f800000u;
  // applies fn to the bits of every element and puts them back
  auto each = [&](auto fn) {
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if constexpr (sizeof(T) == 4) x[p][w] = fn(x[p][w]);
        else x[p][w] = (fn(x[p][w] & 0xffff0000u) & 0xffff0000u) | (fn(x[p][w] << 16) >> 16);
      }
  };
  if (!finite) {
    // NaN becomes 0, an infinity the largest code of a block scaled by its finite values;
    // recorded for the host
    if (threadIdx.x == 0) record_status(7u, 705);
    uint32_t fin = 0;
    each([&](uint32_t v) {
      const uint32_t m = v & 0x7fffffffu;
      if (m < 0x7f800000u) fin = max(fin, m);
      return m > 0x7f800000u ? 0u : v;
    });
    mx = block_max(fin);
  }
  const float s = fmaxf(q8_scale_of<FMT>(mx), old);
  const float inv = 1.f / s;                       // exact: powers of two
  float up = inv;
  if (!finite) {
    // all elements times 2^-10, so that an infinity's stand-in qmax s is finite under every s
    // (what becomes subnormal is a code of 0 either way)
    uint32_t top = __float_as_uint((FMT == kQ8E4M3 ? 448.f : 127.f) * 0x1p-10f * s);
    if constexpr (sizeof(T) == 2) top = (top + 0xffffu) & 0xffff0000u;
    each([&](uint32_t v) {
      return (v & 0x7fffffffu) == 0x7f800000u ? (v & 0x80000000u) | top : __float_as_uint(__uint_as_float(v) * 0x1p-10f);
    });
    up = inv * 0x1p10f;
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if (!mine[p]) continue;
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) f[e] = __uint_as_float(x[p][4 * q + e]);
        else f[e] = __uint_as_float((e & 1) ? x[p][2 * q + e / 2] & 0xffff0000u : x[p][2 * q + e / 2] << 16);
      }
      c[q] = q8_narrow4<FMT>(f, up);
    }
    *reinterpret_cast<uint4*>(codes + (base + row0 + p * rpp) * cs + piece * 16) = make_uint4(c[0], c[1], c[2], c[3]);
  }
  if (start > base && s > old) {
    // the block's scale grew: the rows already there move to it
    const float ratio = old * inv;
    const int n = (int)(start - base) * (D / 16);
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      uint4* p = reinterpret_cast<uint4*>(codes + (base + i / (D / 16)) * cs) + i % (D / 16);
      uint4 v = *p;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[4];
        q8_widen4<FMT>(w[q], f);
        w[q] = q8_narrow4<FMT>(f, ratio);
      }
      *p = v;
    }
  }
  // every thread has read the old scale before block_max's barriers
  if (blockDim.x <= 32) __syncwarp();
  if (threadIdx.x == 0) *sc = s;
}

// -------------------------------------------------------------------------- read --
// 32 bytes of values to global memory in one store
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// N = 32 / sizeof(T) codes at src times s as 32 bytes of T at dst
template <typename T, int FMT>
__device__ __forceinline__ void q8_widen_store(const uint32_t* c, float s, T* dst) {
  constexpr int N = 32 / sizeof(T);
  float f[N];
#pragma unroll
  for (int q = 0; q < N / 4; ++q) q8_widen4<FMT>(c[q], f + 4 * q);
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (sizeof(T) == 2) w[e] = bf16x2_rn(f[2 * e] * s, f[2 * e + 1] * s);
    else w[e] = __float_as_uint(f[e] * s);
  }
  st_global_32(dst, w);
}
template <int BYTES>
__device__ __forceinline__ void q8_load_codes(const uint8_t* p, uint32_t* c) {
  if constexpr (BYTES == 16) {
    const uint4 v = ld_once16(p);
    c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    c[0] = v.x; c[1] = v.y;
  }
}

struct CacheReadArgs {
  const uint8_t* codes[2];
  const float* scale[2];
  void* out[2];             // [B, n, Hkv, D]; null: not wanted
  const int32_t* idx;       // null, or [B, n]
  int64_t n_cap, nblk, start, n;
  int hkv, d, bshift;
};

constexpr int kReadThreads = 256, kReadPer = 4;

// How threads lie over result rows of `pieces` 32-byte pieces: a CTA takes up to 256
// columns (more: several CTAs side by side) and as many rows a pass as fit, kReadPer
// passes. A thread keeps its column, so only rows change from piece to piece.
struct ReadTile {
  int cols, col_ctas, rows;   // columns and column CTAs, rows of a pass
  __host__ __device__ explicit ReadTile(int pieces) {
    cols = pieces < kReadThreads ? pieces : kReadThreads;
    col_ctas = (pieces + kReadThreads - 1) / kReadThreads;
    rows = kReadThreads / cols;
  }
};

// Codes at pos[u] (negative: zeros) of a thread's column, times their scales, to rows
// row0 + u * rows of the result.
template <typename T, int FMT>
__device__ __forceinline__ void q8_move(const uint8_t* codes, const float* scale, uint32_t row_bytes, int hkv,
                                        int bshift, const int (&pos)[kReadPer], T* out, int64_t row0, int rows,
                                        int64_t n) {
  constexpr int N = 32 / sizeof(T);
  uint32_t c[kReadPer][N / 4];
  float s[kReadPer];
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    // (a row that is not wanted loads row 0: a branch here would put each conversion
    // behind its own load)
    const uint32_t at = max(pos[u], 0);
    q8_load_codes<N>(codes + (uint64_t)at * row_bytes, c[u]);
    s[u] = scale[(uint64_t)(at >> bshift) * (uint32_t)hkv];
  }
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    if (pos[u] < 0) {
      s[u] = 0.f;
#pragma unroll
      for (int q = 0; q < N / 4; ++q) c[u][q] = 0u;
    }
  }
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    const int64_t r = row0 + u * rows;
    if (r < n) q8_widen_store<T, FMT>(c[u], s[u], out + r * row_bytes);      // row_bytes elements a row
  }
}

// Row (b, r) of the result is cache row start + r, or idx[b, r] (zeros where that is not a
// row of the cache). A thread makes 32 bytes of the result from 16 (8) codes, kReadPer
// rows with their loads in flight together (2, 4, 8 rows: 7.7, 7.4, 8.3 us for 8192 listed
// rows of 8 heads of 128, 31.1, 31.1, 31.3 for 32000 consecutive ones). Bound by HBM, two
// thirds of it writes: 197 MB in 30.9 us, 6.36 TB/s; to fp32 328 MB in 50.2 us, 6.53 TB/s (a
// device copy of 262 MB: 41.6 us, 6.30 TB/s).
// grid (row tiles * column CTAs, B, operands).
template <typename T, int FMT>
__global__ void __launch_bounds__(kReadThreads) cache_read_q8_kernel(const CacheReadArgs a) {
  constexpr int N = 32 / sizeof(T);
  const int op = blockIdx.z, b = blockIdx.y;
  // (indexed by op, the arguments would be copied to local memory)
  T* out = static_cast<T*>(op ? a.out[1] : a.out[0]);
  if (!out) return;
  const uint32_t row_bytes = (uint32_t)(a.hkv * a.d);
  const ReadTile tile(row_bytes / N);
  const int rt = blockIdx.x / tile.col_ctas, cc = blockIdx.x - rt * tile.col_ctas;
  const int tr = threadIdx.x / tile.cols, col = cc * kReadThreads + threadIdx.x - tr * tile.cols;
  if (tr >= tile.rows || col * N >= row_bytes) return;
  const int64_t row0 = (int64_t)rt * (tile.rows * kReadPer) + tr;
  pdl_wait();
  int pos[kReadPer];
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    const int64_t r = row0 + u * tile.rows;
    pos[u] = r < a.n ? (a.idx ? a.idx[(int64_t)b * a.n + r] : (int)(a.start + r)) : -1;
  }
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) pos[u] = pos[u] < a.n_cap ? pos[u] : -1;
  q8_move<T, FMT>((op ? a.codes[1] : a.codes[0]) + (int64_t)b * a.n_cap * row_bytes + col * N,
                  (op ? a.scale[1] : a.scale[0]) + (int64_t)b * a.nblk * a.hkv + col * N / a.d, row_bytes, a.hkv, a.bshift, pos,
                  out + (int64_t)b * a.n * row_bytes + col * N, row0, tile.rows, a.n);
}

// The whole key list of a chunk (initial, selected, local and the chunk itself; one list
// per sequence, or one per KV head) as bf16 rows [B, t_pad, Hkv, D] for the tensor-core
// attention; rows behind the list are zeros, to the end of its last key tile.
// grid as above.
struct CacheStageArgs {
  const uint8_t* codes[2];
  const float* scale[2];
  __nv_bfloat16* out[2];
  KeyList keys;
  int64_t n_cap, nblk, c0, t_pad;
  int lq, hkv, d, lists, bshift;
};
constexpr int kStageTile = 128;           // keys of a tile of the attention; t_pad is a multiple

template <int FMT>
__global__ void __launch_bounds__(kReadThreads) cache_stage_q8_kernel(const CacheStageArgs a) {
  const int op = blockIdx.z, b = blockIdx.y;
  const uint32_t row_bytes = (uint32_t)(a.hkv * a.d);
  const ReadTile tile(row_bytes / 16);
  const int rt = blockIdx.x / tile.col_ctas, cc = blockIdx.x - rt * tile.col_ctas;
  const int tr = threadIdx.x / tile.cols, col = cc * kReadThreads + threadIdx.x - tr * tile.cols;
  if (tr >= tile.rows || col * 16 >= row_bytes) return;
  const int64_t row0 = (int64_t)rt * (tile.rows * kReadPer) + tr;
  pdl_wait();
  const int g = col * 16 / a.d, list = a.lists > 1 ? b * a.lists + g : b;
  const int cnt = min(max(a.keys.count[list], 0), (int)a.keys.idx_stride);
  const int64_t n_keys = a.keys.ni + cnt + (a.c0 - a.keys.lo) + a.lq;
  int pos[kReadPer];
#pragma unroll
  for (int u = 0; u < kReadPer; ++u) {
    const int64_t t = row0 + u * tile.rows;
    pos[u] = t < n_keys ? (int)a.keys.pos(list, cnt, t) : -1;
  }
  q8_move<__nv_bfloat16, FMT>(a.codes[op] + (int64_t)b * a.n_cap * row_bytes + col * 16,
                              a.scale[op] + (int64_t)b * a.nblk * a.hkv + g, row_bytes, a.hkv, a.bshift, pos,
                              a.out[op] + (int64_t)b * a.t_pad * row_bytes + col * 16, row0, tile.rows,
                              (n_keys + kStageTile - 1) / kStageTile * kStageTile);
}

}  // namespace esa
