// paged.cuh -- kernels of the paged prefix-KV cache (include/mot_paged.h):
// norm + rotation + cache write of a chunk, dense <-> pages, and grouped-query
// attention of few query rows per sequence over the pages.
#pragma once

#include <cfloat>
#include <climits>
#include <type_traits>

#include "ptx.cuh"

namespace mot {

// ---------------------------------------------------------------- e4m3 rows
// value of an e8m0 scale byte: 2^(b - 127), 255 = NaN (2^-127 is an f32 subnormal)
__device__ __forceinline__ float e8m0_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}

// Scale byte of a row with largest magnitude amax: 127 + e, e the smallest
// integer with amax <= 448 * 2^e, at least -64; 255 when amax is not finite.
// amax = m 2^x with 1 <= m < 2 and 448 = 1.75 * 2^8, so e = x - 8, or x - 7 when
// m > 1.75: adding 2^21 - 1 to the bits carries into the exponent exactly then.
__device__ __forceinline__ uint32_t e8m0_of_amax(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  if (bits >= 0x7f800000u) return 255u;
  const int e = static_cast<int>((bits + 0x1fffffu) >> 23) - 8;
  return static_cast<uint32_t>(max(e, 127 - 64));
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// two e4m3 (low half of w) -> f16 pair, exact
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}

// four e4m3 -> two f16 pairs, exact
__device__ __forceinline__ void e4m3x4_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// untiled bulk copy: addresses and size multiples of 16 bytes
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Biased exponent x of the power of two that a query row with largest magnitude
// amax is divided by to be held in f16: amax / 2^(x - 127) < 4, both 2^(x - 127) and
// its inverse normal f32. A row that is not finite stays as it is.
__device__ __forceinline__ uint32_t query_exponent(float amax) {
  const uint32_t x = (__float_as_uint(amax) >> 23) & 255u;
  return x == 255u ? 127u : min(max(x, 1u), 253u);
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& w, float (&f)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&f)[8]) {
  return make_uint4(pack_bf162(f[0], f[1]), pack_bf162(f[2], f[3]), pack_bf162(f[4], f[5]), pack_bf162(f[6], f[7]));
}

// largest magnitude of 8 values; a NaN among them comes out as NaN
__device__ __forceinline__ float amax8(const float (&f)[8]) {
  float m = fmax3_nan(fabsf(f[0]), fabsf(f[1]), fabsf(f[2]));
  m = fmax3_nan(m, fabsf(f[3]), fabsf(f[4]));
  m = fmax3_nan(m, fabsf(f[5]), fabsf(f[6]));
  return fmax3_nan(m, fabsf(f[7]), 0.f);
}

__device__ __forceinline__ uint2 quant8(const float (&f)[8], uint32_t scale) {
  if (scale == 255u) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
  const float inv = __uint_as_float((254u - scale) << 23);  // 2^-e, exact (scale in [63, 247])
  return make_uint2(pack_e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                    pack_e4m3x4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
}

// 8 e4m3 values times the row's scale as bf16 (exact)
__device__ __forceinline__ uint4 dequant8(uint2 w, float scale) {
  float f[8];
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_f16x2(u[i >> 1] >> (16 * (i & 1)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    f[2 * i] = v.x * scale;
    f[2 * i + 1] = v.y * scale;
  }
  return pack_bf16x8(f);
}

// ---------------------------------------------------------------- RoPE table
struct RopeFreq {
  double inv[64];
};

// (cos, sin) of p theta^(-2j/128), angle in f64, rounded to f32
__global__ void __launch_bounds__(256) paged_rope_kernel(float2* tab, int positions, const RopeFreq freq) {
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < positions * 64ll; i += gridDim.x * 256ll) {
    double s, c;
    sincos(static_cast<double>(i >> 6) * freq.inv[i & 63], &s, &c);
    tab[i] = make_float2(static_cast<float>(c), static_cast<float>(s));
  }
}

// ---------------------------------------------------------------- pool view
struct PagedPool {
  uint8_t *k, *v;
  uint8_t *ks, *vs;  // e8m0 rows, e4m3 pools only
};

// ---------------------------------------------------------------- append
struct PagedAppendParams {
  const uint4* qkv;    // bf16 [T, Hq + 2 Hkv, 128]
  uint4* q;            // bf16 [T, Hq, 128]
  PagedPool pool;
  const float* gains;  // q_norm [128], k_norm [128]
  const float2* rope;  // [positions, 64]
  const int2* tok;     // per token: position, page
  int T, Hq, Hkv, page_mask, page_shift;
  float eps;
};

// Eight lanes share a head, lane e holding dims 8e..8e+7 and 64 + 8e..+7, so that
// the rotate-half pair (j, j + 64) sits in one lane, all loads and stores are 16
// bytes, the norm is three shuffles, and the eight (cos, sin) pairs of a lane
// serve all its heads; a warp has four heads at a time, and the loads of kQuads
// such fours are issued before the first is used. kWhole: a warp takes a whole
// token, the next fours on their way; else a token is cut into strips of kQuads.
// Few tokens: a warp's chain of loads and norms. Many: no unit is full (bytes 4.5 of
// 6.6 TB/s, issue 54%); two sets of four heads in 128 registers leave 16 warps an SM.
// 2 x 4096 tokens of 32/8 heads into e4m3 41 us, 4.5 TB/s, into bf16 42 us, 4.75; one
// token 1.8 us in a graph, 4.0 us called from Python.
template <bool kE4m3, int kQuads, bool kWhole>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
  grid_dep_launch();
  const int H = p.Hq + 2 * p.Hkv;
  const int quads = (H + 3) >> 2;
  const int strips = kWhole ? 1 : (quads + kQuads - 1) / kQuads;  // pieces a token is cut into
  const long long work = static_cast<long long>(p.T) * strips;
  const int lane = lane_id(), sub = lane >> 3, e = lane & 7;
  long long w = blockIdx.x * 8ll + warp_id();
  int2 tok = make_int2(0, 0);
  if (w < work) tok = p.tok[w / strips];  // the batch's tables are written by copies, never by a kernel
  grid_dep_wait();
  while (w < work) {
    const int t = static_cast<int>(w / strips);
    const int q_begin = kWhole ? 0 : static_cast<int>(w % strips) * kQuads, q_end = kWhole ? quads : q_begin + 1;
    const uint4* src = p.qkv + (static_cast<long long>(t) * H + sub) * 16 + e;
    uint4 x[kQuads][2], y[kQuads][2];
    auto load = [&](uint4 (&v)[kQuads][2], int q0) {
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
        if (4 * (q0 + i) + sub < H) {
          v[i][0] = __ldcs(src + 64 * (q0 + i));
          v[i][1] = __ldcs(src + 64 * (q0 + i) + 8);
        }
      }
    };
    load(x, q_begin);
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float4 r = __ldg(reinterpret_cast<const float4*>(p.rope + static_cast<long long>(tok.x) * 64 + 8 * e) + (i >> 1));
      cs[i] = r.x;
      sn[i] = r.y;
      cs[i + 1] = r.z;
      sn[i + 1] = r.w;
    }
    const long long page_row = static_cast<long long>(tok.y) * p.Hkv;
    const int off = tok.x & p.page_mask;
    const long long next = w + gridDim.x * 8ll;
    if (next < work) tok = p.tok[next / strips];
    for (int q0 = q_begin; q0 < q_end; q0 += kQuads) {
      if (kWhole && q0 + kQuads < q_end) load(y, q0 + kQuads);
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const int h = 4 * (q0 + i) + sub;
        if (4 * (q0 + i) >= H) break;
        const bool live = h < H, is_v = h >= p.Hq + p.Hkv;
        const bool some_qk = 4 * (q0 + i) < p.Hq + p.Hkv, some_kv = 4 * (q0 + i) + 3 >= p.Hq;  // of the warp's four
        float a[8], b[8];
        unpack_bf16x8(x[i][0], a);
        unpack_bf16x8(x[i][1], b);
        if (some_qk) {
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int d = 0; d < 8; d += 2) {
            ffma2(s0, s1, a[d], a[d + 1], a[d], a[d + 1], s0, s1);
            ffma2(s0, s1, b[d], b[d + 1], b[d], b[d + 1], s0, s1);
          }
          float ss = s0 + s1;
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (!is_v) {
            const float rstd = __frsqrt_rn(ss * (1.0f / 128.0f) + p.eps);
            const float4* gain = reinterpret_cast<const float4*>(p.gains + (h < p.Hq ? 0 : 128) + 8 * e);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 ga = __ldg(gain + q), gb = __ldg(gain + 16 + q);
              const float fa[4] = {ga.x, ga.y, ga.z, ga.w}, fb[4] = {gb.x, gb.y, gb.z, gb.w};
#pragma unroll
              for (int k = 0; k < 4; k += 2) {
                const int d = 4 * q + k;
                float u0, u1, v0, v1, t0, t1;
                fmul2(u0, u1, a[d], a[d + 1], rstd, rstd);
                fmul2(v0, v1, b[d], b[d + 1], rstd, rstd);
                fmul2(u0, u1, u0, u1, fa[k], fa[k + 1]);
                fmul2(v0, v1, v0, v1, fb[k], fb[k + 1]);
                fmul2(t0, t1, v0, v1, sn[d], sn[d + 1]);
                ffma2(a[d], a[d + 1], u0, u1, cs[d], cs[d + 1], -t0, -t1);
                fmul2(t0, t1, u0, u1, sn[d], sn[d + 1]);
                ffma2(b[d], b[d + 1], v0, v1, cs[d], cs[d + 1], t0, t1);
              }
            }
          }
        }
        if (kE4m3 && some_kv) {
          float m = fmax3_nan(amax8(a), amax8(b), 0.f);
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) m = fmax3_nan(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
          if (live && h >= p.Hq) {
            const int g = h - p.Hq - (is_v ? p.Hkv : 0);
            const long long row = ((page_row + g) << p.page_shift) + off;
            uint8_t* dst = (is_v ? p.pool.v : p.pool.k) + row * 128;
            const uint32_t sc = e8m0_of_amax(m);
            reinterpret_cast<uint2*>(dst)[e] = quant8(a, sc);
            reinterpret_cast<uint2*>(dst)[8 + e] = quant8(b, sc);
            if (e == 0) (is_v ? p.pool.vs : p.pool.ks)[row] = static_cast<uint8_t>(sc);
          }
        }
        if (live && (!kE4m3 || h < p.Hq)) {
          uint4* dst;
          if (h < p.Hq) {
            dst = p.q + (static_cast<long long>(t) * p.Hq + h) * 16;
          } else {
            const int g = h - p.Hq - (is_v ? p.Hkv : 0);
            dst = reinterpret_cast<uint4*>((is_v ? p.pool.v : p.pool.k) + (((page_row + g) << p.page_shift) + off) * 256);
          }
          dst[e] = is_v ? x[i][0] : pack_bf16x8(a);
          dst[8 + e] = is_v ? x[i][1] : pack_bf16x8(b);
        }
      }
      if (kWhole) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          x[i][0] = y[i][0];
          x[i][1] = y[i][1];
        }
      }
    }
    w = next;
  }
}

// ---------------------------------------------------------------- dense <-> pages
// 32 bytes of one lane, a whole sector, where the address allows (whole: 32-byte aligned)
__device__ __forceinline__ void load32(const uint4* src, uint4& a, uint4& b, bool whole) {
  if (whole) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(src));
  } else {
    a = src[0];
    b = src[1];
  }
}
__device__ __forceinline__ void store32(uint4* dst, const uint4& a, const uint4& b, bool whole) {
  if (whole) {
    st_global_v8(dst, a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w);
  } else {
    dst[0] = a;
    dst[1] = b;
  }
}

struct PagedCopyParams {
  uint4* dense[2];  // k, v: bf16 [B, Hkv, rows, 128]
  PagedPool pool;
  const int4* entries;   // per table entry in use: page, sequence, first token, tokens
  const int* n_entries;  // entries of the batch as it is set now
  int rows, Hkv, page_shift;
};

// A warp takes 16 rows of one (entry, head, k or v): a page is contiguous per
// head, and so is the dense cache, so both sides are straight runs of 16 rows;
// all of a lane's loads are issued before the first is used. Eight lanes share
// a row, 16 values each (32 bytes of bf16, 16 of e4m3), four rows at a time.
// kStore: dense -> pages; otherwise pages -> dense. Bound by bytes: 56 prompts of
// 300 to 500 tokens into e4m3 24 us (5.7 TB/s), into bf16 28.6 (6.3), three e4m3
// sequences of about 4450 back 14.4 us (5.7, part of it from L2).
template <bool kE4m3, bool kStore>
__global__ void __launch_bounds__(256) paged_copy_kernel(const __grid_constant__ PagedCopyParams p) {
  grid_dep_launch();
  const int lane = lane_id(), sub = lane >> 3, e = lane & 7;
  const int runs = 1 << (p.page_shift - 4);
  const long long items = static_cast<long long>(*p.n_entries) * p.Hkv * 2 * runs;
  bool waited = false;  // the batch's tables are written by copies, never by a kernel: read before the wait
  for (long long w = blockIdx.x * 8ll + warp_id(); w < items; w += gridDim.x * 8ll) {
    const int run = static_cast<int>(w & (runs - 1));
    long long r = w >> (p.page_shift - 4);
    const int kv = static_cast<int>(r & 1);
    r >>= 1;
    const int head = static_cast<int>(r % p.Hkv);
    const int4 entry = p.entries[r / p.Hkv];
    const int seq = entry.y, j0 = entry.z + run * 16;
    const int live = min(entry.w, p.rows - entry.z) - run * 16;  // rows of this run that the sequence (and the dense cache) has
    if (!waited) {
      grid_dep_wait();
      waited = true;
    }
    if (live <= 0) continue;
    const long long prow = ((static_cast<long long>(entry.x) * p.Hkv + head) << p.page_shift) + run * 16;
    const long long drow = (static_cast<long long>(seq) * p.Hkv + head) * p.rows + j0;
    uint4* dense = p.dense[kv] + drow * 16;
    const bool whole = (reinterpret_cast<uintptr_t>(dense) & 31u) == 0u;
    uint8_t* page = (kv ? p.pool.v : p.pool.k) + prow * (kE4m3 ? 128 : 256);
    uint8_t* scale = kE4m3 ? (kv ? p.pool.vs : p.pool.ks) + prow : nullptr;
    if (!kE4m3) {
      uint4* pg = reinterpret_cast<uint4*>(page);
      const uint4* src = kStore ? dense : pg;
      uint4* dst = kStore ? pg : dense;
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (2 * i + (lane >> 4) < live) x[i] = src[i * 32 + lane];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (2 * i + (lane >> 4) < live) dst[i * 32 + lane] = x[i];
    } else if (kStore) {
      uint4 x[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + sub;
        x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        if (row < live) load32(dense + row * 16 + 2 * e, x[i][0], x[i][1], whole);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + sub;
        float a[8], b[8];
        unpack_bf16x8(x[i][0], a);
        unpack_bf16x8(x[i][1], b);
        float m = fmax3_nan(amax8(a), amax8(b), 0.f);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = fmax3_nan(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
        const uint32_t sc = e8m0_of_amax(m);
        const uint2 lo = quant8(a, sc), hi = quant8(b, sc);
        if (row < live) {
          reinterpret_cast<uint4*>(page + row * 128)[e] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          if (e == 0) scale[row] = static_cast<uint8_t>(sc);
        }
      }
    } else {
      uint4 x[4];
      uint32_t sc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + sub;
        if (row < live) {
          x[i] = reinterpret_cast<const uint4*>(page + row * 128)[e];
          sc[i] = scale[row];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + sub;
        if (row < live) {
          const float s = e8m0_value(sc[i]);
          store32(dense + row * 16 + 2 * e, dequant8(make_uint2(x[i].x, x[i].y), s), dequant8(make_uint2(x[i].z, x[i].w), s), whole);
        }
      }
    }
  }
  if (!waited) grid_dep_wait();
}

// ---------------------------------------------------------------- attention, few rows
// A unit is a tile of query rows of one (sequence, KV head) and a range of its
// keys. Query rows are (token, head of the group) pairs, head fastest, so the
// tile reads the KV head's keys once for the whole group. The record holds all
// that a CTA has to know of the sequence, so that it is one load away.
struct __align__(16) PagedUnit {
  int seq, head, row0, key0, key1;
  int slot0;    // first partial slot of the tile (nsplit > 1)
  int split;    // this range's number | nsplit << 16
  int counter;  // arrival counter of the tile
  int q0;       // first token of the chunk in the packed tensors
  int rows;     // query rows of the chunk
  int past;     // position of its first token
  int vis;      // keys that all its queries see
  int page0;    // first entry of the sequence in the page list
  int pad[3];
};

// a record, read anew (not kept in registers from an earlier read)
__device__ __forceinline__ PagedUnit read_unit(const PagedUnit* u) {
  PagedUnit r;
  int* w = reinterpret_cast<int*>(&r);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3]) : "l"(reinterpret_cast<const int4*>(u) + i));
  return r;
}

struct PagedAttnParams {
  const uint4* q;  // bf16 [T, Hq, 128]
  uint4* o;        // bf16 [T, Hq, 128]
  float* lse;      // [T, Hq] or null
  PagedPool pool;
  const int* pages;
  const PagedUnit* units;
  const int* cta_unit0;  // units of CTA i: [cta_unit0[i], cta_unit0[i + 1])
  int* counters;
  float* part;  // slots: [rows][128] f32 sums, then [rows] (m, l)
  int Hq, Hkv, group, page_shift;
  float scale_log2;  // log2(e) / sqrt(128)
  int* status;
};

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

// natural-log sum of exponentials from the base-2 running max and sum
__device__ __forceinline__ float lse_of(float m2, float l) { return (m2 + log2f(l)) * 0.69314718055994531f; }

template <bool kBf16>
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if (kBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Eight-row matrices of 16-byte rows in the operand layout of mma.sync, four at
// a time; lane i gives the address of row i % 8 of matrix i / 8.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

constexpr int kSmallRows = 8;  // query rows of a unit
constexpr int kSmallSlot = kSmallRows * 128 + kSmallRows * 2;  // floats of a partial

struct PagedSmallParams {
  // 2D rows of the pool; bf16: box {64, rows}, e4m3: bytes, box {128, rows}; 128-byte swizzle; rows = min(page, stage)
  CUtensorMap k_map, v_map;
  PagedAttnParams a;
};

// A warp takes 16 keys of a stage; two CTAs an SM, three stages of 32 KB of keys
// and values each: 192 KB in flight an SM.
template <bool kE4m3>
struct SmallShape {
  static constexpr int kWarps = kE4m3 ? 8 : 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kKeys = 16 * kWarps;
  static constexpr int kStages = 3;
  static constexpr uint32_t kHalf = 16384;  // keys, then values
  static constexpr uint32_t kLine = kKeys * 128;  // bf16: dims 0-63 of all rows, then dims 64-127
  static constexpr uint32_t kScale = kStages * 2 * kHalf;  // e4m3: [stage][keys, values][128] bytes
  static constexpr uint32_t kBytes = kScale + (kE4m3 ? kStages * 256 : 0) + 1024;
};

// Values that only some of the tile's rows see: an infinity or NaN times a zero
// weight would reach the rows that do not see it, so it is taken out (set to
// zero) and its key remembered per dim; rows whose limit is past that key get NaN
// at the end. Values behind the last key are whatever the page holds there, and
// become zero.
struct Unseen {
  int live;   // keys of the 16 that the unit uses
  int key0;   // position of the first
  bool some;  // the rows differ in what they see
  int* poison;

  // a bf16 pair: the values of keys k and k + 1 (of the 16) in dim d
  __device__ __forceinline__ uint32_t bf16_pair(uint32_t w, int k, int d) const {
    if (k >= live) return 0u;
    if (k + 1 >= live) w &= 0xffffu;
    if (some) {
      if ((w & 0x7f80u) == 0x7f80u) {
        atomicMin(poison + d, key0 + k);
        w &= 0xffff0000u;
      }
      if ((w & 0x7f800000u) == 0x7f800000u) {
        atomicMin(poison + d, key0 + k + 1);
        w &= 0xffffu;
      }
    }
    return w;
  }
  // four e4m3: key k, dims d..d + 3
  __device__ __forceinline__ uint32_t e4m3_quad(uint32_t w, int k, int d) const {
    if (k >= live) return 0u;
    if (some) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (((w >> (8 * i)) & 0x7fu) == 0x7fu) {
          atomicMin(poison + d + i, key0 + k);
          w &= ~(0xffu << (8 * i));
        }
    }
    return w;
  }
  // a value scale: key k; `part` of 4 of the dims
  __device__ __forceinline__ uint32_t scale(uint32_t b, int k, int part) const {
    if (k >= live) return 0u;
    if (some && b == 255u) {
#pragma unroll 1
      for (int d = 0; d < 32; ++d) atomicMin(poison + 32 * part + d, key0 + k);
      return 0u;
    }
    return b;
  }
};

// Attention of up to 8 query rows per unit over a range of keys; bound by the
// bytes of the pages. Each warp takes 16 keys of every stage and keeps its own
// running max, sum and O^T; the warps' results are merged through shared memory
// (over the unit's last stage, while the next unit's first stages are on their
// way), the ranges' results by whichever CTA arrives last, in the order of the
// ranges. Warp 0 also fetches the pages by TMA, two stages ahead (a warp of its
// own for that costs the others registers, and they spill).
// Tensor-core shapes: S^T (16 keys x 8 rows) = K Q^T and O^T (128 dims x 8
// rows) += V^T P^T, so the keys and values are the 16-row operand and no row is
// wasted on padding to 16 query rows; P^T gets into operand layout by
// movmatrix. bf16 pages: operands by ldmatrix; P is split into two bf16 (hi +
// lo), whose products sum in f32, so that the weights are not rounded to 8 bits.
// e4m3 pages: keys and values become f16 exactly (mma.sync on e4m3 is no way
// out: on sm_100 it runs as conversions and f16 products); the dims that each
// register pair stands for are permuted so that a lane reads whole 16-byte
// pieces, Q alike, and the rows of O^T are consecutive dims of a lane. The
// scales are applied in f32, to the scores and to the weights: what meets the
// values in f16 is 2^(score - max + value exponent) relative to a running max of
// its own, per query row and over the keys that the row sees. So a key loses
// weight only against products of weight and value that count in the same row:
// below 2^-21 of the largest one (weights go up to 2^15) it is rounded to a
// multiple of 2^-31 of it. Queries are scaled by a power of two into f16.
// The batch's tables are written by copies, never by a kernel, so they are read
// before the grid this one depends on has completed.
// Measured, one B200: 64 single tokens over ragged e4m3 caches of 0.4 to 8.6
// thousand keys (554 MB) 112 us, 4.9 TB/s (109 with one reference for all rows); the
// same in bf16 168 us, 6.5 TB/s. Under ncu the 8-bit kernel takes 115 us, its loads
// without the arithmetic 96; a plain read of as many bytes takes 78 us. A single
// token over 4496 bf16 keys 9.7 us, of which the keys' bytes are 2.8: the rest is
// launch, dependent loads, and the merge of 18 ranges.
template <bool kE4m3>
__global__ void __launch_bounds__(SmallShape<kE4m3>::kThreads, 2)
paged_attn_small_kernel(const __grid_constant__ PagedSmallParams sp) {
  using SM = SmallShape<kE4m3>;
  const PagedAttnParams& p = sp.a;
  extern __shared__ uint8_t smem_raw[];
  __shared__ float2 s_ml[SM::kWarps][kSmallRows];
  __shared__ int s_poison[128];
  __shared__ int s_last;
  __shared__ uint32_t s_abort;
  __shared__ uint64_t s_full[SM::kStages], s_empty[SM::kStages];
  grid_dep_launch();
  const int warp = warp_id(), lane = lane_id(), g = lane >> 2, c = lane & 3;
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int u_begin = p.cta_unit0[blockIdx.x], u_end = p.cta_unit0[blockIdx.x + 1];
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < SM::kStages; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], SM::kWarps);
    }
    s_abort = 0u;
    fence_mbar_init();
  }
  __syncthreads();
  const WaitGuard wg{&s_abort, p.status};
  // warp 0: the stage to be fetched next is that of unit f_unit at f_key; lane i takes box i
  const int ps = min(1 << p.page_shift, SM::kKeys), page_mask = (1 << p.page_shift) - 1;
  int f_unit = u_begin, f_key = -1, f_stage = 0;
  uint32_t f_phase = 1u;
  auto fetch = [&] {
    if (warp != 0 || f_unit >= u_end) return;
    const PagedUnit* un = p.units + f_unit;
    if (f_key < 0) f_key = un->key0;
    const int key1 = un->key1;
    const int boxes = (min(SM::kKeys, key1 - f_key) + ps - 1) / ps;
    const int k = f_key + lane * ps;
    int row = 0;
    if (lane < boxes) row = ((p.pages[un->page0 + (k >> p.page_shift)] * p.Hkv + un->head) << p.page_shift) + (k & page_mask);
    mbar_wait(&s_empty[f_stage], f_phase, wg);
    if (lane == 0) mbar_expect_tx(&s_full[f_stage], static_cast<uint32_t>(boxes * ps) * (kE4m3 ? 258u : 512u));
    __syncwarp();
    if (lane < boxes) {
      uint8_t* dst = stages + f_stage * 2 * SM::kHalf + lane * ps * 128;
      tma_load_2d(dst, &sp.k_map, &s_full[f_stage], 0, row);
      tma_load_2d(dst + SM::kHalf, &sp.v_map, &s_full[f_stage], 0, row);
      if constexpr (kE4m3) {
        uint8_t* sc = stages + SM::kScale + f_stage * 256 + lane * ps;
        bulk_load(sc, p.pool.ks + row, ps, &s_full[f_stage]);
        bulk_load(sc + 128, p.pool.vs + row, ps, &s_full[f_stage]);
      } else {
        tma_load_2d(dst + SM::kLine, &sp.k_map, &s_full[f_stage], 64, row);
        tma_load_2d(dst + SM::kHalf + SM::kLine, &sp.v_map, &s_full[f_stage], 64, row);
      }
    }
    f_key += SM::kKeys;
    if (f_key >= key1) {
      ++f_unit;
      f_key = -1;
    }
    if (++f_stage == SM::kStages) {
      f_stage = 0;
      f_phase ^= 1u;
    }
  };
  int stage = 0;
  uint32_t phase = 0;
  auto advance = [&] {
    if (++stage == SM::kStages) {
      stage = 0;
      phase ^= 1u;
    }
  };

  const int key_w = 16 * warp;  // this warp's keys of a stage
  grid_dep_wait();
  // every stage but one is fetched ahead; the one more follows where a stage has been read
  for (int i = 0; i + 1 < SM::kStages; ++i) fetch();
  for (int u = u_begin; u < u_end; ++u) {
    const PagedUnit un = p.units[u];
    const int rows = min(kSmallRows, un.rows - un.row0);
    auto limit_of = [&](int r) { return max(un.vis, un.past + (un.row0 + min(r, rows - 1)) / p.group + 1); };
    const int lim_min = limit_of(0), lim_max = limit_of(rows - 1);

    // query row g as the B operand. bf16: words 2s, 2s + 1 hold dims 16s + 2c, + 1 and 16s + 8 + 2c, + 1; e4m3 (as f16):
    // dims 32c + 2i, + 1 in word i
    uint32_t q[16];
    float qf[2] = {p.scale_log2, p.scale_log2};  // score factor of rows 2c, 2c + 1
    {
      const int rr = un.row0 + g;
      const bool live = g < rows;
      const uint4* src = p.q + (static_cast<long long>(un.q0 + rr / p.group) * p.Hq + un.head * p.group + rr % p.group) * 16;
      if constexpr (!kE4m3) {
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = live ? __ldg(reinterpret_cast<const uint32_t*>(src) + 4 * i + c) : 0u;
      } else {
        float f[4][8];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = live ? __ldg(src + 4 * c + i) : make_uint4(0, 0, 0, 0);
          unpack_bf16x8(w, f[i]);
          m = fmax3_nan(m, amax8(f[i]), 0.f);
        }
        m = fmax3_nan(m, __shfl_xor_sync(0xffffffffu, m, 1), 0.f);
        m = fmax3_nan(m, __shfl_xor_sync(0xffffffffu, m, 2), 0.f);
        const uint32_t ex = query_exponent(m);
        const float down = __uint_as_float((254u - ex) << 23), up = __uint_as_float(ex << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) q[i] = pack_half2(f[i >> 2][2 * (i & 3)] * down, f[i >> 2][2 * (i & 3) + 1] * down);
        qf[0] *= __shfl_sync(0xffffffffu, up, 8 * c);      // row 2c is lane group g = 2c
        qf[1] *= __shfl_sync(0xffffffffu, up, 8 * c + 4);
      }
    }
    if (lim_max != lim_min) {
      for (int i = threadIdx.x; i < 128; i += SM::kWarps * 32) s_poison[i] = INT_MAX;
      named_bar_sync(1, SM::kWarps * 32);
    }

    float o[8][4];
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[t][i] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    // e4m3: O^T counts in units of 2^(r_run - kUp), r_run the running max of score - m_run + value exponent
    float r_run[2] = {-INFINITY, -INFINITY};
    constexpr float kUp = 7.f;

    // the 16 keys from `key` on; kWhole: every row sees all of them (the other case, code of its own, is rare)
    auto take = [&](int key, auto whole_c) {
      constexpr bool whole = decltype(whole_c)::value;
        const uint8_t* kt = stages + stage * 2 * SM::kHalf;
        const uint32_t k_addr = smem_u32(kt) + key_w * 128;
        float s[2][4] = {};  // two sums: shorter chains
        float x[4];          // base-2 scores; x[0], x[1]: key g, rows 2c, 2c + 1; x[2], x[3]: key g + 8
        [[maybe_unused]] uint32_t vs[2] = {0u, 0u};
        if constexpr (!kE4m3) {
          // k-step i: rows 0-7 | 8-15 of pieces 2i, then of 2i + 1
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t a[4];
            ldmatrix4(a, k_addr + (i >> 2) * SM::kLine + (lane & 15) * 128 + (((2 * (i & 3) + (lane >> 4)) ^ (lane & 7)) << 4));
            mma_16816<true>(s[i & 1], a[0], a[1], a[2], a[3], q[2 * i], q[2 * i + 1]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = (s[0][i] + s[1][i]) * qf[i & 1];
        } else {
          const uint8_t* sc = stages + SM::kScale + stage * 256 + key_w + g;
          const float kf[2] = {e8m0_value(sc[0]), e8m0_value(sc[8])};
          vs[0] = sc[128];
          vs[1] = sc[136];
          const uint8_t* kr = kt + (key_w + g) * 128;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 ka = *reinterpret_cast<const uint4*>(kr + (((2 * c + i) ^ g) << 4));
            const uint4 kb = *reinterpret_cast<const uint4*>(kr + 1024 + (((2 * c + i) ^ g) << 4));
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t a0, a1, b0, b1;
              e4m3x4_f16x4(word(ka, h), a0, a1);
              e4m3x4_f16x4(word(kb, h), b0, b1);
              mma_16816<false>(s[h & 1], a0, b0, a1, b1, q[8 * i + 2 * h], q[8 * i + 2 * h + 1]);
            }
          }
          const float top = fmaxf(qf[0], qf[1]) * fmaxf(kf[0], kf[1]);
          if (top <= FLT_MAX) {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = (s[0][i] + s[1][i]) * (qf[i & 1] * kf[i >> 1]);
          } else {  // their product may be infinite though the score is not
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = (s[0][i] + s[1][i]) * qf[i & 1] * kf[i >> 1];
          }
        }
        const Unseen unseen{min(lim_max, un.key1) - key, key, lim_max != lim_min, s_poison};
        if (!whole) {
          const int lim0 = min(limit_of(2 * c), un.key1), lim1 = min(limit_of(2 * c + 1), un.key1);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key + g + 8 * (i >> 1) >= ((i & 1) ? lim1 : lim0)) x[i] = -INFINITY;
          if constexpr (kE4m3) {
            vs[0] = unseen.scale(vs[0], g, c);
            vs[1] = unseen.scale(vs[1], g + 8, c);
          }
        }
        // the running max moves only when a score passes it by 2^8; r_run alike
        const float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
        bool grow = mx0 > m_run[0] + kLazyRescaleLog2 || mx1 > m_run[1] + kLazyRescaleLog2;
        float d[4];  // base-2 logs of the weights
        [[maybe_unused]] float y[4], vx[2];  // e4m3: with the values' exponents, and those
        auto logs = [&] {
          const float m0 = finite_or_zero(m_run[0]), m1 = finite_or_zero(m_run[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            d[i] = x[i] - ((i & 1) ? m1 : m0);
            if constexpr (kE4m3) y[i] = d[i] + vx[i >> 1];
          }
        };
        if constexpr (kE4m3) {
#pragma unroll
          for (int r = 0; r < 2; ++r) vx[r] = vs[r] == 255u ? NAN : static_cast<float>(static_cast<int>(vs[r]) - 127);
        }
        logs();
        if constexpr (kE4m3)
          grow = grow || fmaxf(y[0], y[2]) > r_run[0] + kLazyRescaleLog2 || fmaxf(y[1], y[3]) > r_run[1] + kLazyRescaleLog2;
        if (__any_sync(0xffffffffu, grow)) {
          float a[2] = {mx0, mx1}, f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) a[i] = fmaxf(a[i], __shfl_xor_sync(0xffffffffu, a[i], o));
            a[i] = fmaxf(a[i], m_run[i]);
            f[i] = ex2_approx(m_run[i] - finite_or_zero(a[i]));
            if constexpr (kE4m3) r_run[i] = m_run[i] == -INFINITY ? -INFINITY : r_run[i] - (a[i] - m_run[i]);
            m_run[i] = a[i];
            l_run[i] *= f[i];
          }
          logs();
          if constexpr (kE4m3) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float b = fmaxf(y[i], y[2 + i]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
              b = fmaxf(b, r_run[i]);
              f[i] = ex2_approx(r_run[i] - finite_or_zero(b));
              r_run[i] = b;
            }
          }
#pragma unroll
          for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][i] *= f[i & 1];
        }
        float pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pr[i] = ex2_approx(d[i]);
        l_run[0] += pr[0] + pr[2];
        l_run[1] += pr[1] + pr[3];
        if constexpr (!kE4m3) {
          const uint32_t h0 = pack_bf162(pr[0], pr[1]), h1 = pack_bf162(pr[2], pr[3]);
          const uint32_t l0 = pack_bf162(pr[0] - __uint_as_float(h0 << 16), pr[1] - __uint_as_float(h0 & 0xffff0000u));
          const uint32_t l1 = pack_bf162(pr[2] - __uint_as_float(h1 << 16), pr[3] - __uint_as_float(h1 & 0xffff0000u));
          const uint32_t b0 = transpose_8x8(h0), b1 = transpose_8x8(h1);
          const uint32_t d0 = transpose_8x8(l0), d1 = transpose_8x8(l1);
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            // keys 0-7 | 8-15 of dims 16t.. (pieces 2t, 2t + 1), transposed: dims 16t + g, + 8; keys 2c, + 1, then + 8
            uint32_t a[4];
            ldmatrix4_trans(a, k_addr + SM::kHalf + (t >> 2) * SM::kLine + ((lane & 7) + ((lane >> 4) << 3)) * 128 +
                                   (((2 * (t & 3) + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
            if (!whole) {
#pragma unroll
              for (int i = 0; i < 4; ++i) a[i] = unseen.bf16_pair(a[i], 2 * c + 8 * (i >> 1), 16 * t + g + 8 * (i & 1));
            }
            mma_16816<true>(o[t], a[0], a[1], a[2], a[3], b0, b1);
            mma_16816<true>(o[t], a[0], a[1], a[2], a[3], d0, d1);
          }
        } else {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = ex2_approx(y[i] - (finite_or_zero(r_run[i & 1]) - kUp));
          const uint32_t b0 = transpose_8x8(pack_half2(w[0], w[1])), b1 = transpose_8x8(pack_half2(w[2], w[3]));
          // keys 2c, 2c + 1, 2c + 8, 2c + 9, dims 16g..16g + 15: eight lanes hit all banks once
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 2 * c + (i & 1) + 8 * (i >> 1);
            v[i] = *reinterpret_cast<const uint4*>(kt + SM::kHalf + (key_w + r) * 128 + ((g ^ (r & 7)) << 4));
            if (!whole)
              v[i] = make_uint4(unseen.e4m3_quad(v[i].x, r, 16 * g), unseen.e4m3_quad(v[i].y, r, 16 * g + 4),
                                unseen.e4m3_quad(v[i].z, r, 16 * g + 8), unseen.e4m3_quad(v[i].w, r, 16 * g + 12));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              // dims 16g + 4i + 2d, + 1 (h = 0) and 8 behind (h = 1): bytes (key a, key b) per dim
              uint32_t e[2][2][2];  // [h][key pair][dim]
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int kp = 0; kp < 2; ++kp)
                  e4m3x4_f16x4(__byte_perm(word(v[2 * kp], 2 * h + i), word(v[2 * kp + 1], 2 * h + i), d ? 0x7362 : 0x5140),
                               e[h][kp][0], e[h][kp][1]);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                mma_16816<false>(o[4 * i + 2 * d + k], e[0][0][k], e[1][0][k], e[0][1][k], e[1][1][k], b0, b1);
            }
        }
    };
    for (int key_s = un.key0;; key_s += SM::kKeys) {
      const int key = key_s + key_w;
      const bool more = key_s + SM::kKeys < un.key1;
      if (key_s > un.key0) fetch();  // over the stage before this one
      mbar_wait(&s_full[stage], phase, wg);
      if (key + 16 <= min(lim_min, un.key1))
        take(key, std::true_type{});
      else if (key < un.key1)
        take(key, std::false_type{});
      if (!more) break;  // the unit's last stage stays this CTA's for the merge
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_empty[stage]);
      advance();
    }

    // Merge of the warps. A warp's sums, f32 [8 rows][128], lie over its own rows of the last stage: rows 0-3 over its
    // keys (bf16: line 0), rows 4-7 over its values (line 1 of the keys); dims are permuted by the row so that the
    // warp's stores hit all banks.
    auto sum_at = [&](int w, int r, int d) {
      return reinterpret_cast<float*>(stages + stage * 2 * SM::kHalf + (r >> 2) * (kE4m3 ? SM::kHalf : SM::kLine) + w * 2048) +
             (r & 3) * 128 + (d ^ ((r >> 1) << 3));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], d);
    }
    // back to units of 1, in two steps (2^135 is no f32)
    float half[2] = {1.f, 1.f};
    if constexpr (kE4m3) {
#pragma unroll
      for (int i = 0; i < 2; ++i) half[i] = ex2_approx(0.5f * (finite_or_zero(r_run[i]) - kUp));
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * c + i;
      if (g == 0) s_ml[warp][r] = make_float2(m_run[i], l_run[i]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (kE4m3) {
#pragma unroll
          for (int t = 0; t < 8; t += 4)
            *reinterpret_cast<float4*>(sum_at(warp, r, 16 * g + 8 * j + t)) =
                make_float4(o[t][2 * j + i] * half[i] * half[i], o[t + 1][2 * j + i] * half[i] * half[i],
                            o[t + 2][2 * j + i] * half[i] * half[i], o[t + 3][2 * j + i] * half[i] * half[i]);
        } else {
#pragma unroll
          for (int t = 0; t < 8; ++t) *sum_at(warp, r, 16 * t + 8 * j + g) = o[t][2 * j + i];
        }
      }
    }
    named_bar_sync(1, SM::kWarps * 32);
    const int nsplit = un.split >> 16, split = un.split & 0xffff;
    auto write_row = [&](int r, float m, float l, const float4& v) {
      const int rr = un.row0 + r;
      const long long out_row = static_cast<long long>(un.q0 + rr / p.group) * p.Hq + un.head * p.group + rr % p.group;
      const float inv = 1.0f / l;
      reinterpret_cast<uint2*>(p.o + out_row * 16)[lane] = make_uint2(pack_bf162(v.x * inv, v.y * inv), pack_bf162(v.z * inv, v.w * inv));
      if (p.lse && lane == 0) p.lse[out_row] = lse_of(m, l);
    };
    auto add = [](float4& acc, float w, const float4& v) {
      acc.x = fmaf(v.x, w, acc.x);
      acc.y = fmaf(v.y, w, acc.y);
      acc.z = fmaf(v.z, w, acc.z);
      acc.w = fmaf(v.w, w, acc.w);
    };
#pragma unroll 1
    for (int r = warp; r < rows; r += SM::kWarps) {  // a warp a row
      float m = -INFINITY, l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < SM::kWarps; ++i) m = fmaxf(m, s_ml[i][r].x);
      const float m0 = finite_or_zero(m);
#pragma unroll
      for (int i = 0; i < SM::kWarps; ++i) {
        const float2 ml = s_ml[i][r];
        const float w = ex2_approx(ml.x - m0);
        l = fmaf(ml.y, w, l);
        add(acc, w, *reinterpret_cast<const float4*>(sum_at(i, r, 4 * lane)));
      }
      if (lim_max != lim_min) {
        const int lr = limit_of(r);
        if (s_poison[4 * lane] < lr) acc.x = NAN;
        if (s_poison[4 * lane + 1] < lr) acc.y = NAN;
        if (s_poison[4 * lane + 2] < lr) acc.z = NAN;
        if (s_poison[4 * lane + 3] < lr) acc.w = NAN;
      }
      if (nsplit == 1) {
        write_row(r, m, l, acc);
      } else {
        float* slot = p.part + static_cast<long long>(un.slot0 + split) * kSmallSlot;
        reinterpret_cast<float4*>(slot + r * 128)[lane] = acc;
        if (lane == 0) reinterpret_cast<float2*>(slot + kSmallRows * 128)[r] = make_float2(m, l);
      }
    }
    fence_proxy_async_smem();  // the stage goes back to the TMA
    named_bar_sync(1, SM::kWarps * 32);
    if (lane == 0) mbar_arrive(&s_empty[stage]);
    advance();
    __syncwarp();
    fetch();
    if (nsplit > 1) {
      if (threadIdx.x == 0) {
        // one fence for the CTA's writes, which the barrier put before it; the counter wraps to 0 with the last
        // arrival: ready for the next call
        __threadfence();
        s_last = atomicInc(reinterpret_cast<unsigned*>(p.counters) + un.counter, nsplit - 1) == nsplit - 1;
        __threadfence();
      }
      named_bar_sync(1, SM::kWarps * 32);
      const float* slots = p.part + static_cast<long long>(un.slot0) * kSmallSlot;
      const bool last = s_last;
      named_bar_sync(1, SM::kWarps * 32);  // read by all before the next unit may write it
#pragma unroll 1
      for (int r = last ? warp : rows; r < rows; r += SM::kWarps) {
        // lane i holds the max and sum of range 32 b + i; the sums of eight ranges are in flight at a time
        auto ml_of = [&](int i) {
          return i < nsplit ? __ldcg(reinterpret_cast<const float2*>(slots + static_cast<long long>(i) * kSmallSlot + kSmallRows * 128) + r)
                            : make_float2(-INFINITY, 0.f);
        };
        const float2 first = ml_of(lane);
        float m = first.x, l = 0.f;
        for (int b = 32; b < nsplit; b += 32) m = fmaxf(m, ml_of(b + lane).x);
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float m0 = finite_or_zero(m);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b = 0; b < nsplit; b += 32) {
          const float2 ml = b == 0 ? first : ml_of(b + lane);
          const float wl = ex2_approx(ml.x - m0);
          float part_l = b + lane < nsplit ? ml.y * wl : 0.f;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) part_l += __shfl_xor_sync(0xffffffffu, part_l, d);
          l += part_l;
          const int n = min(32, nsplit - b);
          for (int i = 0; i < n; i += 8) {
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              v[k] = __ldcg(reinterpret_cast<const float4*>(slots + static_cast<long long>(b + min(i + k, n - 1)) * kSmallSlot + r * 128) + lane);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float w = __shfl_sync(0xffffffffu, wl, i + k);
              if (i + k < n) add(acc, w, v[k]);
            }
          }
        }
        write_row(r, m, l, acc);
      }
    }
  }
}

}  // namespace mot
