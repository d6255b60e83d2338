// paged_tile.cuh -- attention of chunks over the pages (include/mot_paged.h,
// mot_paged_attend) on the 5th-generation tensor cores.
//
// A unit is 256 query rows of one (sequence, KV head) -- (token, head of the
// group) pairs, head fastest, as two 128-row tiles -- and a range of 128-key
// tiles. Per key tile S_t = Q_t K^T into TMEM, softmax in registers, P_t (16-bit
// pairs) over S_t's own columns, O_t += P_t V with P_t as the TMEM operand; the
// tensor core works on one query tile while the other's softmax runs. One CTA
// per SM runs its list of units back to back.
//
// Warps 0-3 and 4-7: softmax of tile 0 and 1, one thread per query row with its
// 128 scores in registers, so that the running max and sum need no exchange.
// Warp 12: MMA issue; warp 13: the query tiles, loaded while the unit before
// still runs; warp 14: the pages. bf16 pages: one TMA box per page and 64 dims
// (128-byte swizzle, which is why page_size is a multiple of the 8-row swizzle
// atom) straight into the operand tiles. e4m3 pages: boxes of raw rows and their
// scales into a staging tile each for keys and values, from which warps 8-11
// make f16 operand tiles: e4m3 -> f16 is one exact instruction per pair, and the
// row's scale relative to the tile's largest an exact factor, a power of two. The
// tile's largest scale goes into the scores (keys), and into the weights
// relative to the largest so far (values), as one factor per tile; queries are
// made f16 in place, each row scaled by a power of two that its thread puts back.
// Where a unit's scales lie too far apart for that (`kKeySpan`, `kValueSpan`; warps
// 8-11 read those of the first unit, warp 15 the others a unit or two ahead), the
// operand tiles are bf16 instead, which holds payload times scale, and the queries,
// as they are.
// Scores of unseen keys become -infinity. Their values meet weights of zero, so in
// tiles that not all rows of a unit see warps 8-11 take out what is not finite,
// and rows that do see it get NaN in those dims at the end (bf16 pages go through
// these warps only there and at the last key).
// The registers are split by setmaxnreg: 2 x 192 + 2 x 64 (e4m3: 176 and 80) of
// the 4 x 128 a thread that the block starts with.
//
// Probabilities are of the values' type, since they meet them in one MMA: bf16
// ones lose about what the bf16 output itself does (half a step, averaged over
// the keys), f16 ones an eighth of that; the row sum is taken in f32 from the
// unrounded ones. The running max is raised, and O_t rescaled through TMEM, only
// when a row's max grows by more than 2^8.
//
// What bounds it, measured on one B200: per key tile and pair of query tiles the
// MMAs take 2048 clocks (64 each, on one SM as on all), while by time stamps in
// the kernel a query tile's chain S -> softmax -> P V -> next S takes about 3000:
// 950 waiting for S, 170 to read it, 200 for the max, 1500 for exponentials and P
// (1024 of the MUFU). Two query tiles overlap but do not hide it, and TMEM has no
// room for a third. 2 x 4096 image tokens over 4496 keys (603 GFLOP): 551 us back
// to back (1.09 PFLOP/s). Prompt chunks of 129 to 512 tokens, bf16: 75 us. A mixed
// e4m3 batch 248 us, 324 when every unit is wide; one chunk of 64 tokens over 64 e4m3
// keys 14 us, over 4500 39 us. Of these the care for wide units, large scores and
// values that are not finite costs up to 1% (image, chunks), 4%, 2.5 and 2.4 us; the scan
// of a unit's scales alone 1.2 us a call. Spills, -Xptxas -v: 8 bytes stored (bf16), 236
// (e4m3). Tried against the kernel of the time and slower: a quarter of the
// exponentials by polynomial (image 564 against 555 us, a mixed e4m3 batch 289 against
// 269), a second MMA warp (image 565 against 552), e4m3 conversion on eight warps with
// fewer registers for the softmax (the mixed batch 272 against 251).
#pragma once

#include "paged.cuh"

namespace mot {

constexpr int kTileRows = 256;  // query rows of a unit
constexpr int kTileKeys = 128;
// Floats of a partial: 32 groups of 4 dims, each [256 rows][4], so that the
// threads of a warp, a row each, write and read 512 bytes in a row; then the
// rows' (max, sum).
constexpr int kTileSlot = kTileRows * 128 + kTileRows * 2;

struct PagedTileParams {
  // 2D {128, n_pages * Hkv * page_size}; bf16: box {64, page_size}, 128-byte swizzle; e4m3: bytes, box {128, page_size}
  CUtensorMap k_map, v_map;
  CUtensorMap q_map;         // 3D {128, Hq, T}, box {64, group, 128 / group} (q_tma)
  int q_tma;                 // the group is a power of two
  PagedAttnParams a;
};

struct TileSmem {
  static constexpr uint32_t kTile = 32768;  // 128 rows x 128 bf16
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + 2 * kTile;
  static constexpr uint32_t kV = kK + 2 * kTile;
  static constexpr uint32_t kBar = kV + 2 * kTile;
  static constexpr uint32_t kPoison = kBar + 512;  // per dim: first key of the unit whose value is not finite
  static constexpr uint32_t kRaw = kPoison + 512;  // e4m3: [keys, values] 128 rows of 128 bytes, then 2 x 128 scales
  static constexpr uint32_t kRawTile = 16384;
  static constexpr uint32_t kScale = kRaw + 2 * kRawTile;
  static constexpr uint32_t kRef = kScale + 256;   // e4m3: largest scale bytes, keys [4 tiles] (| kWide), values [4 tiles]
  static constexpr uint32_t kQScale = kRef + 64;   // e4m3: [2 units][256 rows] 127 + exponent of a query row's factor
  static constexpr uint32_t bytes(bool e4m3) { return (e4m3 ? kQScale + 512 : kRaw) + 1024; }
};

constexpr int kTileThreads = 512;

template <int kRegs>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// One lane of a converged warp. The MMA warp runs its loop with all lanes and
// lets the elected one issue: under `if (lane == 0)` the compiler cannot keep
// descriptors in uniform registers, and each tcgen05.mma then took 110 clocks to
// issue, more than the 64 it takes to run.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
  return p != 0u;
}

// Byte offset of 16-byte piece `piece` (0..15) of row `row` in a 128 x 128 bf16
// tile: two boxes of 64 dims, 128 bytes a row, pieces permuted by row & 7.
__device__ __forceinline__ uint32_t tile_offset(int row, int piece) {
  return static_cast<uint32_t>((piece >> 3) * 16384 + row * 128 + (((piece & 7) ^ (row & 7)) << 4));
}

// An 8-bit unit is wide when its scales differ by more than f16 operands bear: a
// key scale by more than 2^kKeySpan (a row's factor relative to its tile's largest
// would no longer be exact), a value scale by more than 2^kValueSpan (weights
// relative to the unit's largest value scale would lose bits: what f16 takes from a
// weight is at most 2^-32 of the row's largest (weights go up to 2^15), times 448
// units of 2^kValueSpan of a row with a largest value of at least 224: 2^-24 of
// the largest value that a query sees, a key, whatever the size of those that it
// does not see). Wide units run on bf16 operands, which hold every row as it is.
// So do units with a key scale above 2^(kKeyTop - 127): below it the factor of a row's
// scores, at most 2^123 from the query's side, is an f32.
constexpr int kKeySpan = 14, kValueSpan = 7;
constexpr int kKeyTop = 131;
constexpr float kWeightUp = 7.f;  // weights of f16 units are 2^kWeightUp times as large
constexpr uint32_t kWide = 256u;

// Running max from which on it is not subtracted from the scores in one fused step: what the max lost when it was
// rounded, up to 2^-24 of it, would be left in every exponent. Such scores are rounded by themselves first.
constexpr float kFarScore = 1048576.f;

// largest and smallest scale byte of `rem` rows from `src` on (16 at most); 255 (NaN) counts as neither
struct ScaleSpan {
  uint32_t top = 0u, low = 0x00ff00ffu;  // pairs; top: plus 1, 0 = none
  __device__ __forceinline__ void take(const uint4& v, int rem) {
    const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = rem - 4 * i;
      const uint32_t w = n >= 4 ? w4[i] : n <= 0 ? 0xffffffffu : w4[i] | (0xffffffffu << (8 * n));
      const uint32_t a = w & 0x00ff00ffu, b = (w >> 8) & 0x00ff00ffu;
      top = __vmaxu2(top, __vmaxu2((a + 0x00010001u) & 0x00ff00ffu, (b + 0x00010001u) & 0x00ff00ffu));
      low = __vminu2(low, __vminu2(a, b));
    }
  }
  // over the warp: largest plus 1 (0: none), smallest
  __device__ __forceinline__ uint32_t largest() const { return __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16)); }
  __device__ __forceinline__ uint32_t smallest() const { return __reduce_min_sync(0xffffffffu, min(low & 0xffffu, low >> 16)); }
};

// whether a unit is wide, from the largest (plus 1, 0: none) and smallest scale bytes
__device__ __forceinline__ bool is_wide(uint32_t k_top, uint32_t k_low, uint32_t v_top, uint32_t v_low) {
  return static_cast<int>(k_top) - 1 > kKeyTop || static_cast<int>(k_top - 1u - k_low) > kKeySpan ||
         static_cast<int>(v_top - 1u - v_low) > kValueSpan;
}

// a unit's scales, pieces of 16 rows from the unit's `first` on, every `stride`-th
__device__ __forceinline__ void scan_scales(const PagedAttnParams& p, const PagedUnit& un, int first, int stride, ScaleSpan& keys,
                                            ScaleSpan& values) {
  const int ps16 = p.page_shift - 4;
  const int* pages = p.pages + un.page0;
  constexpr int kAhead = 4;  // pieces of a lane on their way
#pragma unroll 1
  for (int c0 = (un.key0 >> 4) + first; c0 * 16 < un.key1; c0 += stride * kAhead) {
    uint4 k[kAhead], v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int c = c0 + stride * i;
      if (c * 16 < un.key1) {
        const int row = ((pages[c >> ps16] * p.Hkv + un.head) << p.page_shift) + ((c & ((1 << ps16) - 1)) << 4);
        k[i] = *reinterpret_cast<const uint4*>(p.pool.ks + row);
        v[i] = *reinterpret_cast<const uint4*>(p.pool.vs + row);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int rem = un.key1 - (c0 + stride * i) * 16;
      if (rem > 0) {
        keys.take(k[i], rem);
        values.take(v[i], rem);
      }
    }
  }
}

// f16 pair of 2^(b - ref) (b at most kKeySpan below ref, or 255: NaN); b * 0x04000400 +
// near_base(ref) is the same where b is not 255.
__device__ __forceinline__ uint32_t near_base(uint32_t ref) { return 0x3c003c00u - ref * 0x04000400u; }
__device__ __forceinline__ uint32_t near_factor(uint32_t b, uint32_t ref) {
  return b == 255u ? 0x7e007e00u : b * 0x04000400u + near_base(ref);
}

// eight e4m3 times a factor (a pair of it) as f16
__device__ __forceinline__ uint4 e4m3x8_f16(uint2 w, uint32_t f) {
  const __half2 f2 = *reinterpret_cast<const __half2*>(&f);
  uint32_t r[4];
  e4m3x4_f16x4(w.x, r[0], r[1]);
  e4m3x4_f16x4(w.y, r[2], r[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&r[i]), f2);
    r[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// max of a row's 128 scores, in four chains; NaN comes out as NaN
__device__ __forceinline__ float scores_max(const uint32_t (&s)[4][32]) {
  float m[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) m[c] = __uint_as_float(s[c][0]);
#pragma unroll
  for (int i = 1; i < 31; i += 2)
#pragma unroll
    for (int c = 0; c < 4; ++c) m[c] = fmax3_nan(m[c], __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
  m[0] = fmax3_nan(m[0], __uint_as_float(s[0][31]), m[1]);
  m[2] = fmax3_nan(m[2], __uint_as_float(s[2][31]), m[3]);
  return fmax3_nan(m[0], m[2], fmax3_nan(__uint_as_float(s[1][31]), __uint_as_float(s[3][31]), -INFINITY));
}

// p = 2^(s scale - m) of 32 scores as 16 pairs (bf16 or f16) at taddr; adds them to sum.
template <bool kBf16>
__device__ __forceinline__ void scores_exp32(const uint32_t (&s)[32], uint32_t taddr, float scale, float neg_m,
                                             float (&sum)[4]) {
  uint32_t pk[16];
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float x0, x1, p0, p1;
    ffma2(x0, x1, __uint_as_float(s[i]), __uint_as_float(s[i + 1]), scale, scale, neg_m, neg_m);
    p0 = ex2_approx(x0);
    p1 = ex2_approx(x1);
    if ((i >> 1) & 1)
      fadd2(sum[2], sum[3], sum[2], sum[3], p0, p1);
    else
      fadd2(sum[0], sum[1], sum[0], sum[1], p0, p1);
    pk[i >> 1] = kBf16 ? pack_bf162(p0, p1) : pack_half2(p0, p1);
  }
  tmem_st16(taddr, pk);
}

// 32 dims of an output row times f, as bf16; whole 32-byte sectors where the
// output is so aligned
__device__ __forceinline__ void store_row32(uint4* dst, const uint32_t (&r)[32], float f) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_bf162(__uint_as_float(r[2 * i]) * f, __uint_as_float(r[2 * i + 1]) * f);
  if ((reinterpret_cast<uintptr_t>(dst) & 31u) == 0u) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      st_global_v8(dst + 2 * i, w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3], w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

// Keys that every row of a unit sees: those behind may meet a weight of zero.
__device__ __forceinline__ int seen_by_all(const PagedUnit& un, int group) {
  return max(un.vis, un.past + un.row0 / group + 1);
}

// The values of a ring tile that some rows of the unit do not see: zero times an
// infinity or NaN would reach those rows, so what is not finite becomes zero, and
// its key is remembered per dim; rows that see it get NaN at the end. A thread
// takes pieces piece0 and piece1 (eight dims each) of rows sub, sub + 16, ... below
// `live`, the first of which is key `key`. The code is kept small: it runs once or
// twice a unit, from a cold instruction cache (unrolled it took 4 us a tile).
template <bool kBf16>
__device__ __forceinline__ void clean_tile(uint8_t* tile, int key, int live, int sub, int piece0, int piece1, int* poison,
                                           volatile uint32_t* poisoned) {
  constexpr uint32_t kExp = kBf16 ? 0x7f807f80u : 0x7c007c00u, kOne = kBf16 ? 0x00800080u : 0x04000400u;
  auto all_ones = [](uint32_t w) { return ((w & kExp) + kOne) & 0x80008000u; };  // exponents, either half
  uint32_t some = 0u;
#pragma unroll 2
  for (int r = sub; r < live; r += 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(tile + tile_offset(r, piece0));
    const uint4 w = *reinterpret_cast<const uint4*>(tile + tile_offset(r, piece1));
    some |= all_ones(v.x) | all_ones(v.y) | all_ones(v.z) | all_ones(v.w) | all_ones(w.x) | all_ones(w.y) | all_ones(w.z) | all_ones(w.w);
  }
  if (some == 0u) return;
  *poisoned = 1u;
#pragma unroll 1
  for (int r = sub; r < live; r += 16)
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const int piece = i < 8 ? piece0 : piece1;
      uint16_t* at = reinterpret_cast<uint16_t*>(tile + tile_offset(r, piece)) + (i & 7);
      if ((*at & kExp & 0xffffu) == (kExp & 0xffffu)) {
        atomicMin(poison + 8 * piece + (i & 7), key + r);
        *at = 0;
      }
    }
}

template <bool kE4m3>
__global__ void __launch_bounds__(kTileThreads, 1) paged_attn_tile_kernel(const __grid_constant__ PagedTileParams tp) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const PagedAttnParams& p = tp.a;
  constexpr uint32_t T32 = TileSmem::kTile;
  uint8_t* sQ = smem + TileSmem::kQ;
  uint8_t* sK = smem + TileSmem::kK;
  uint8_t* sV = smem + TileSmem::kV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + TileSmem::kBar);
  uint64_t* q_full = bars + 0;    // [2] query tiles
  uint64_t* k_full = bars + 2;    // [2] ring stages
  uint64_t* k_empty = bars + 4;   // [2]
  uint64_t* v_full = bars + 6;    // [2]
  uint64_t* v_empty = bars + 8;   // [2]
  uint64_t* s_full = bars + 10;   // [2] query tiles
  uint64_t* p_full = bars + 12;   // [2 tiles][2 halves of the keys]
  uint64_t* o_full = bars + 16;   // [2]
  uint64_t* q_empty = bars + 18;  // [2]
  uint64_t* raw_full = bars + 20;   // [2] keys, values (e4m3)
  uint64_t* raw_empty = bars + 22;  // [2]
  uint64_t* q_raw = bars + 24;      // [2] query tiles before their conversion (e4m3)
  uint64_t* wide_full = bars + 26;   // [2] units: whether the unit is wide (e4m3)
  uint64_t* wide_empty = bars + 28;  // [2]
  uint64_t* v_raw = bars + 30;       // [2] values that are still to be cleaned (bf16)
  uint64_t* poison_empty = bars + 32;  // [2] query tiles: `poison` read
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 34);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile uint32_t* last_flag = tmem_slot + 2;
  volatile uint32_t* wide_flag = tmem_slot + 3;  // [2] units (e4m3)
  volatile uint32_t* poisoned = tmem_slot + 5;   // some value of the unit was taken out
  volatile uint32_t* span = tmem_slot + 6;       // the first unit's scales: keys largest, smallest, values (e4m3)
  int* poison = reinterpret_cast<int*>(smem + TileSmem::kPoison);

  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], kE4m3 ? 4 : 1);
      mbar_init(&k_full[i], kE4m3 ? 4 : 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], kE4m3 ? 4 : 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[2 * i], 4);
      mbar_init(&p_full[2 * i + 1], 4);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(&q_empty[0], 1);
    mbar_init(&q_empty[1], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
      mbar_init(&q_raw[i], 1);
      mbar_init(&wide_full[i], 1);
      mbar_init(&wide_empty[i], 4);
      mbar_init(&v_raw[i], 1);
      mbar_init(&poison_empty[i], 4);
    }
    *abort_flag = 0u;
    span[0] = span[2] = 0u;
    span[1] = span[3] = 255u;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_launch();
  grid_dep_wait();
  const WaitGuard wg{abort_flag, p.status};
  const int u_begin = p.cta_unit0[blockIdx.x], u_end = p.cta_unit0[blockIdx.x + 1];

  if (warp >= 8 && warp < 12) {
    regs_down<kE4m3 ? 80 : 64>();
    // eight lanes a row, four rows a warp at a time; lane e has pieces 2e and 2e + 1, those of the second 64 dims take
    // the odd one first, so that the eight lanes of a row hit all banks once
    const int ct = threadIdx.x - 8 * 32, sub = ct >> 3, e = ct & 7;
    const bool odd = e >= 4;
    const int piece0 = 2 * e + (odd ? 1 : 0), piece1 = 2 * e + (odd ? 0 : 1);
    int n_masked[2] = {0, 0};  // units that a query tile has read `poison` of
    // the values in a ring tile from `key` on, some of whose keys not all of the unit's rows see; `first`: of the unit
    auto clean = [&](uint8_t* tile, int key, int live, bool first, int rows, auto bf16_c) {
      if (first) {
        mbar_wait(&poison_empty[0], (n_masked[0] & 1) ^ 1u, wg);
        mbar_wait(&poison_empty[1], (n_masked[1] & 1) ^ 1u, wg);
        ++n_masked[0];
        if (rows > 128) ++n_masked[1];
        poison[ct] = INT_MAX;
        if (ct == 0) *poisoned = 0u;
        named_bar_sync(2, 128);
      }
      clean_tile<decltype(bf16_c)::value>(tile, key, live, sub, piece0, piece1, poison, poisoned);
    };
    if constexpr (!kE4m3) {
      // ---------------------------------------------------------- values on their way to the MMAs that some row must not meet
      int it = 0, n_raw[2] = {0, 0};
      for (int u = u_begin; u < u_end; ++u) {
        const PagedUnit un = p.units[u];
        const int all = seen_by_all(un, p.group);
        for (int key = un.key0; key < un.key1; key += kTileKeys, ++it) {
          const int s = it & 1, live = min(kTileKeys, un.key1 - key);
          if (live == kTileKeys && key + kTileKeys <= all) continue;
          mbar_wait(&v_raw[s], n_raw[s] & 1, wg);
          ++n_raw[s];
          uint8_t* tile = sV + s * T32;
          if (key + live > all) clean(tile, key, live, key == un.key0 || key <= all, un.rows - un.row0, std::true_type{});
          // what lies behind the last key must not reach the sum, whatever it is: zero
          for (int r = sub; r < kTileKeys; r += 16)
            if (r >= live) {
              *reinterpret_cast<uint4*>(tile + tile_offset(r, piece0)) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(tile + tile_offset(r, piece1)) = make_uint4(0, 0, 0, 0);
            }
          fence_proxy_async_smem();
          named_bar_sync(2, 128);
          if (ct == 0) mbar_arrive(&v_full[s]);
        }
      }
    } else {
      // ---------------------------------------------------------- e4m3 pages, bf16 queries -> f16 operand tiles
      volatile uint32_t* refs = reinterpret_cast<volatile uint32_t*>(smem + TileSmem::kRef);
      uint8_t* q_scale = smem + TileSmem::kQScale;
      int it = 0, n_unit[2] = {0, 0};
      // A tile; `masked`: its values are still to be cleaned. Code of its own for wide units: in the others' loop it cost
      // them 35 us of 240 (and the softmax's part another 30).
      auto convert = [&](int live, bool masked, auto wide_c) {
        constexpr bool kW = decltype(wide_c)::value;
        const int s = it & 1;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          mbar_wait(&raw_full[kv], it & 1, wg);
          const uint8_t* raw = smem + TileSmem::kRaw + kv * TileSmem::kRawTile;
          const uint8_t* scale = smem + TileSmem::kScale + kv * 128;
          uint8_t* dst = (kv ? sV : sK) + s * T32;
          // the tile's largest scale: lane i looks at rows 4i..4i+3; NaN rows and those behind the last key do not count
          uint32_t top = 0u;
          bool some_nan = false;
          {
            const uint32_t w = reinterpret_cast<const uint32_t*>(scale)[lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t b = (w >> (8 * i)) & 255u;
              if (4 * lane + i < live) {
                if (b != 255u) top = max(top, b);
                some_nan |= b == 255u;
              }
            }
          }
          const uint32_t ref = kW ? 127u : __reduce_max_sync(0xffffffffu, top);
          const bool near = !__any_sync(0xffffffffu, some_nan);
          // all of a tile is read before its place in the ring is waited for
          uint2 x0[8], x1[8];
          uint32_t f[8];
          {
            const uint8_t* src = raw + sub * 128 + e * 16;
            const uint32_t base = near_base(ref);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              x0[i] = *reinterpret_cast<const uint2*>(src + (odd ? 8 : 0) + i * 2048);
              x1[i] = *reinterpret_cast<const uint2*>(src + (odd ? 0 : 8) + i * 2048);
              f[i] = scale[16 * i + sub];
            }
            if constexpr (kW) {
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = __float_as_uint(e8m0_value(f[i]));
            } else if (near) {
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = f[i] * 0x04000400u + base;
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = near_factor(f[i], ref);
            }
            if (live < kTileKeys) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                // what lies behind the last key must not reach the sum, whatever it is
                if (16 * i + sub >= live) {
                  f[i] = 0u;
                  x0[i] = x1[i] = make_uint2(0u, 0u);
                }
              }
            }
          }
          mbar_wait(kv ? &v_empty[s] : &k_empty[s], ((it >> 1) & 1) ^ 1u, wg);
          if (ct == 0) refs[kv * 4 + (it & 3)] = ref | (kW && kv == 0 ? kWide : 0u);
          uint8_t* dst0 = dst + tile_offset(sub, piece0);
          uint8_t* dst1 = dst + tile_offset(sub, piece1);
          if constexpr (kW) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              *reinterpret_cast<uint4*>(dst0 + i * 2048) = dequant8(x0[i], __uint_as_float(f[i]));
              *reinterpret_cast<uint4*>(dst1 + i * 2048) = dequant8(x1[i], __uint_as_float(f[i]));
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              *reinterpret_cast<uint4*>(dst0 + i * 2048) = e4m3x8_f16(x0[i], f[i]);
              *reinterpret_cast<uint4*>(dst1 + i * 2048) = e4m3x8_f16(x1[i], f[i]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (!kv || !masked) mbar_arrive(kv ? &v_full[s] : &k_full[s]);
            mbar_arrive(&raw_empty[kv]);
          }
        }
      };
      // a unit's queries, in place: |q| / 2^x < 4 for the largest of a row; as they are where the unit is wide
      auto convert_queries = [&](int u, const PagedUnit& un, auto wide_c) {
        constexpr bool kW = decltype(wide_c)::value;
        const int rows = min(kTileRows, un.rows - un.row0);
        for (int t = 0; t * 128 < rows; ++t) {
          mbar_wait(&q_raw[t], n_unit[t] & 1, wg);
          ++n_unit[t];
          uint8_t* qt = sQ + t * T32;
          if (kW) q_scale[(u & 1) * 256 + t * 128 + ct] = 127u;
#pragma unroll 2
          for (int i = kW ? 8 : 0; i < 8; ++i) {
            const int r = 16 * i + sub;
            uint4* pa = reinterpret_cast<uint4*>(qt + tile_offset(r, e));
            uint4* pb = reinterpret_cast<uint4*>(qt + tile_offset(r, 8 + e));
            float a[8], b[8];
            unpack_bf16x8(*pa, a);
            unpack_bf16x8(*pb, b);
            float m = fmax3_nan(amax8(a), amax8(b), 0.f);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) m = fmax3_nan(m, __shfl_xor_sync(0xffffffffu, m, o), 0.f);
            const uint32_t ex = query_exponent(m);
            const float down = __uint_as_float((254u - ex) << 23);
            if (e == 0) q_scale[(u & 1) * 256 + t * 128 + r] = static_cast<uint8_t>(ex);
            *pa = make_uint4(pack_half2(a[0] * down, a[1] * down), pack_half2(a[2] * down, a[3] * down),
                             pack_half2(a[4] * down, a[5] * down), pack_half2(a[6] * down, a[7] * down));
            *pb = make_uint4(pack_half2(b[0] * down, b[1] * down), pack_half2(b[2] * down, b[3] * down),
                             pack_half2(b[4] * down, b[5] * down), pack_half2(b[6] * down, b[7] * down));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[t]);
        }
      };
      auto run_unit = [&](int u, const PagedUnit& un, auto wide_c) {
        const int all = seen_by_all(un, p.group);
        for (int key = un.key0; key < un.key1; key += kTileKeys, ++it) {
          const int live = min(kTileKeys, un.key1 - key);
          const bool masked = key + live > all;
          convert(live, masked, wide_c);
          if (masked) {
            // each thread what it has just written
            clean(sV + (it & 1) * T32, key, live, key == un.key0 || key <= all, un.rows - un.row0, wide_c);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&v_full[it & 1]);
          }
          if (key == un.key0) convert_queries(u, un, wide_c);
        }
      };
      for (int u = u_begin; u < u_end; ++u) {
        const PagedUnit un = p.units[u];
        bool wide;
        if (u == u_begin) {
          // the first unit's scales by all four warps: nothing can start before
          ScaleSpan keys, values;
          scan_scales(p, un, ct, 128, keys, values);
          const uint32_t k_top = keys.largest(), k_low = keys.smallest(), v_top = values.largest(), v_low = values.smallest();
          if (lane == 0) {
            uint32_t* sp = const_cast<uint32_t*>(span);
            atomicMax(sp + 0, k_top);
            atomicMin(sp + 1, k_low);
            atomicMax(sp + 2, v_top);
            atomicMin(sp + 3, v_low);
          }
          named_bar_sync(2, 128);
          wide = is_wide(span[0], span[1], span[2], span[3]);
        } else {
          const int n = u - u_begin - 1, slot = n & 1;
          mbar_wait(&wide_full[slot], (n >> 1) & 1, wg);
          wide = wide_flag[slot] != 0u;
          __syncwarp();
          if (lane == 0) mbar_arrive(&wide_empty[slot]);
        }
        if (wide)
          run_unit(u, un, std::true_type{});
        else
          run_unit(u, un, std::false_type{});
      }
    }
  } else if (warp >= 12) {
    regs_down<kE4m3 ? 80 : 64>();
    if (warp == 13) {
      // ---------------------------------------------------------- query tiles, a unit ahead
      int n_unit[2] = {0, 0};
      for (int u = u_begin; u < u_end; ++u) {
        const PagedUnit un = p.units[u];
        const int q0 = un.q0;
        const int rows = min(kTileRows, un.rows - un.row0);
        for (int t = 0; t * 128 < rows; ++t) {
          mbar_wait(&q_empty[t], (n_unit[t] & 1) ^ 1u, wg);
          ++n_unit[t];
          uint64_t* full = kE4m3 ? &q_raw[t] : &q_full[t];
          if (tp.q_tma) {
            // 128 / group tokens of the group's heads are the tile's rows in order; rows behind the sequence's last
            // are the next one's, or zero, and go nowhere
            if (lane == 0) {
              const int token = q0 + un.row0 / p.group + t * (128 / p.group);
              mbar_expect_tx(full, T32);
              tma_load_3d(sQ + t * T32, &tp.q_map, full, 0, un.head * p.group, token);
              tma_load_3d(sQ + t * T32 + 16384, &tp.q_map, full, 64, un.head * p.group, token);
            }
          } else {
#pragma unroll 4
            for (int i = lane; i < 128 * 16; i += 32) {
              const int r = t * 128 + (i >> 4), rr = un.row0 + r;
              uint4 w = make_uint4(0, 0, 0, 0);
              if (r < rows)
                w = __ldg(p.q + (static_cast<long long>(q0 + rr / p.group) * p.Hq + un.head * p.group + rr % p.group) * 16 + (i & 15));
              *reinterpret_cast<uint4*>(sQ + t * T32 + tile_offset(i >> 4, i & 15)) = w;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
          }
          __syncwarp();
        }
      }
    }
    if (warp == 14) {
      // ---------------------------------------------------------- pages; lane i takes page i of a tile
      const int ps = 1 << p.page_shift;
      int it = 0;  // key tiles so far, over all units
      for (int u = u_begin; u < u_end; ++u) {
        const PagedUnit un = p.units[u];
        const int* pages = p.pages + un.page0;
        const int all = seen_by_all(un, p.group);
        for (int key = un.key0; key < un.key1; key += kTileKeys, ++it) {
          const int s = it & 1;
          const uint32_t ph = (it >> 1) & 1;
          const int live = min(kTileKeys, un.key1 - key);  // keys of the tile that the unit uses
          const int n_pages = (live + ps - 1) >> p.page_shift;
          int row = 0;  // first pool row of the page
          if (lane < n_pages) row = (pages[(key >> p.page_shift) + lane] * p.Hkv + un.head) << p.page_shift;
          if constexpr (kE4m3) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              if (lane == 0) {
                mbar_wait(&raw_empty[kv], (it & 1) ^ 1u, wg);
                mbar_expect_tx(&raw_full[kv], static_cast<uint32_t>(n_pages * ps) * 129u);
              }
              __syncwarp();
              if (lane < n_pages) {
                tma_load_2d(smem + TileSmem::kRaw + kv * TileSmem::kRawTile + lane * ps * 128, kv ? &tp.v_map : &tp.k_map,
                            &raw_full[kv], 0, row);
                bulk_load(smem + TileSmem::kScale + kv * 128 + lane * ps, (kv ? p.pool.vs : p.pool.ks) + row, ps, &raw_full[kv]);
              }
            }
          } else {
            const uint32_t bytes = static_cast<uint32_t>(n_pages * ps) * 256u;
            if (lane == 0) {
              mbar_wait(&k_empty[s], ph ^ 1u, wg);
              mbar_expect_tx(&k_full[s], bytes);
            }
            __syncwarp();
            if (lane < n_pages) {
              uint8_t* dst = sK + s * T32 + lane * (ps * 128);
              tma_load_2d(dst, &tp.k_map, &k_full[s], 0, row);
              tma_load_2d(dst + 16384, &tp.k_map, &k_full[s], 64, row);
            }
            uint64_t* vb = live < kTileKeys || key + kTileKeys > all ? &v_raw[s] : &v_full[s];  // warps 8-11 clean it first
            if (lane == 0) {
              mbar_wait(&v_empty[s], ph ^ 1u, wg);
              mbar_expect_tx(vb, bytes);
            }
            __syncwarp();
            if (lane < n_pages) {
              uint8_t* dst = sV + s * T32 + lane * (ps * 128);
              tma_load_2d(dst, &tp.v_map, vb, 0, row);
              tma_load_2d(dst + 16384, &tp.v_map, vb, 64, row);
            }
          }
        }
      }
    }
    if constexpr (kE4m3) {
      if (warp == 15) {
        // -------------------------------------------------------- is the unit wide? A unit or two ahead, after the first
        for (int u = u_begin + 1; u < u_end; ++u) {
          const PagedUnit un = p.units[u];
          ScaleSpan keys, values;
          scan_scales(p, un, lane, 32, keys, values);
          const bool wide = is_wide(keys.largest(), keys.smallest(), values.largest(), values.smallest());
          const int n = u - u_begin - 1, slot = n & 1;
          if (lane == 0) {
            mbar_wait(&wide_empty[slot], ((n >> 1) & 1) ^ 1u, wg);
            wide_flag[slot] = wide;
            mbar_arrive(&wide_full[slot]);
          }
          __syncwarp();
        }
      }
    }
    // ------------------------------------------------------------ MMA issue
    if (warp == 12) {
      const bool leader = elect_one();
      int it = 0, n_unit[2] = {0, 0}, n_p[2] = {0, 0};  // key tiles; units and key tiles per query tile
      const uint64_t q_desc = kmajor_desc(smem_u32(sQ), 0, 16384), k_desc = kmajor_desc(smem_u32(sK), 0, 16384);
      const uint64_t v_desc = mnmajor_desc(smem_u32(sV), 0, 16384);
      auto issue_s = [&](int t, int stage, bool last, uint32_t idesc_qk) {
        const uint64_t qd = q_desc + t * (T32 >> 4), kd = k_desc + stage * (T32 >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t step = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            umma_ss(tmem + t * 128u, qd + step, kd + step, idesc_qk, kk > 0);
          }
          umma_commit(&s_full[t]);
          if (last) umma_commit(&q_empty[t]);
        }
      };
      auto run_unit = [&](const PagedUnit& un, auto bf16_c) {
        constexpr bool kB = decltype(bf16_c)::value;
        constexpr uint32_t idesc_qk = idesc_f16(128, 128, kB, kB, false, false);
        constexpr uint32_t idesc_pv = idesc_f16(128, 128, kB, kB, false, true);
        const int rows = un.rows - un.row0;
        const int nt = rows > 128 ? 2 : 1;
        const int tiles = (un.key1 - un.key0 + kTileKeys - 1) / kTileKeys;
        for (int j = 0; j < tiles; ++j, ++it) {
          const int s = it & 1;
          const uint32_t ph = (it >> 1) & 1;
          if (j == 0) {
            mbar_wait(&k_full[s], ph, wg);
            for (int t = 0; t < nt; ++t) {
              mbar_wait(&q_full[t], n_unit[t] & 1, wg);
              ++n_unit[t];
              tc_fence_after();
              __syncwarp();
              issue_s(t, s, tiles == 1, idesc_qk);
            }
            if (leader) umma_commit(&k_empty[s]);
          }
          const bool more = j + 1 < tiles;
          const int s1 = (it + 1) & 1;
          mbar_wait(&v_full[s], ph, wg);
          const uint64_t vd = v_desc + s * (T32 >> 4);
          for (int t = 0; t < nt; ++t) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              mbar_wait(&p_full[2 * t + half], n_p[t] & 1, wg);
              tc_fence_after();
              __syncwarp();
              if (leader) {
#pragma unroll
                for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                  umma_ts(tmem + 256u + t * 128u, tmem + t * 128u + kk * 8u, vd + kk * 128u, idesc_pv, (j | kk) != 0);
              }
            }
            ++n_p[t];
            if (leader && !more) umma_commit(&o_full[t]);
            if (leader && t == nt - 1) umma_commit(&v_empty[s]);
            if (more) {
              if (t == 0) {
                mbar_wait(&k_full[s1], ((it + 1) >> 1) & 1, wg);
                tc_fence_after();
                __syncwarp();
              }
              issue_s(t, s1, j + 2 == tiles, idesc_qk);  // overwrites P_t only after the P V MMAs above (in-order issue)
              if (leader && t == nt - 1) umma_commit(&k_empty[s1]);
            }
          }
        }
      };
      for (int u = u_begin; u < u_end; ++u) {
        const PagedUnit un = p.units[u];
        if constexpr (kE4m3) {
          mbar_wait(&k_full[it & 1], (it >> 1) & 1, wg);  // the flag stands beside the first key tile's reference
          if (reinterpret_cast<const volatile uint32_t*>(smem + TileSmem::kRef)[it & 3] & kWide)
            run_unit(un, std::true_type{});
          else
            run_unit(un, std::false_type{});
        } else {
          run_unit(un, std::true_type{});
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax, one thread per query row
    regs_up<kE4m3 ? 176 : 192>();
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t * 128u + lane_off;
    const uint32_t tO = tmem + 256u + t * 128u + lane_off;
    const volatile uint32_t* refs = reinterpret_cast<const volatile uint32_t*>(smem + TileSmem::kRef);
    int n_s = 0, n_unit = 0;
    int it = 0;  // key tiles so far, over all units
    for (int u = u_begin; u < u_end; ++u) {
      int key0, key1, limit;
      bool active, masked;
      {
        const PagedUnit un = read_unit(p.units + u);
        key0 = un.key0;
        key1 = un.key1;
        const int unit_rows = min(kTileRows, un.rows - un.row0);
        active = t * 128 < unit_rows;
        masked = seen_by_all(un, p.group) < un.key1;
        limit = max(un.vis, un.past + (un.row0 + min(t * 128 + row, unit_rows - 1)) / p.group + 1);
      }
      if (!active) {
        it += (key1 - key0 + kTileKeys - 1) / kTileKeys;
        continue;
      }
      float m_run = -INFINITY, l_run = 0.f;
      float q_factor = p.scale_log2;
      int v_ref = 0;  // e4m3: largest value scale so far; O counts in units of 2^(v_ref - 127 - kWeightUp), or of 1 (wide)
      auto run_tiles = [&](auto bf16_c) {
        constexpr bool kB = decltype(bf16_c)::value;  // operands
        bool first = true, far = false;
        for (int key = key0; key < key1; key += kTileKeys, ++n_s, ++it) {
          mbar_wait(&s_full[t], n_s & 1, wg);
          tc_fence_after();
          const int valid = limit - key;  // keys of this tile that this row sees
          // warp-uniform, as the tcgen05 instructions in the branches are
          const bool full = __all_sync(0xffffffffu, valid >= kTileKeys);
          uint32_t s[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
          tmem_ld_wait();
          if (!full) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (c * 32 + i >= valid) s[c][i] = __float_as_uint(-INFINITY);
          }
          const float mx = scores_max(s);
          float scale = p.scale_log2, v_down = 0.f;
          bool v_grow = false;
          if constexpr (kE4m3) {
            if (first) q_factor *= __uint_as_float(static_cast<uint32_t>((smem + TileSmem::kQScale)[(u & 1) * 256 + t * 128 + row]) << 23);
            // at least 2^-126: as good as 0 for scores, and -infinity times it is -infinity
            scale = fmaxf(q_factor * e8m0_value(refs[it & 3] & 255u), FLT_MIN);
          }
          if constexpr (!kB) {
            mbar_wait(&v_full[it & 1], (it >> 1) & 1, wg);  // the values' scales; long there but for the first tile
            const int v_tile = static_cast<int>(refs[4 + (it & 3)]);
            if (first) v_ref = v_tile;
            v_grow = v_tile > v_ref;
            v_down = v_grow ? static_cast<float>(v_ref - v_tile) : 0.f;  // of what O holds
            v_ref = max(v_ref, v_tile);
          }
          float m_tile = mx * scale;
          if (m_tile == INFINITY) m_tile = NAN;  // infinite scores have no softmax
          // raised by -inf -> finite, by more than 2^8, and for good by a NaN
          const bool need = !(m_tile <= m_run + kLazyRescaleLog2);
          if (__any_sync(0xffffffffu, need) || v_grow) {
            const float m_new = need ? m_tile : m_run;
            const float alpha = need ? ex2_approx(m_run - m_new) : 1.f;
            m_run = m_new;
            far = __any_sync(0xffffffffu, fabsf(m_run) >= kFarScore && m_run > -INFINITY);
            if (!first) {
              const float o_down = kB ? alpha : alpha * ex2_approx(v_down);
              // S of this tile was issued after the previous P V, which is therefore complete
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                uint32_t r[16];
                tmem_ld16(tO + c * 16, r);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * o_down);
                tmem_st16(tO + c * 16, r);
              }
              l_run *= alpha;
            }
          }
          first = false;
          float neg_m = -finite_or_zero(m_run), p_up = 1.f;
          if (far) {
            // Through TMEM and rolled up, to stay out of the loop's way. All rows of the warp take part.
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t r[16];
              tmem_ld16(tS + c * 16, r);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                r[i] = c * 16 + i >= valid ? __float_as_uint(-INFINITY)
                                           : __float_as_uint(__fadd_rn(__fmul_rn(__uint_as_float(r[i]), scale), neg_m));
              tmem_st16(tS + c * 16, r);
            }
            tmem_st_wait();
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
            tmem_ld_wait();
            scale = 1.f;
            neg_m = 0.f;
          }
          if constexpr (!kB) {
            // weights relative to the largest value scale; the row sum without it
            const float up = fmaxf(static_cast<float>(static_cast<int>(refs[4 + (it & 3)]) - v_ref), -100.f) + kWeightUp;
            neg_m += up;
            p_up = ex2_approx(-up);
          }
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
#pragma unroll
            for (int c = 2 * half; c < 2 * half + 2; ++c) scores_exp32<kB>(s[c], tS + c * 16, scale, neg_m, sum);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * t + half]);
          }
          const float tile_sum = (sum[0] + sum[1]) + (sum[2] + sum[3]);
          l_run = kB ? l_run + tile_sum : fmaf(tile_sum, p_up, l_run);
        }
      };
      bool wide = false;
      if constexpr (kE4m3) {
        mbar_wait(&s_full[t], n_s & 1, wg);
        wide = (refs[it & 3] & kWide) != 0u;
        if (wide)
          run_tiles(std::true_type{});
        else
          run_tiles(std::false_type{});
      } else {
        run_tiles(std::true_type{});
      }
      mbar_wait(&o_full[t], n_unit & 1, wg);
      ++n_unit;
      tc_fence_after();
      const PagedUnit un = read_unit(p.units + u);
      const int unit_rows = min(kTileRows, un.rows - un.row0);
      const bool live = t * 128 + row < unit_rows;
      auto out_row_of = [&](int r) {  // row of [T, Hq] of the unit's row r
        const int rr = un.row0 + r;
        return static_cast<long long>(un.q0 + rr / p.group) * p.Hq + un.head * p.group + rr % p.group;
      };
      const int nsplit = un.split >> 16, split = un.split & 0xffff;
      const float inv_l = nsplit == 1 ? 1.0f / l_run : 1.0f;
      const float unit_v = kE4m3 && !wide ? e8m0_value(static_cast<uint32_t>(v_ref)) * 0.0078125f : 1.0f;  // 2^-kWeightUp
      const float inv = inv_l * unit_v;
      const long long orow = out_row_of(min(t * 128 + row, unit_rows - 1));
      float* slot = p.part + static_cast<long long>(un.slot0 + split) * kTileSlot;
      const bool some_nan = masked && *poisoned != 0u;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        tmem_ld32(tO + c * 32, r);
        tmem_ld_wait();
        if (some_nan) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (poison[c * 32 + i] < limit) r[i] = 0x7fc00000u;
        }
        if (live && nsplit == 1) {
          store_row32(p.o + orow * 16 + c * 4, r, inv);
        } else if (live) {
          float4* dst = reinterpret_cast<float4*>(slot) + c * 8 * kTileRows + t * 128 + row;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i * kTileRows] = make_float4(__uint_as_float(r[4 * i]) * unit_v, __uint_as_float(r[4 * i + 1]) * unit_v,
                                             __uint_as_float(r[4 * i + 2]) * unit_v, __uint_as_float(r[4 * i + 3]) * unit_v);
        }
        __syncwarp();
      }
      if (live) {
        if (nsplit > 1)
          reinterpret_cast<float2*>(slot + kTileRows * 128)[t * 128 + row] = make_float2(m_run, l_run);
        else if (p.lse)
          p.lse[orow] = lse_of(m_run, l_run);
      }
      if (masked && lane == 0) mbar_arrive(&poison_empty[t]);  // the warp has read it: converged since the loads above
      if (nsplit > 1) {
        // the last range to arrive merges all, in the order of the ranges
        const int threads = unit_rows > 128 ? 256 : 128;
        named_bar_sync(1, threads);
        if (threadIdx.x == 0) {
          // one fence for the writes that the barrier put before it
          __threadfence();
          *last_flag = atomicInc(reinterpret_cast<unsigned*>(p.counters) + un.counter, nsplit - 1) == nsplit - 1;
          __threadfence();
        }
        named_bar_sync(1, threads);
        const bool last = *last_flag != 0u;
        named_bar_sync(1, threads);  // read by all before the next unit may write it
        if (last && live) {
          const float* slots = p.part + static_cast<long long>(un.slot0) * kTileSlot;
          const int my = t * 128 + row;
          auto ml_of = [&](int i) {
            return __ldcg(reinterpret_cast<const float2*>(slots + static_cast<long long>(i) * kTileSlot + kTileRows * 128) + my);
          };
          float m = -INFINITY, l = 0.f;
#pragma unroll 4
          for (int i = 0; i < nsplit; ++i) m = fmaxf(m, ml_of(i).x);
          const float m0 = finite_or_zero(m);
#pragma unroll 4
          for (int i = 0; i < nsplit; ++i) {
            const float2 ml = ml_of(i);
            l = fmaf(ml.y, ex2_approx(ml.x - m0), l);
          }
          if (p.lse) p.lse[orow] = lse_of(m, l);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float acc[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0.f;
#pragma unroll 3
            for (int i = 0; i < nsplit; ++i) {
              const float4* src = reinterpret_cast<const float4*>(slots + static_cast<long long>(i) * kTileSlot) + c * 8 * kTileRows + my;
              float4 v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) v[k] = __ldcg(src + k * kTileRows);
              const float w = ex2_approx(ml_of(i).x - m0);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                acc[4 * k] = fmaf(v[k].x, w, acc[4 * k]);
                acc[4 * k + 1] = fmaf(v[k].y, w, acc[4 * k + 1]);
                acc[4 * k + 2] = fmaf(v[k].z, w, acc[4 * k + 2]);
                acc[4 * k + 3] = fmaf(v[k].w, w, acc[4 * k + 3]);
              }
            }
            uint32_t r[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(acc[i]);
            store_row32(p.o + orow * 16 + c * 4, r, 1.0f / l);
          }
        }
      }
      tc_fence_before();  // the next unit's MMAs overwrite O after this thread's q_full arrival
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace mot
