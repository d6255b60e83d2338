// mot_paged.cuh -- C ABI of the paged prefix-KV cache (see
// include/mot_paged.h). Same translation unit as mot_attn.cu.
//
// One launch per call:
//   append   norm + rotation + cache write of the chunk
//   store    dense cache -> pages
//   load     pages -> dense cache
//   attend   attention units cut over the SMs by mot_paged_batch_set: one
//            launch for the sequences with few query rows, one for the others
#pragma once

#include "mot_paged.h"
#include "paged.cuh"
#include "paged_tile.cuh"

struct mot_paged {
  mot_paged_config cfg;
  int device = 0;
  int num_sms = 148;
  int ctas[2] = {0, 0};    // grids of the few-rows and of the 256-row attention
  float* gains = nullptr;  // q_norm [128], k_norm [128]
  float2* rope = nullptr;  // [max_positions, 64]
  int* status = nullptr;
};

namespace {

// Device tables of a batch object, at fixed offsets (32-bit words) so that a
// captured call finds them after the batch is set again. [0]: the few-rows
// attention, [1]: the 256-row one.
struct PagedTables {
  size_t counters[2], cta_unit0[2], n_entries, head_words;  // one block, one copy
  size_t pages, entries, tok, units[2], words;
  int unit_cap[2];
};

static_assert(TileSmem::bytes(true) <= 232448, "shared memory");

// Query rows (tokens times heads of the group) up to which a sequence goes to the
// few-rows kernel, which reads the keys once for every 8 of them; `mid`: how many
// (sequence, KV head) pairs have 9 to 32 rows. A rule on q_len alone, so that a
// captured call keeps its launches. Measured, us of the few-rows | the 256-row
// kernel at 16 / 24 / 32 rows: bf16, 1 sequence of 4000 keys 12.5 / 14 / 15 | 24,
// 8 of 2000 24 / 31 / 34 | 24, 64 of 2000 165 / 204 / 312 | 105; e4m3 11.6 / 12.8 /
// 13.5 | 28, 20.5 / 27 / 30 | 32, 105 / 153 / 196 | 157. Not followed at 25 to 32 rows of
// one or two bf16 sequences, where the few-rows kernel would be the faster one over
// long caches (15 against 20 to 24 us; the same at 500 keys).
constexpr int kSmallMaxRows = 32;
int small_rows(bool e4m3, long long mid) {
  return e4m3 ? (mid <= 64 ? 32 : 24) : mid <= 16 ? 24 : mid <= 64 ? 16 : 8;
}

PagedTables paged_tables(const mot_paged_config& c, const int (&ctas)[2]) {
  PagedTables t;
  size_t off = 0;
  auto take = [&](size_t words) {
    const size_t o = off;
    off += round_up(words, 4);
    return o;
  };
  const size_t B = c.max_batch, T = c.max_tokens, G = c.n_q_heads / c.n_kv_heads;
  for (int i = 0; i < 2; ++i) t.counters[i] = take(ctas[i]);
  for (int i = 0; i < 2; ++i) t.cta_unit0[i] = take(ctas[i] + 1);
  t.n_entries = take(1);
  t.head_words = off;
  t.pages = take(c.max_pages);
  t.entries = take(4 * static_cast<size_t>(c.max_pages));
  t.tok = take(2 * T);
  const size_t seqs = std::min(B, T);
  const size_t tiles[2] = {seqs * (kSmallMaxRows / kSmallRows), T * G / kTileRows + seqs};
  for (int i = 0; i < 2; ++i) {
    t.unit_cap[i] = static_cast<int>(tiles[i] * c.n_kv_heads + ctas[i]);  // every cut makes one more
    t.units[i] = take(static_cast<size_t>(t.unit_cap[i]) * (sizeof(PagedUnit) / 4));
  }
  t.words = off;
  return t;
}

mot_status check_paged_config(const mot_paged_config* c) {
  if (!c || c->n_q_heads <= 0 || c->n_kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0 || c->max_positions <= 0 ||
      c->max_batch <= 0 || c->max_tokens <= 0 || c->max_pages <= 0 || !(c->rms_eps >= 0.f) || !(c->rope_theta > 0.0) ||
      (c->kv_dtype != MOT_PAGED_BF16 && c->kv_dtype != MOT_PAGED_E4M3))
    return MOT_ERR_INVALID_ARGUMENT;
  if (c->head_dim != 128 || c->n_q_heads % c->n_kv_heads != 0 || c->n_q_heads / c->n_kv_heads > 64 ||
      c->n_q_heads > 1024 ||
      (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) ||
      c->max_positions > (1 << 22) || c->max_batch > 4096 || c->max_tokens > (1 << 20) || c->max_pages > (1 << 22) ||
      static_cast<long long>(c->max_tokens) * c->n_q_heads > (1ll << 26))
    return MOT_ERR_UNSUPPORTED_SHAPE;
  return MOT_OK;
}

void release_paged(mot_paged* h) {
  if (!h) return;
  cudaFree(h->gains);
  cudaFree(h->rope);
  cudaFree(h->status);
  delete h;
}

}  // namespace

struct mot_paged_batch {
  mot_paged* h = nullptr;
  PagedTables t;
  int* dev = nullptr;
  std::vector<int> host;        // mirror of the device tables
  std::vector<uint32_t> stamp;  // per page of the pool: set number, for repeated pages
  std::vector<uint8_t> times;
  uint32_t set_no = 0;
  // what the last set described
  int batch = 0, tokens = 0, entries = 0, n_pages = 0, kv_max = 0, units[2] = {0, 0};
  bool repeated = false, repeated_written = false;
};

namespace {

// a CUDA call has failed: its error must not be taken for that of a later call
mot_status cuda_failed() {
  cudaGetLastError();
  return MOT_ERR_CUDA;
}

int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// How the attention's tiles -- (sequence, KV head, query rows), each with its
// own number of keys -- go to the CTAs. Either whole, the longest first, each to
// the CTA with the least work so far; or cut: the CTAs take equal shares of the
// work in tile order, a tile that straddles a boundary is split there, at a
// multiple of `granule` keys, and its ranges are merged on the device. The
// cheaper by this count of work, in granules: a unit's prologue and epilogue cost
// `unit`, a range of a split tile `split` more (its partial result and the
// merge), and a share is at least `min_share`, one more where a tile has more than
// `many` granules. Measured. Costs: 64 sequences of 1000 8-bit keys, few rows, 32 us,
// 37.5 with a unit at 1 and a split at 0; 256 rows: 2 us a key tile, 3 us a unit, 4-5
// us more a range. min_share | one more, us in a graph, one sequence of 1000 / 2000 /
// 3000 / 4500 keys: few rows bf16 7.2 / 7.7 / 8.0 / 9.7 | 9.1 / 8.9 / 9.1 / 9.7, e4m3
// 7.1 / 7.9 / 8.7 / 10.6 | 7.9 / 8.2 / 9.2 / 9.8; 64 tokens of 4 heads a group bf16
// 19.7 / 22.2 / 25.4 / 28.1 | 21.1 / 23.7 / 24.5 / 27.4, e4m3 32.4 / 34.8 / 38.7 / 44.9 |
// 33.4 / 35.8 / 37.2 / 41.9; no difference from 8000 keys or 8 sequences on.
struct CutRule {
  int granule, unit, split, min_share, many;
};
constexpr CutRule kCutRules[2] = {{128, 2, 2, 5, 30}, {kTileKeys, 2, 2, 7, 20}};

struct PagedTile {
  int seq, row0, keys;
};

int granules_of(const PagedTile& t, const CutRule& rule) { return (t.keys + rule.granule - 1) / rule.granule; }

PagedUnit unit_of(const PagedTile& t, int head, int key0, int key1) {
  return PagedUnit{t.seq, head, t.row0, key0, key1, 0, 1 << 16, 0, 0, 0, 0, 0, 0, {0, 0, 0}};
}

// Cut into shares of `share`; returns whether that fits. `units` null: only the test.
bool cut_units(const std::vector<PagedTile>& tiles, int heads, int ctas, long long share, const CutRule& rule,
               PagedUnit* units, int unit_cap, int* cta_unit0, int* n_units) {
  int cta = 0, n = 0, slots = 0, counters = 0;
  long long load = 0;
  if (units) cta_unit0[0] = 0;
  for (const PagedTile& tl : tiles) {
    const int granules = granules_of(tl, rule);
    for (int head = 0; head < heads; ++head) {
      const int first = n;
      int at = 0;
      while (at < granules) {
        const bool whole = at == 0 && load + rule.unit + granules <= share;
        const long long room = whole ? granules : share - load - rule.unit - rule.split;
        if (load > 0 && room < 1) {
          if (++cta >= ctas) return false;
          if (units) cta_unit0[cta] = n;
          load = 0;
          continue;
        }
        const int take = static_cast<int>(std::min<long long>(std::max<long long>(room, 1), granules - at));
        if (units) {
          if (n >= unit_cap) return false;
          units[n] = unit_of(tl, head, at * rule.granule, std::min(tl.keys, (at + take) * rule.granule));
        }
        ++n;
        at += take;
        load += take + rule.unit + (whole ? 0 : rule.split);
      }
      const int pieces = n - first;
      if (units)
        for (int i = 0; i < pieces; ++i) {
          units[first + i].slot0 = slots;
          units[first + i].split = i | (pieces << 16);
          units[first + i].counter = counters;
        }
      if (pieces > 1) {
        slots += pieces;
        ++counters;
      }
    }
  }
  if (units) {
    for (int i = cta + 1; i <= ctas; ++i) cta_unit0[i] = n;
    *n_units = n;
  }
  return true;
}

bool plan_units(const std::vector<PagedTile>& tiles, int heads, int ctas, const CutRule& rule, PagedUnit* units,
                int unit_cap, int* cta_unit0, int* n_units) {
  long long total = 0;
  int longest = 0;
  for (const PagedTile& tl : tiles) {
    total += static_cast<long long>(granules_of(tl, rule) + rule.unit) * heads;
    longest = std::max(longest, granules_of(tl, rule));
  }
  // smallest share that fits
  long long lo = std::max<long long>(rule.min_share + (longest > rule.many), (total + ctas - 1) / ctas), hi = lo;
  while (!cut_units(tiles, heads, ctas, hi, rule, nullptr, 0, nullptr, nullptr)) {
    lo = hi + 1;
    hi *= 2;
  }
  while (lo < hi) {
    const long long mid = lo + (hi - lo) / 2;
    if (cut_units(tiles, heads, ctas, mid, rule, nullptr, 0, nullptr, nullptr))
      hi = mid;
    else
      lo = mid + 1;
  }
  // whole tiles, the longest first, to the CTA with the least work so far
  const int n = static_cast<int>(tiles.size()) * heads;
  std::vector<int> order(n), owner(n);
  for (int i = 0; i < n; ++i) order[i] = i;
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return tiles[a / heads].keys > tiles[b / heads].keys; });
  std::priority_queue<std::pair<long long, int>, std::vector<std::pair<long long, int>>, std::greater<>> free_cta;
  for (int i = 0; i < ctas; ++i) free_cta.push({0, i});
  long long largest = 0;
  for (int i : order) {
    auto [load, cta] = free_cta.top();
    free_cta.pop();
    owner[i] = cta;
    load += granules_of(tiles[i / heads], rule) + rule.unit;
    largest = std::max(largest, load);
    free_cta.push({load, cta});
  }
  if (lo < largest) return cut_units(tiles, heads, ctas, lo, rule, units, unit_cap, cta_unit0, n_units);
  if (n > unit_cap) return false;
  std::fill(cta_unit0, cta_unit0 + ctas + 1, 0);
  for (int i = 0; i < n; ++i) ++cta_unit0[owner[i] + 1];
  for (int i = 0; i < ctas; ++i) cta_unit0[i + 1] += cta_unit0[i];
  std::vector<int> at(cta_unit0, cta_unit0 + ctas);
  for (int i : order) units[at[owner[i]]++] = unit_of(tiles[i / heads], i % heads, 0, tiles[i / heads].keys);
  *n_units = n;
  return true;
}

// device memory of the current device
bool on_current_device(const void* p) {
  int dev = -1;
  cudaPointerAttributes a{};
  if (cudaGetDevice(&dev) == cudaSuccess && cudaPointerGetAttributes(&a, p) == cudaSuccess)
    return a.type == cudaMemoryTypeManaged || (a.type == cudaMemoryTypeDevice && a.device == dev);
  cudaGetLastError();
  return false;
}

bool paged_device_ok(const mot_paged* h) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == h->device;
}

// what append, store, load and attend check alike
mot_status check_paged_call(mot_paged_t h, mot_paged_batch_t bt, const mot_paged_pool* pool) {
  if (!h || !bt || bt->h != h || !pool || !pool->k || !pool->v || bt->batch <= 0) return MOT_ERR_INVALID_ARGUMENT;
  const bool e4m3 = h->cfg.kv_dtype == MOT_PAGED_E4M3;
  if (e4m3 != (pool->k_scale != nullptr) || e4m3 != (pool->v_scale != nullptr) || pool->n_pages < bt->n_pages)
    return MOT_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {pool->k, pool->v, pool->k_scale, pool->v_scale};
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return MOT_ERR_ALIGNMENT;
  if (!paged_device_ok(h)) return MOT_ERR_INVALID_ARGUMENT;
  return MOT_OK;
}

PagedPool pool_view(const mot_paged_pool* p) {
  return PagedPool{static_cast<uint8_t*>(p->k), static_cast<uint8_t*>(p->v), static_cast<uint8_t*>(p->k_scale),
                   static_cast<uint8_t*>(p->v_scale)};
}

// rows of 128 bytes, box of `box_rows` rows, as they are or in the 128-byte swizzle
bool map_bytes(CUtensorMap* m, const void* ptr, uint64_t rows, uint32_t box_rows, bool swizzle) {
  const cuuint64_t dims[2] = {128, rows}, strides[1] = {128};
  const cuuint32_t box[2] = {128, box_rows}, es[2] = {1, 1};
  return encode_ready() && g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, es,
                                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

mot_status paged_copy(mot_paged_t h, mot_paged_batch_t bt, void* k, void* v, int32_t rows, const mot_paged_pool* pool,
                      bool store, cudaStream_t st) {
  if (rows < bt->kv_max || (store && bt->repeated)) return MOT_ERR_INVALID_ARGUMENT;
  if (rows == 0) return MOT_OK;
  if (!k || !v || (!store && k == v)) return MOT_ERR_INVALID_ARGUMENT;
  if (!aligned16(k) || !aligned16(v)) return MOT_ERR_ALIGNMENT;
  const mot_paged_config& c = h->cfg;
  PagedCopyParams p{};
  p.dense[0] = static_cast<uint4*>(k);
  p.dense[1] = static_cast<uint4*>(v);
  p.pool = pool_view(pool);
  p.entries = reinterpret_cast<const int4*>(bt->dev + bt->t.entries);
  p.n_entries = bt->dev + bt->t.n_entries;
  p.rows = rows;
  p.Hkv = c.n_kv_heads;
  p.page_shift = log2_of(c.page_size);
  const long long items = static_cast<long long>(bt->entries) * c.n_kv_heads * 2 * (c.page_size / 16);
  // launched for an empty batch too: a captured call must find what the batch holds when it is replayed
  const int grid = static_cast<int>(std::min<long long>(std::max<long long>((items + 7) / 8, 1), 128ll * h->num_sms));
  const bool e4m3 = c.kv_dtype == MOT_PAGED_E4M3;
  auto kern = e4m3 ? (store ? paged_copy_kernel<true, true> : paged_copy_kernel<true, false>)
                   : (store ? paged_copy_kernel<false, true> : paged_copy_kernel<false, false>);
  return launch_pdl(kern, dim3(grid), dim3(256), 0, st, p) == cudaSuccess ? MOT_OK : cuda_failed();
}

}  // namespace

extern "C" {

mot_status mot_paged_create(const mot_paged_config* cfg, const mot_paged_weights* w, void* stream, mot_paged_t* out) {
  if (!out) return MOT_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  const mot_status st = check_paged_config(cfg);
  if (st != MOT_OK) return st;
  if (!w || !w->q_norm || !w->k_norm) return MOT_ERR_INVALID_ARGUMENT;
  if (!aligned16(w->q_norm) || !aligned16(w->k_norm)) return MOT_ERR_ALIGNMENT;
  // the kernels below read them: another GPU's memory would be an illegal address
  if (!on_current_device(w->q_norm) || !on_current_device(w->k_norm)) return MOT_ERR_INVALID_ARGUMENT;
  mot_paged* h = new (std::nothrow) mot_paged();
  if (!h) return MOT_ERR_CUDA;
  h->cfg = *cfg;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaGetLastError();  // asked for below: not an earlier call's
  const bool e4m3 = cfg->kv_dtype == MOT_PAGED_E4M3;
  set_smem_attr(e4m3 ? paged_attn_tile_kernel<true> : paged_attn_tile_kernel<false>, TileSmem::bytes(e4m3));
  const uint32_t small_smem = e4m3 ? SmallShape<true>::kBytes : SmallShape<false>::kBytes;
  set_smem_attr(e4m3 ? paged_attn_small_kernel<true> : paged_attn_small_kernel<false>, small_smem);
  int per_sm = 0;
  bool ok = cudaGetDevice(&h->device) == cudaSuccess &&
            cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) == cudaSuccess &&
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, e4m3 ? paged_attn_small_kernel<true> : paged_attn_small_kernel<false>,
                                                          e4m3 ? SmallShape<true>::kThreads : SmallShape<false>::kThreads, small_smem) ==
                cudaSuccess &&
            per_sm > 0 && encode_ready() && cudaMalloc(&h->gains, 256 * sizeof(float)) == cudaSuccess &&
            cudaMalloc(&h->rope, static_cast<size_t>(cfg->max_positions) * 64 * sizeof(float2)) == cudaSuccess &&
            cudaMalloc(&h->status, sizeof(int)) == cudaSuccess;
  if (ok) {
    h->ctas[0] = per_sm * h->num_sms;
    h->ctas[1] = h->num_sms;
    RopeFreq f;
    for (int j = 0; j < 64; ++j) f.inv[j] = std::pow(cfg->rope_theta, -2.0 * j / 128.0);
    bf16_to_f32_kernel<<<1, 128, 0, s>>>(static_cast<const __nv_bfloat16*>(w->q_norm), h->gains, 128);
    bf16_to_f32_kernel<<<1, 128, 0, s>>>(static_cast<const __nv_bfloat16*>(w->k_norm), h->gains + 128, 128);
    paged_rope_kernel<<<4 * h->num_sms, 256, 0, s>>>(h->rope, cfg->max_positions, f);
    ok = cudaGetLastError() == cudaSuccess && cudaMemsetAsync(h->status, 0, sizeof(int), s) == cudaSuccess &&
         cudaStreamSynchronize(s) == cudaSuccess;
  }
  if (!ok) {
    release_paged(h);
    return cuda_failed();
  }
  *out = h;
  return MOT_OK;
}

void mot_paged_destroy(mot_paged_t h) { release_paged(h); }

mot_status mot_paged_batch_create(mot_paged_t h, mot_paged_batch_t* out) {
  if (!out) return MOT_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (!h || !paged_device_ok(h)) return MOT_ERR_INVALID_ARGUMENT;
  mot_paged_batch* bt = new (std::nothrow) mot_paged_batch();
  if (!bt) return MOT_ERR_CUDA;
  bt->h = h;
  bt->t = paged_tables(h->cfg, h->ctas);
  bool ok = true;
  try {
    bt->host.resize(bt->t.words);
  } catch (...) {
    ok = false;
  }
  ok = ok && cudaMalloc(&bt->dev, bt->t.words * sizeof(int)) == cudaSuccess;
  if (!ok) {
    delete bt;
    return cuda_failed();
  }
  *out = bt;
  return MOT_OK;
}

void mot_paged_batch_destroy(mot_paged_batch_t bt) {
  if (!bt) return;
  cudaFree(bt->dev);
  delete bt;
}

mot_status mot_paged_batch_check(const mot_paged_config* cfg, int32_t batch, const int32_t* q_len,
                                 const int32_t* kv_len, const int32_t* visible, const int32_t* table,
                                 int32_t table_stride, int32_t n_pages) {
  const mot_status st = check_paged_config(cfg);
  if (st != MOT_OK) return st;
  if (!q_len || !kv_len || batch <= 0 || table_stride < 0 || n_pages <= 0) return MOT_ERR_INVALID_ARGUMENT;
  if (batch > cfg->max_batch) return MOT_ERR_UNSUPPORTED_SHAPE;
  // rows of the pool, as TMA coordinates count them
  if (static_cast<long long>(n_pages) * cfg->n_kv_heads * cfg->page_size > INT_MAX) return MOT_ERR_UNSUPPORTED_SHAPE;
  long long tokens = 0, entries = 0;
  for (int b = 0; b < batch; ++b) {
    if (q_len[b] < 0 || kv_len[b] < q_len[b]) return MOT_ERR_INVALID_ARGUMENT;
    if (visible && (visible[b] < 0 || visible[b] > kv_len[b])) return MOT_ERR_INVALID_ARGUMENT;
    if (kv_len[b] > cfg->max_positions) return MOT_ERR_UNSUPPORTED_SHAPE;
    const int used = (kv_len[b] + cfg->page_size - 1) / cfg->page_size;
    if (used > table_stride || (used > 0 && !table)) return MOT_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < used; ++i) {
      const int id = table[static_cast<size_t>(b) * table_stride + i];
      if (id < 0 || id >= n_pages) return MOT_ERR_INVALID_ARGUMENT;
    }
    tokens += q_len[b];
    entries += used;
  }
  return tokens > cfg->max_tokens || entries > cfg->max_pages ? MOT_ERR_UNSUPPORTED_SHAPE : MOT_OK;
}

mot_status mot_paged_batch_set(mot_paged_batch_t bt, int32_t batch, const int32_t* q_len, const int32_t* kv_len,
                               const int32_t* visible, const int32_t* table, int32_t table_stride, int32_t n_pages,
                               void* stream) {
  if (!bt) return MOT_ERR_INVALID_ARGUMENT;
  mot_paged* h = bt->h;
  const mot_paged_config& c = h->cfg;
  const mot_status cs = mot_paged_batch_check(&c, batch, q_len, kv_len, visible, table, table_stride, n_pages);
  if (cs != MOT_OK) return cs;
  const int shift = log2_of(c.page_size);
  long long tokens = 0, entries = 0;
  int kv_max = 0;
  for (int b = 0; b < batch; ++b) {
    tokens += q_len[b];
    entries += (kv_len[b] + c.page_size - 1) >> shift;
    kv_max = std::max(kv_max, kv_len[b]);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
  if (!paged_device_ok(h)) return MOT_ERR_INVALID_ARGUMENT;
  if (cudaStreamIsCapturing(st, &capturing) != cudaSuccess || capturing != cudaStreamCaptureStatusNone) {
    cudaGetLastError();
    return MOT_ERR_INVALID_ARGUMENT;
  }
  const PagedTables& t = bt->t;
  int n_units[2] = {0, 0};
  try {
    if (bt->stamp.size() < static_cast<size_t>(n_pages)) {
      bt->stamp.resize(n_pages, 0u);
      bt->times.resize(n_pages, 0);
    }
    std::vector<PagedTile> tiles[2];
    struct Seq {
      int q0, page0, past, vis;
    };
    std::vector<Seq> seqs(batch);
    bt->batch = 0;  // nothing is described until the copies below are enqueued
    ++bt->set_no;
    int* w = bt->host.data();
    int q0 = 0, e0 = 0;
    bool repeated = false;
    const int group = c.n_q_heads / c.n_kv_heads;
    long long mid = 0;
    for (int b = 0; b < batch; ++b)
      if (q_len[b] * group > kSmallRows && q_len[b] * group <= kSmallMaxRows) mid += c.n_kv_heads;
    const int few = small_rows(c.kv_dtype == MOT_PAGED_E4M3, mid);
    for (int b = 0; b < batch; ++b) {
      const int used = (kv_len[b] + c.page_size - 1) >> shift, past = kv_len[b] - q_len[b];
      const int* row = table + static_cast<size_t>(b) * table_stride;
      const int vis = visible ? visible[b] : 0;
      seqs[b] = Seq{q0, e0, past, vis};
      for (int i = 0; i < used; ++i) {
        const int id = row[i];
        if (bt->stamp[id] != bt->set_no) {
          bt->stamp[id] = bt->set_no;
          bt->times[id] = 1;
        } else {
          bt->times[id] = 2;
          repeated = true;
        }
        w[t.pages + e0 + i] = id;
        int* entry = w + t.entries + 4 * (e0 + i);
        entry[0] = id;
        entry[1] = b;
        entry[2] = i << shift;
        entry[3] = std::min(c.page_size, kv_len[b] - (i << shift));
      }
      for (int i = 0; i < q_len[b]; ++i) {
        const int pos = past + i;
        w[t.tok + 2 * (q0 + i)] = pos;
        w[t.tok + 2 * (q0 + i) + 1] = row[pos >> shift];
      }
      const int rows = q_len[b] * group, kind = rows <= few ? 0 : 1, step = kind ? kTileRows : kSmallRows;
      for (int r = 0; r < rows; r += step) {
        const int last = std::min(rows, r + step) - 1;
        tiles[kind].push_back(PagedTile{b, r, std::max(vis, past + last / group + 1)});
      }
      q0 += q_len[b];
      e0 += used;
    }
    w[t.n_entries] = e0;
    bt->repeated = repeated;
    bt->repeated_written = false;
    if (repeated)
      for (int b = 0; b < batch; ++b)
        if (q_len[b] > 0)
          for (int i = (kv_len[b] - q_len[b]) >> shift; i <= (kv_len[b] - 1) >> shift; ++i)
            bt->repeated_written |= bt->times[table[static_cast<size_t>(b) * table_stride + i]] > 1;
    for (int i = 0; i < 2; ++i) {
      std::fill(w + t.counters[i], w + t.counters[i] + h->ctas[i], 0);
      if (!plan_units(tiles[i], c.n_kv_heads, h->ctas[i], kCutRules[i], reinterpret_cast<PagedUnit*>(w + t.units[i]),
                      t.unit_cap[i], w + t.cta_unit0[i], &n_units[i]))
        return MOT_ERR_UNSUPPORTED_SHAPE;
      PagedUnit* units = reinterpret_cast<PagedUnit*>(w + t.units[i]);
      for (int k = 0; k < n_units[i]; ++k) {
        PagedUnit& un = units[k];
        const Seq& sq = seqs[un.seq];
        un.q0 = sq.q0;
        un.rows = q_len[un.seq] * group;
        un.past = sq.past;
        un.vis = sq.vis;
        un.page0 = sq.page0;
      }
    }
  } catch (...) {
    return MOT_ERR_CUDA;
  }
  const size_t pieces[][2] = {{0, t.head_words},
                              {t.pages, static_cast<size_t>(entries)},
                              {t.entries, static_cast<size_t>(4 * entries)},
                              {t.tok, static_cast<size_t>(2 * tokens)},
                              {t.units[0], static_cast<size_t>(n_units[0]) * (sizeof(PagedUnit) / 4)},
                              {t.units[1], static_cast<size_t>(n_units[1]) * (sizeof(PagedUnit) / 4)}};
  for (const auto& pc : pieces)
    if (pc[1] > 0 && cudaMemcpyAsync(bt->dev + pc[0], bt->host.data() + pc[0], pc[1] * sizeof(int), cudaMemcpyHostToDevice,
                                     st) != cudaSuccess)
      return cuda_failed();
  bt->batch = batch;
  bt->tokens = static_cast<int>(tokens);
  bt->entries = static_cast<int>(entries);
  bt->n_pages = n_pages;
  bt->kv_max = kv_max;
  bt->units[0] = n_units[0];
  bt->units[1] = n_units[1];
  return MOT_OK;
}

mot_status mot_paged_query_workspace(mot_paged_batch_t bt, size_t* workspace_bytes) {
  if (!bt || !workspace_bytes) return MOT_ERR_INVALID_ARGUMENT;
  // a cut makes at most two ranges, and there are fewer cuts than CTAs
  *workspace_bytes = (static_cast<size_t>(bt->h->ctas[0]) * 2 * kSmallSlot +
                      static_cast<size_t>(bt->h->ctas[1]) * 2 * kTileSlot) * sizeof(float);
  return MOT_OK;
}

mot_status mot_paged_append(mot_paged_t h, mot_paged_batch_t bt, const void* qkv, const mot_paged_pool* pool, void* q,
                            void* stream) {
  const mot_status cs = check_paged_call(h, bt, pool);
  if (cs != MOT_OK) return cs;
  if (bt->repeated_written) return MOT_ERR_INVALID_ARGUMENT;
  if (bt->tokens == 0) return MOT_OK;
  if (!qkv || !q || qkv == q) return MOT_ERR_INVALID_ARGUMENT;
  if (!aligned16(qkv) || !aligned16(q)) return MOT_ERR_ALIGNMENT;
  const mot_paged_config& c = h->cfg;
  PagedAppendParams p{};
  p.qkv = static_cast<const uint4*>(qkv);
  p.q = static_cast<uint4*>(q);
  p.pool = pool_view(pool);
  p.gains = h->gains;
  p.rope = h->rope;
  p.tok = reinterpret_cast<const int2*>(bt->dev + bt->t.tok);
  p.T = bt->tokens;
  p.Hq = c.n_q_heads;
  p.Hkv = c.n_kv_heads;
  p.page_shift = log2_of(c.page_size);
  p.page_mask = c.page_size - 1;
  p.eps = c.rms_eps;
  const int quads = (c.n_q_heads + 2 * c.n_kv_heads + 3) / 4;
  // Four heads a warp while that is one wave of warps (24 an SM); sixteen up to two waves (16 an SM); then a token.
  // us at 32/8 heads, e4m3, for 64 / 256 / 700 / 1300 / 2368 / 8192 tokens: 2.8 / 3.2 / 7.0 / 11.4 / 20.7 / 71,
  // 3.7 / 4.4 / 4.8 / 9.1 / 15.0 / 47 and 6.9 / 7.0 / 9.4 / 10.2 / 12.1 / 41.
  const long long t = p.T;
  const int mode = t * quads <= 24ll * h->num_sms ? 0 : t * ((quads + 3) / 4) <= 32ll * h->num_sms ? 1 : 2;
  const int strips = mode == 0 ? quads : mode == 1 ? (quads + 3) / 4 : 1;
  const int grid = static_cast<int>(std::min<long long>((t * strips + 7) / 8, 128ll * h->num_sms));
  const bool e4m3 = c.kv_dtype == MOT_PAGED_E4M3;
  auto kern = mode == 0   ? (e4m3 ? paged_append_kernel<true, 1, false> : paged_append_kernel<false, 1, false>)
              : mode == 1 ? (e4m3 ? paged_append_kernel<true, 4, false> : paged_append_kernel<false, 4, false>)
                          : (e4m3 ? paged_append_kernel<true, 4, true> : paged_append_kernel<false, 4, true>);
  return launch_pdl(kern, dim3(grid), dim3(256), 0, static_cast<cudaStream_t>(stream), p) == cudaSuccess ? MOT_OK
                                                                                                          : cuda_failed();
}

mot_status mot_paged_store(mot_paged_t h, mot_paged_batch_t bt, const void* k, const void* v, int32_t rows,
                           const mot_paged_pool* pool, void* stream) {
  const mot_status cs = check_paged_call(h, bt, pool);
  if (cs != MOT_OK) return cs;
  return paged_copy(h, bt, const_cast<void*>(k), const_cast<void*>(v), rows, pool, true, static_cast<cudaStream_t>(stream));
}

mot_status mot_paged_load(mot_paged_t h, mot_paged_batch_t bt, const mot_paged_pool* pool, void* k, void* v,
                          int32_t rows, void* stream) {
  const mot_status cs = check_paged_call(h, bt, pool);
  if (cs != MOT_OK) return cs;
  return paged_copy(h, bt, k, v, rows, pool, false, static_cast<cudaStream_t>(stream));
}

mot_status mot_paged_attend(mot_paged_t h, mot_paged_batch_t bt, const void* q, const mot_paged_pool* pool, void* o,
                            float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const mot_status cs = check_paged_call(h, bt, pool);
  if (cs != MOT_OK) return cs;
  if (bt->tokens == 0) return MOT_OK;
  if (!q || !o || q == o || !workspace) return MOT_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q, o, lse, workspace};
  for (const void* ptr : ptrs)
    if (ptr && !aligned16(ptr)) return MOT_ERR_ALIGNMENT;
  size_t need = 0;
  mot_paged_query_workspace(bt, &need);
  if (workspace_bytes < need) return MOT_ERR_WORKSPACE_TOO_SMALL;
  const mot_paged_config& c = h->cfg;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool e4m3 = c.kv_dtype == MOT_PAGED_E4M3;
  PagedSmallParams small{};
  PagedTileParams tp{};
  PagedAttnParams& p = tp.a;
  p.q = static_cast<const uint4*>(q);
  p.o = static_cast<uint4*>(o);
  p.lse = lse;
  p.pool = pool_view(pool);
  p.pages = bt->dev + bt->t.pages;
  p.Hq = c.n_q_heads;
  p.Hkv = c.n_kv_heads;
  p.group = c.n_q_heads / c.n_kv_heads;
  p.page_shift = log2_of(c.page_size);
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(128.0));
  p.status = h->status;
  cudaError_t e = cudaSuccess;
  for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
    if (bt->units[i] == 0) continue;
    p.units = reinterpret_cast<const PagedUnit*>(bt->dev + bt->t.units[i]);
    p.cta_unit0 = bt->dev + bt->t.cta_unit0[i];
    p.counters = bt->dev + bt->t.counters[i];
    p.part = static_cast<float*>(workspace) + (i ? static_cast<size_t>(h->ctas[0]) * 2 * kSmallSlot : 0);
    const uint64_t rows = static_cast<uint64_t>(pool->n_pages) * c.n_kv_heads * c.page_size;
    CUtensorMap &km = i ? tp.k_map : small.k_map, &vm = i ? tp.v_map : small.v_map;
    const uint32_t box = i ? c.page_size : std::min(c.page_size, e4m3 ? SmallShape<true>::kKeys : SmallShape<false>::kKeys);
    if (e4m3 ? !map_bytes(&km, pool->k, rows, box, i == 0) || !map_bytes(&vm, pool->v, rows, box, i == 0)
             : !map2d(&km, pool->k, true, 128, rows, 128, box) || !map2d(&vm, pool->v, true, 128, rows, 128, box))
      return MOT_ERR_CUDA;
    if (i == 0) {
      small.a = p;
      e = launch_pdl(e4m3 ? paged_attn_small_kernel<true> : paged_attn_small_kernel<false>, dim3(h->ctas[0]),
                     dim3(e4m3 ? SmallShape<true>::kThreads : SmallShape<false>::kThreads),
                     e4m3 ? SmallShape<true>::kBytes : SmallShape<false>::kBytes, st, small);
    } else {
      // a tile's 128 rows are whole tokens where the group divides 128: one box
      tp.q_tma = 128 % p.group == 0;
      const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(c.n_q_heads), static_cast<cuuint64_t>(bt->tokens)};
      const cuuint64_t strides[2] = {256, static_cast<cuuint64_t>(c.n_q_heads) * 256};
      const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.group), static_cast<cuuint32_t>(128 / p.group)};
      if (tp.q_tma && !encode(&tp.q_map, q, true, 3, dims, strides, box)) return MOT_ERR_CUDA;
      e = launch_pdl(e4m3 ? paged_attn_tile_kernel<true> : paged_attn_tile_kernel<false>, dim3(h->ctas[1]),
                     dim3(kTileThreads), TileSmem::bytes(e4m3), st, tp);
    }
  }
  return e == cudaSuccess ? MOT_OK : cuda_failed();
}

mot_status mot_dev_paged_plan(int32_t kind, const int32_t* tiles, int32_t n_tiles, int32_t heads, int32_t ctas,
                              int32_t* units, int32_t unit_cap, int32_t* cta_unit0, int32_t* n_units) {
  if (kind < 0 || kind > 1 || (n_tiles > 0 && !tiles) || n_tiles < 0 || heads <= 0 || ctas <= 0 || !units || !cta_unit0 || !n_units)
    return MOT_ERR_INVALID_ARGUMENT;
  try {
    std::vector<PagedTile> tl;
    for (int i = 0; i < n_tiles; ++i) tl.push_back(PagedTile{tiles[3 * i], tiles[3 * i + 1], tiles[3 * i + 2]});
    if (!plan_units(tl, heads, ctas, kCutRules[kind], reinterpret_cast<PagedUnit*>(units), unit_cap, cta_unit0, n_units))
      return MOT_ERR_UNSUPPORTED_SHAPE;
  } catch (...) {
    return MOT_ERR_CUDA;
  }
  return MOT_OK;
}

mot_status mot_paged_get_device_status(mot_paged_t h, void* stream) {
  if (!h || !paged_device_ok(h)) return MOT_ERR_INVALID_ARGUMENT;
  int v = 0;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return cuda_failed();
  if (cudaMemcpy(&v, h->status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return cuda_failed();
  if (cudaMemset(h->status, 0, sizeof(int)) != cudaSuccess) return cuda_failed();
  return (v & DEV_ERR_TIMEOUT) ? MOT_ERR_TIMEOUT : MOT_OK;
}

}  // extern "C"
