/*
 * mot_paged.h -- C ABI of the paged prefix-KV cache on B200 (sm_100a).
 *
 *   "SenseNova-U1" (DiffSynth-Studio docs), architecture note: the prompt is
 *     encoded once into past_key_values, and at every denoise step the image
 *     tokens attend to that cache.
 *   "Setup notes" (LoRA trainer docs), "Why bf16 base on CPU + tower
 *     offload?": the static prefix-KV caches of all samples are kept (about
 *     59 MB per sample), in bf16.
 *
 * mot_attn.h's layer takes the cache of one call as a dense bf16 tensor. Here
 * the keys and values of many requests of different lengths live in one pool
 * of fixed-size pages, in bf16 or in 8 bits, and prompts may be encoded in
 * chunks and answered token by token: the serving form of the same cache.
 *   "SenseNova-U1.5" (vLLM-Omni recipe): text is decoded over a paged K/V cache,
 *     under a captured CUDA graph. The recipe gives no layout; pages, batches,
 *     8-bit rows and masks below are this library's own.
 *
 * append takes the projections as they are, before norm and rotation. The
 * attention layer's calls do not give those (its QKV GEMM norms and rotates),
 * and none takes a pool: a caller brings the projections, and goes through store
 * and load between a pool and mot_attn_prefix_forward or mot_attn_forward.
 *
 * Pool of one layer: n_pages pages of page_size rows,
 *   k, v              [n_pages, Hkv, page_size, 128]   bf16 or e4m3
 *   k_scale, v_scale  [n_pages, Hkv, page_size]        e8m0 (e4m3 pools only)
 * The e4m3 pool stands for payload * 2^(scale - 127): the scale of a row (one
 * token and head) is 2^e, e the smallest integer with amax <= 448 * 2^e and
 * e >= -64, the payload x * 2^-e rounded once to nearest. A row that holds an
 * infinity or a NaN is stored as NaN (scale byte 255). A power of two costs
 * no precision in a floating-point payload and makes every stored value
 * exact in bf16.
 *
 * A batch object describes a ragged set of sequences: sequence b holds
 * kv_len[b] tokens, listed in its row of the page table (token j sits in row
 * j % page_size of page table[b][j / page_size]); its last q_len[b] tokens are
 * the chunk that a call adds or asks for. Packed token tensors hold the
 * chunks one after another: T = sum_b q_len[b] rows, sequence 0 first. The
 * position of a token is its index in the sequence.
 *
 * Conventions as mot_attn.h (dense row-major tensors, 16-byte alignment,
 * validation on the host before anything is enqueued), and:
 *   - Every call must be made with the handle's device current
 *     (MOT_ERR_INVALID_ARGUMENT otherwise).
 *   - A batch object is used by one stream at a time: mot_paged_attend keeps
 *     arrival counters in it, and mot_paged_batch_set rewrites its device
 *     tables in stream order. The same holds for a workspace.
 *   - append, store, load and attend may be captured into a CUDA graph; a
 *     captured call may be replayed after mot_paged_batch_set has given the
 *     batch other kv_len, visible or tables, as long as batch and q_len are
 *     those of the capture, n_pages and the longest kv_len are within the
 *     captured pool's pages and dense rows, and no page appears twice that the
 *     captured call refuses to find twice (nothing checks a replay).
 *     mot_paged_batch_set itself is refused on a capturing stream.
 *   - Outputs must not overlap inputs or one another.
 *   - After MOT_ERR_TIMEOUT from mot_paged_get_device_status set the batch again
 *     before it is used.
 */
#ifndef MOT_PAGED_H
#define MOT_PAGED_H

#include <stddef.h>
#include <stdint.h>

#include "mot_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mot_paged* mot_paged_t;             /* opaque handle */
typedef struct mot_paged_batch* mot_paged_batch_t; /* opaque batch  */

typedef enum { MOT_PAGED_BF16 = 0, MOT_PAGED_E4M3 = 1 } mot_paged_dtype;

/* Supported: head_dim == 128, n_q_heads % n_kv_heads == 0, at most 64 query
 * heads per KV head, page_size in {16, 32, 64, 128}. */
typedef struct {
  int32_t n_q_heads;     /* Hq (32)                                          */
  int32_t n_kv_heads;    /* Hkv (8)                                          */
  int32_t head_dim;      /* 128                                              */
  int32_t page_size;     /* rows of a page                                   */
  int32_t kv_dtype;      /* mot_paged_dtype                                  */
  float rms_eps;         /* QK-RMSNorm epsilon (1e-6)                        */
  double rope_theta;     /* RoPE base (1e6)                                  */
  int32_t max_positions; /* largest kv_len                                   */
  int32_t max_batch;     /* largest number of sequences of a batch (<= 4096) */
  int32_t max_tokens;    /* largest T                                        */
  int32_t max_pages;     /* largest number of table entries in use           */
} mot_paged_config;

/* Norm gains, bf16 [128] in memory of the current device; copied at create. */
typedef struct {
  const void *q_norm, *k_norm;
} mot_paged_weights;

/* One layer's pool (device pointers); the scales are NULL for a bf16 pool. */
typedef struct {
  void *k, *v;
  void *k_scale, *v_scale;
  int32_t n_pages;
} mot_paged_pool;

/* Create: validates, copies the gains to f32 and builds the RoPE table of
 * max_positions rows (angles in f64, cos and sin rounded to f32). */
mot_status mot_paged_create(const mot_paged_config* cfg, const mot_paged_weights* weights, void* stream,
                            mot_paged_t* out);

/* A batch object with device tables for the handle's maxima. The handle must
 * outlive it. */
mot_status mot_paged_batch_create(mot_paged_t h, mot_paged_batch_t* out);

/* Describe the sequences. All arguments are host memory, read before return.
 *   q_len    int32 [batch], 0 <= q_len[b] <= kv_len[b]
 *   kv_len   int32 [batch], 0 <= kv_len[b] <= max_positions; the chunk's own
 *            tokens included
 *   visible  int32 [batch] or NULL (all 0), 0 <= visible[b] <= kv_len[b]: every
 *            query of b sees the keys j < visible[b] besides those up to its
 *            own position (0: causal; kv_len: bidirectional, as image tokens
 *            attend; between: a bidirectional prefix)
 *   table    int32 [batch, table_stride] page numbers; entry [b][i] is read for
 *            i < ceil(kv_len[b] / page_size) and must be in [0, n_pages)
 * A page may appear more than once in the table (sequences that share a
 * prompt); mot_paged_append refuses a batch in which a page that a chunk is
 * written to appears twice, mot_paged_store one in which any page does.
 * Enqueues its copies on `stream`, from pageable host memory of the batch: for large
 * tables the driver may make the host wait for earlier work of the stream. Measured
 * behind a busy stream it returned after 0.1 to 0.17 ms, planning included, for 7 to
 * 16000 pages in use, long before the stream was done. */
mot_status mot_paged_batch_set(mot_paged_batch_t bt, int32_t batch, const int32_t* q_len, const int32_t* kv_len,
                               const int32_t* visible, const int32_t* table, int32_t table_stride, int32_t n_pages,
                               void* stream);

/* What mot_paged_batch_set refuses in its arguments. Host-only; no CUDA calls. */
mot_status mot_paged_batch_check(const mot_paged_config* cfg, int32_t batch, const int32_t* q_len,
                                 const int32_t* kv_len, const int32_t* visible, const int32_t* table,
                                 int32_t table_stride, int32_t n_pages);

/* Device workspace bytes mot_paged_attend needs for any batch of this object. */
mot_status mot_paged_query_workspace(mot_paged_batch_t bt, size_t* workspace_bytes);

/* Norm, rotate and cache the chunk:
 *   qkv  device bf16 [T, (Hq + 2 Hkv) * 128]: the projections of the chunk, q heads,
 *        then k heads, then v heads
 *   q    device bf16 [T, Hq, 128]: RoPE_p(RMSNorm(q_h) * q_norm), one rounding
 * and into the pages, at each token's row, RoPE_p(RMSNorm(k_h) * k_norm) and
 * v_h. Statistics and rotation are f32 (a head whose sum of squares passes f32, from
 * magnitudes of about 2^60 on, comes out as zeros); k goes to the pages with one
 * rounding.
 * The rest of the pool is left as it was. */
mot_status mot_paged_append(mot_paged_t h, mot_paged_batch_t bt, const void* qkv, const mot_paged_pool* pool, void* q,
                            void* stream);

/* Dense cache -> pages: rows [0, kv_len[b]) of every sequence.
 *   k, v  device bf16 [batch, Hkv, rows, 128], keys normed and rotated: what
 *         mot_attn_prefix_forward writes. rows >= every kv_len. */
mot_status mot_paged_store(mot_paged_t h, mot_paged_batch_t bt, const void* k, const void* v, int32_t rows,
                           const mot_paged_pool* pool, void* stream);

/* Pages -> dense cache, the reverse: rows [0, kv_len[b]) of k, v device bf16
 * [batch, Hkv, rows, 128] are written (the cache mot_attn_forward takes), the
 * rows behind them left as they were. e4m3 rows come back exactly. */
mot_status mot_paged_load(mot_paged_t h, mot_paged_batch_t bt, const mot_paged_pool* pool, void* k, void* v,
                          int32_t rows, void* stream);

/* Attention of the chunk over the pages (its own rows already in them):
 *   o_i = softmax over j < limit_i of (q_i K_j / sqrt(128)) V_j,
 *   limit_i = max(visible, p_i + 1), p_i = kv_len - q_len + i; query head h reads KV
 *   head h / (Hq / Hkv).
 *   q    device bf16 [T, Hq, 128]
 *   o    device bf16 [T, Hq, 128]
 *   lse  device f32 [T, Hq] or NULL: natural log of the sum of exp(scores)
 *   workspace  device, workspace_bytes from mot_paged_query_workspace
 * Rows of a page behind kv_len are never used, whatever they hold. An infinity
 * or NaN among the cached rows reaches the outputs of the queries that see it
 * (as NaN or infinity), and of no others; a finite row that a query does not see,
 * whatever its size, changes at most which of the roundings below its weights take.
 *
 * Scores, statistics and sums are f32 and a result does not depend on timing (fixed
 * order of every sum). In fewer bits, each rounding relative to what is rounded:
 *   - weights where they meet the values in the tensor cores, but not in their own
 *     sum. bf16 pools: 16 bits (bf16 hi + lo) in chunks of few query rows, else 8
 *     (bf16; the output's error grows from 1.7e-3 to 2.3e-3 of its norm). e4m3
 *     pools: 11 bits (f16), or 8 in a range of keys of a chunk of many rows whose
 *     value scales span more than 2^7, key scales more than 2^14, or key scales
 *     reach above 2^4. Over rows that append and store write, with values of 2^-56
 *     and more, f16 weights add at most kv_len * 2^-24 of the largest |value| that
 *     the query sees;
 *   - e4m3 pools: queries in f16 relative to their row's largest magnitude (exact
 *     down to 2^-17 of it, off by at most 2^-25 of it below), or as they are in the
 *     ranges just named.
 * A weight is at most 2^8 before its sum divides it: where kv_len * 2^8 * |value|
 * passes the f32 range, so may a sum. */
mot_status mot_paged_attend(mot_paged_t h, mot_paged_batch_t bt, const void* q, const mot_paged_pool* pool, void* o,
                            float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* Synchronise `stream`, return and clear the latched device status. */
mot_status mot_paged_get_device_status(mot_paged_t h, void* stream);

/* Free. NULL is ignored; destroy batches before their handle. */
void mot_paged_batch_destroy(mot_paged_batch_t bt);
void mot_paged_destroy(mot_paged_t h);

#ifdef __cplusplus
}
#endif

#endif /* MOT_PAGED_H */
