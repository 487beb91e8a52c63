/*
 * tq2_attn.h -- C ABI of libtq2's paged key/value cache: appending new tokens
 * (with normalisation and rotation on the way) and attention over the cache.
 *
 * The conventions of tq2.h hold: device pointers of the caller, nothing
 * allocated or synchronised, work only enqueued on `stream`, negative
 * tq2_status values for errors and nothing enqueued with them.
 *
 * Cache.  Keys and values lie in pages of `page` tokens.  Element (p, h, t, i)
 * of a cache, page p, key head h, token t of the page, component i, is at
 * p * page_stride + h * head_stride + t * token_stride + i (strides in
 * elements), so both [pages, heads, page, dim] and [pages, page, heads, dim]
 * are passed as they are.  Place n of sequence b is token n % page of page
 * table[b * table_stride + n / page].  Sequence b holds kv_len[b] tokens, the
 * new ones of the present call included.
 * 8-bit caches hold e4m3 codes of value / scale with one f32 scale per key
 * head.  tq2_paged_attention multiplies by any finite scale, also zero (the
 * codes count as zeros) and negative ones; tq2_kv_append divides by it.
 *
 * New tokens.  cu_q[b] .. cu_q[b + 1] are the rows of q, k, v and out that
 * belong to sequence b, in order; they are the last tokens of the sequence.
 * cu_q == NULL means one new token for each sequence (tokens == batch).
 *
 * What device arrays hold cannot be checked before the launch.  The kernels
 * check it themselves: a place outside the table's columns, or whose table
 * entry is not a page of the cache, is not written by tq2_kv_append and takes
 * no part in tq2_paged_attention.  Rows of q that no sequence owns are left
 * alone.  cu_q must not decrease.
 */
#ifndef TQ2_ATTN_H
#define TQ2_ATTN_H

#include "tq2.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
#define TQ2_TYPE_F32 0
#define TQ2_TYPE_F16 1
#define TQ2_TYPE_BF16 2
#define TQ2_TYPE_E4M3 3

#define TQ2_ATTN_MAX_HEAD_DIM 256
#define TQ2_ATTN_MAX_BATCH 65535
#define TQ2_ATTN_MAX_HEADS 1024

/* The cache and the new tokens' place in it.  All fields are 8 bytes wide. */
typedef struct tq2_paged_cache {
  void* k;
  void* v;
  const float* k_scale;      /* f32 [kv_heads]: 8-bit caches only, else NULL */
  const float* v_scale;
  const int32_t* table;      /* [batch, table_cols], rows table_stride apart; NULL if it has no columns */
  const int32_t* kv_len;     /* [batch] */
  const int32_t* cu_q;       /* [batch + 1] or NULL */
  int64_t batch;
  int64_t tokens;            /* rows of q (new tokens of all sequences) */
  int64_t pages;             /* pages of the cache */
  int64_t page;              /* tokens of a page: a power of two, 16 .. 2^20 */
  int64_t table_cols;
  int64_t table_stride;
  int64_t kv_heads;
  int64_t q_heads;           /* a multiple of kv_heads */
  int64_t head_dim;          /* 64, 96, 128, 192 or 256 */
  int64_t act_type;          /* of q, k, v, out: F32, F16 or BF16 */
  int64_t cache_type;        /* E4M3; or F16 with F32 and F16, BF16 with BF16 */
  int64_t k_page_stride, k_head_stride, k_token_stride;
  int64_t v_page_stride, v_head_stride, v_token_stride;
} tq2_paged_cache;

typedef struct tq2_kv_append_args {
  tq2_paged_cache cache;
  const void* q;             /* [tokens, q_heads, head_dim], or NULL: k and v only */
  const void* k;             /* [tokens, kv_heads, head_dim] */
  const void* v;
  void* q_out;               /* may be q itself (same strides), k and v other columns of its array */
  int64_t q_token_stride, q_head_stride;
  int64_t k_token_stride, k_head_stride;
  int64_t v_token_stride, v_head_stride;
  int64_t q_out_token_stride, q_out_head_stride;
  const double* freqs;       /* f64 [rot / 2], needed if rot > 0 */
  const int32_t* positions;  /* [axes, tokens], or NULL: the place in the cache */
  int64_t rot;               /* leading components that are rotated: a multiple of 8, 0 .. head_dim */
  int64_t axes;              /* 1 .. 3; 1 without positions */
  int64_t section[3];        /* angles of each axis, summing to rot / 2 */
  int64_t interleaved;       /* pairs (2i, 2i + 1) instead of (i, i + rot / 2) */
  const float* q_norm;       /* f32 [head_dim] or NULL: no normalisation of q */
  const float* k_norm;
  double eps;
} tq2_kv_append_args;

/* For each new token: q and k are normalised (x / sqrt(mean x^2 + eps) * norm,
 * if a weight is given) and pair i of them is turned by the angle
 * position * freqs[i] (computed in f64; the position is that of the axis whose
 * section i lies in); q goes to q_out, k and v to their place in the cache,
 * rounded once (e4m3: value / scale, clamped to +-448).
 * Activations and caches: 16-byte aligned, strides multiples of 16 bytes.
 * tokens == 0 or batch == 0 is a no-op.  Errors: INVALID (null pointer, size out of range,
 * a pair of types or head_dim that is not listed, sections that do not sum to
 * rot / 2), SHAPE (page not a power of two, rot not a multiple of 8, q_heads
 * not a multiple of kv_heads), ALIGN, ALIAS (q_out or a cache overlaps another
 * operand, rows of q_out overlap each other or neighbours along an axis of a
 * cache do), DEVICE, LAUNCH. */
int tq2_kv_append(const tq2_kv_append_args* args, void* stream);

typedef struct tq2_paged_attention_args {
  tq2_paged_cache cache;
  const void* q;             /* [tokens, q_heads, head_dim] */
  void* out;                 /* the same shape; may be q itself (same strides) */
  int64_t q_token_stride, q_head_stride;
  int64_t out_token_stride, out_head_stride;
  int64_t max_q;             /* most new tokens of a sequence, most tokens of one: the launch is */
  int64_t max_kv;            /* shaped for them; larger ones in cu_q and kv_len are still done, and */
                             /* far too large values cost time (blocks that find no work) */
  int64_t window;            /* a token sees itself and window - 1 before it; 0: all before it */
  double scale;              /* of the scores, usually 1 / sqrt(head_dim): above 0, below 2^127 */
  void* workspace;           /* NULL if none is needed */
  int64_t workspace_bytes;
} tq2_paged_attention_args;

/* Bytes of workspace that tq2_paged_attention needs for these sizes, types,
 * max_q, max_kv and window (no pointer but whether cu_q is NULL is looked at),
 * or 0; also 0 for sizes that it refuses.  Pure host function. */
size_t tq2_paged_attention_workspace_bytes(const tq2_paged_attention_args* args);

/* out = softmax(scale * q K^T + mask) V for each new token over the tokens of
 * its sequence up to itself, query head h reading key head
 * h / (q_heads / kv_heads).  Rows that see no token give zeros.
 * Keys and values of places that a row does not see do not reach it, whatever
 * they hold.
 * Accuracy: f32 activations as two binary16 parts, products and sums f32,
 * about 1e-6 of sum_j p_j |v_j|; 16-bit activations enter the products as they
 * are and the probabilities are rounded to the cache's type (binary16 for
 * e4m3), half a step each.
 * Activations, caches and workspace: 16-byte aligned, strides multiples of 16
 * bytes; 16 tokens of a page lie within 2^31 bytes; tokens * q_heads is below
 * 2^31 - 4096.  The workspace's content
 * needs no preparation and means nothing afterwards.
 * tokens == 0 or batch == 0 is a no-op.  Errors: INVALID (null pointer, size out of range, a
 * workspace that is too small, types or head_dim not listed), SHAPE, ALIGN,
 * ALIAS (out overlaps a cache, the workspace or a part of q, or rows of out
 * overlap each other), DEVICE, LAUNCH. */
int tq2_paged_attention(const tq2_paged_attention_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ2_ATTN_H */
