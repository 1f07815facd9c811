/*
 * lora_layer.h -- what stands before and behind the operators of lora_base.h
 * in an attention layer of a served model: the norm whose output the 8-bit
 * base product and the adapters read, the cache that the rotated keys and the
 * values go to, and the attention that reads it.
 *
 *   x, residual --lora_norm_apply--> y, q, s --lora_base_product, lora_apply, lora_rotary_apply--> q, k, v heads
 *   k, v --lora_cache_write--> cache;   q, cache --lora_attention_apply--> heads of the output projection
 *
 * Memory, streams and errors as in lora_base.h: every pointer is a DEVICE
 * pointer unless its comment says host; all buffers are the caller's; the
 * library allocates nothing and keeps nothing between calls but the device's
 * compute-unit count and the kernels' LDS limit; every call is asynchronous on
 * `stream` (of the current device) and can be captured in a graph.  What the
 * host can see to be wrong returns a status and launches nothing.  The same
 * inputs give the same bits.
 */
#ifndef RANK_SGMV_BGMV_LORA_LAYER_H
#define RANK_SGMV_BGMV_LORA_LAYER_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "lora_base.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LORA_MAX_NORM_D 65536
#define LORA_MAX_CACHE_HEAD_DIM 256
#define LORA_MAX_CACHE_HEADS 65535
#define LORA_MAX_TREE 64            /* drafted tokens of a sequence */
#define LORA_MAX_CONTEXT (1 << 30)  /* keys of a sequence */

/* Root-mean-square norm. */
typedef struct {
  const float *weight; /* [d] */
  double eps;          /* >= 0 */
  int32_t d;           /* 1 .. LORA_MAX_NORM_D */
} lora_norm;

/* The norm of a row, with what a layer does around it:
 *
 *     h = x[t] + residual[t], rounded to dtype, kept in total[t]   (no residual: h = x[t])
 *     y[t][c] = h[c] * weight[c] / sqrt(mean_c h[c]^2 + eps), rounded to dtype
 *     q[t], scale[t] = lora_quantize_rows of y[t] as it was rounded
 *
 * The mean and y are computed in float64, so that each value is its formula's
 * rounded once (through float32 on its way to bfloat16) and q depends on x
 * alone; a row's bits do not depend on the rows it is in a batch with.  A
 * row of zeros with eps = 0 has y = NaN.
 *   x, residual, total, y  [n_rows][ld] dtype, ld >= d
 *   q                      [n_rows][ldq] int8, scale [n_rows] float32
 * residual may be NULL, then total must be; total may be NULL; y or q may be
 * NULL, not both; scale is NULL where q is.  total may be x or residual
 * itself, and y x itself (the same pointer and row stride); nothing else that
 * is written may overlap anything.  n_rows == 0 launches nothing.
 * LORA_EINVAL: NULL, a bad dtype, pointers not aligned to their element,
 * overlap, eps negative or not finite; LORA_ESHAPE: n_rows < 0, d < 1, ld < d;
 * LORA_EUNSUPPORTED: d > LORA_MAX_NORM_D. */
lora_status lora_norm_apply(const lora_norm *norm, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                            void *total, int64_t ldt, void *y, int64_t ldy, int8_t *q, int64_t ldq, float *scale,
                            int32_t n_rows, lora_dtype dtype, hipStream_t stream);

/* A cache of keys and values in 8 bits, in pages of page_size tokens:
 *
 *     k, v              int8 [n_pages][n_heads][page_size][pitch], pitch = lora_cache_pitch(head_dim)
 *     k_scale, v_scale  float32 [n_pages][n_heads][page_size]
 *
 * where a page is contiguous and pages lie k_page, v_page bytes and
 * k_scale_page, v_scale_page floats apart (keys and values of a page, or of
 * several layers, may lie side by side).  Value i of head h at slot a of page
 * p is k * k_scale there.  A slot of the whole cache is p * page_size + a.
 *   page_size  a power of two, 16 .. 1024
 *   k, v and the scales 16-byte aligned, as are the distances of pages */
typedef struct {
  int8_t *k, *v;
  float *k_scale, *v_scale;
  int64_t k_page, v_page;             /* bytes */
  int64_t k_scale_page, v_scale_page; /* floats */
  int32_t n_pages, n_heads, page_size;
  int32_t head_dim; /* 1 .. LORA_MAX_CACHE_HEAD_DIM */
} lora_cache;

/* Bytes of a row of the cache: head_dim rounded up to 16 (host only); 0 for a bad head_dim. */
int32_t lora_cache_pitch(int32_t head_dim);

/* Heads of tokens: value i of head h of token t is at data + t * token + h * head + i (element strides, not negative). */
typedef struct {
  void *data;
  int64_t token, head;
} lora_heads;

/* Writes n_tokens tokens' keys and values (dtype, n_heads heads of head_dim)
 * to their slots, each head quantised as a row of lora_quantize_rows: a head
 * that holds an infinity or NaN gets scale NaN and zeros, one whose largest
 * value is 2^64 or more as well (attention weighs values by their scales).
 * Bytes between head_dim and the pitch become zeros.
 *   slots  [n_tokens] int32.  A token whose slot is negative, or not in the
 *          cache, is skipped.  Slots of a call must differ: of a slot named
 *          twice the values and scales may come from either token.
 * n_tokens == 0 launches nothing.  LORA_EINVAL: NULL, a bad dtype, alignment,
 * overlap; LORA_ESHAPE: sizes and strides that do not fit what is said above;
 * LORA_EUNSUPPORTED: head_dim or n_heads above their limits. */
lora_status lora_cache_write(const lora_cache *cache, const int32_t *slots, int32_t n_tokens, const lora_heads *k,
                             const lora_heads *v, lora_dtype dtype, hipStream_t stream);

/* Reads slots back: k[t], v[t] = the values times their scale, rounded to
 * dtype (through float32 on its way to bfloat16).  Tokens of a slot that is negative or not in the cache are left as
 * they were.  Errors as above; k and v must keep their values apart. */
lora_status lora_cache_read(const lora_cache *cache, const int32_t *slots, int32_t n_tokens, const lora_heads *k,
                            const lora_heads *v, lora_dtype dtype, hipStream_t stream);

/* Attention of one kind of layer. */
typedef struct {
  int32_t n_heads;  /* query heads, a multiple of the cache's: query head h reads cache head h / (n_heads / cache heads) */
  int32_t window;   /* keys that a query sees, its own the last; 0: all before it */
  int32_t sinks;    /* first keys of a sequence that stay visible beyond the window */
  float scale;      /* of the scores */
  lora_dtype dtype; /* of queries and outputs */
} lora_attention;

/* The sequences of a step.  Sequence s has lens[s] keys in the cache, its page
 * i at pages[s * ld_pages + i], and its last n = q_off[s+1] - q_off[s] tokens
 * are queries, rows q_off[s] .. q_off[s+1] - 1 of the batch (their keys are
 * in the cache already).  Query i stands at p = lens[s] - n + i and sees key j if
 *
 *     j <= p  and  (window == 0  or  p - j < window  or  j < sinks)
 *
 * With `tree` the n queries are drafted tokens, and bit b of tree[row] says
 * whether that query sees the drafted token b (its own bit too: a token that
 * is to see itself sets it).  It stands at p = lens[s] - n + (set bits below
 * its own place), and sees keys j < lens[s] - n as above; the window does not
 * hide drafted tokens.
 *
 * Pages that no query sees are not looked up and may be anything, and so may
 * slots of other pages that none sees (behind a sequence's last key, say; they
 * need never have been written).  Keys of a page outside 0 .. n_pages - 1 are
 * not seen.  A key that has NaN, an infinity or a negative number for a scale
 * makes the outputs of its head NaN that see it.  A query that sees nothing gets
 * zeros; rows that belong to no sequence are left as they were. */
typedef struct {
  int32_t n_tokens, n_seqs;
  int32_t max_q;         /* no sequence has more queries; with `tree` at most LORA_MAX_TREE */
  int32_t max_pages;     /* pages of a sequence; max_pages * page_size <= LORA_MAX_CONTEXT */
  const int32_t *q_off;  /* [n_seqs + 1] */
  const int32_t *lens;   /* [n_seqs] */
  const int32_t *pages;  /* [n_seqs][ld_pages] */
  int64_t ld_pages;      /* >= max_pages */
  const uint64_t *tree;  /* [n_tokens], or NULL */
} lora_attention_batch;

/* Bytes of a plan and of the workspace of lora_attention_apply (host only); 0 for invalid arguments. */
size_t lora_attention_plan_size(const lora_attention *attention, const lora_cache *cache,
                                const lora_attention_batch *batch);
size_t lora_attention_workspace_size(const lora_attention *attention, const lora_cache *cache,
                                     const lora_attention_batch *batch);

/* Cuts a step's work into pieces on the device: which rows read which keys,
 * long sequences in several pieces.  It reads q_off and lens only, so one plan
 * serves every layer of a step that has the same window, sinks and head
 * counts.  A sequence whose offsets are not within 0 .. n_tokens and
 * ascending, that has more than max_q queries or whose length is not within
 * 0 .. max_pages * page_size, is left out and counted
 * (lora_read_device_errors); a sequence whose length is below its number of
 * queries is not: queries before position 0 see nothing.
 * LORA_EINVAL: NULL or alignment (plan: 16 bytes); LORA_ESHAPE: sizes;
 * LORA_EWORKSPACE: a small plan; LORA_EUNSUPPORTED: above the limits. */
lora_status lora_attention_plan(const lora_attention *attention, const lora_cache *cache,
                                const lora_attention_batch *batch, void *plan, size_t plan_bytes, hipStream_t stream);

/* out = softmax(scale * q k^T) v over the keys that each query sees.  Scores,
 * sums and outputs are float32, the weights that meet the values are rounded
 * to 11 bits (dtype bfloat16) or 22 (float32), the output once to dtype.
 * (With dtype bfloat16, rows that are computed many at a time meet keys and
 * values that are rounded to 11 bits once their scales are multiplied in.)
 * A key keeps those bits while its weight times its value's scale is above 2^-13
 * (float32: 2^-12) of the row's largest such product, and is off by no more than
 * 2^-24 (2^-34) of that below.  Scales below 2^-60 lose bits too: of values, an
 * output is then off by 2^-85 more and by 2^-92 for each key that it sees; of keys
 * (dtype bfloat16), a score by 2^-85 scale sum |q|.
 *   q, out  heads of the batch's rows: n_heads of head_dim values.  out may be
 *           q itself (the same strides), or memory that does not meet it
 *   plan    of lora_attention_plan for this attention and batch, and a cache of
 *           these sizes.  On a plan made for other sizes (heads, head_dim, dtype,
 *           window, sinks, n_tokens, n_seqs, max_q, keys of max_pages, tree or
 *           none) nothing is written and its error word counts the call; one made
 *           from other contents of q_off or lens cannot be told from the right one:
 *           after they change, plan anew
 *   ws      16-byte aligned, written before it is read; calls that may overlap
 *           in time need one each (a plan may be shared)
 * n_tokens == 0 launches nothing.  Errors as above. */
lora_status lora_attention_apply(const lora_attention *attention, const lora_cache *cache,
                                 const lora_attention_batch *batch, const void *plan, size_t plan_bytes,
                                 const lora_heads *q, const lora_heads *out, void *ws, size_t ws_bytes,
                                 hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RANK_SGMV_BGMV_LORA_LAYER_H */
