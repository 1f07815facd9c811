/*
 * lora_base.h -- the operators on both sides of lora_apply in an adapted
 * layer of a served model: the 8-bit base product whose output the adapters'
 * products are added to, the quantisation of rows that it needs, and the
 * rotary positions of the query and key heads that follow.
 *
 *   x --lora_quantize_rows--> q, s --lora_base_product--> y --lora_apply--> y --lora_rotary_apply--> heads
 *     \------------- lora_base_apply -------------------/
 *
 * The base weights are shared by every request of a batch, whatever adapters
 * they name, so they are the bytes that a decode step reads besides the
 * adapters; in 8 bits they are half of what bf16 needs.
 *
 * Memory, streams and errors as in lora.h: every pointer is a DEVICE pointer
 * unless its comment says host; all buffers are the caller's; the library
 * allocates nothing, keeps nothing between calls but the device's
 * compute-unit count and the kernels' LDS limit, and every call is
 * asynchronous on `stream` (which must belong to the current device) and can
 * be captured in a graph.  What the host can see to be wrong returns a status
 * and launches nothing.  Rows and columns outside the sizes of a call are
 * never written, and no result depends on what they hold.  Results do not
 * depend on the launch either: the same inputs give the same bits, and a row
 * the same ones whatever rows it is in a batch with.
 */
#ifndef RANK_SGMV_BGMV_LORA_BASE_H
#define RANK_SGMV_BGMV_LORA_BASE_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "lora.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sums of d_in products of 8-bit integers are held in 32 bits: 2^14 * 131071 < 2^31. */
#define LORA_MAX_BASE_D_IN 131071
#define LORA_MAX_HEAD_DIM 1024
#define LORA_MAX_HEADS 65535  /* of one tensor of lora_rotary_apply */

/* Symmetric 8-bit quantisation of rows.  With a = max_c |x[t][c]|,
 *
 *     scale[t] = a / 127        q[t][c] = rint(127 * x[t][c] / a)
 *
 * where the quotient is rounded as if it were known exactly, ties to even, so
 * q is determined by x alone and lies in -127 .. 127.  A row of zeros has
 * scale 0 and q 0.  A row that holds an infinity or a NaN has scale NaN and q
 * 0: what is computed from it is NaN, and other rows are not touched by it.
 * For activations (a scale for each token) and for weights [d_out][d_in] (a
 * scale for each output channel).
 *   x      [n_rows][ldx] dtype, ldx >= d
 *   q      [n_rows][ldq] int8, ldq >= d, must not overlap x
 *   scale  [n_rows] float32
 * n_rows == 0 launches nothing.  LORA_EINVAL: NULL, a bad dtype, x not
 * aligned to its element or scale not to 4 bytes, overlap; LORA_ESHAPE:
 * n_rows < 0, d < 1, ld < d. */
lora_status lora_quantize_rows(const void *x, int64_t ldx, lora_dtype dtype, int32_t n_rows, int32_t d, int8_t *q,
                               int64_t ldq, float *scale, hipStream_t stream);

/* A base weight in 8 bits: W [d_out][ldw] int8 (any values, -128 too), a
 * float32 scale for each output channel, and a float32 bias or NULL. */
typedef struct {
  const int8_t *W;
  const float *scale;  /* [d_out] */
  const float *bias;   /* [d_out], or NULL */
  int64_t ldw;         /* >= d_in */
  int32_t d_in;
  int32_t d_out;
} lora_base_weight;

/* The product of quantised rows and a quantised weight:
 *
 *     y[t][o] = (float(sum_c q[t][c] * W[o][c]) * q_scale[t]) * scale[o] (+ bias[o])
 *
 * for t < n_tokens, o < d_out.  The sum is exact (32-bit integers); the rest
 * is float32, rounded once to y's type.
 *   q        [n_tokens][ldq] int8, ldq >= d_in;  q_scale [n_tokens] float32
 *   y        [n_tokens][ldy] dtype, ldy >= d_out, written (not added to); it
 *            must not overlap what the call reads
 * The fastest kernels need q, W, ldq, ldw and d_in to be multiples of 16.
 * n_tokens == 0 launches nothing.  LORA_EINVAL: NULL, a bad dtype, y not
 * aligned to its element or a float array not to 4 bytes, overlap;
 * LORA_ESHAPE: n_tokens < 0, a size < 1, ld < d; LORA_EUNSUPPORTED: d_in >
 * LORA_MAX_BASE_D_IN. */
lora_status lora_base_product(const lora_base_weight *weight, const int8_t *q, int64_t ldq, const float *q_scale,
                              int32_t n_tokens, void *y, int64_t ldy, lora_dtype dtype, hipStream_t stream);

/* Bytes of workspace that lora_base_apply needs for n_tokens rows (host only,
 * nothing is launched); 0 for an invalid weight or n_tokens < 1.  Never
 * smaller for more tokens. */
size_t lora_base_workspace_size(const lora_base_weight *weight, int32_t n_tokens);

/* lora_quantize_rows and lora_base_product in one call: y from x of the same
 * type, with the quantised rows in the workspace.  The workspace is written
 * before it is read, so it needs no initialisation; calls that may overlap in
 * time need one each.
 *   x  [n_tokens][ldx] dtype, ldx >= d_in;  y [n_tokens][ldy] dtype, ldy >= d_out
 *   ws 16-byte aligned, at least lora_base_workspace_size bytes (LORA_EWORKSPACE)
 * x, y and ws must not overlap; other errors as above. */
lora_status lora_base_apply(const lora_base_weight *weight, const void *x, int64_t ldx, int32_t n_tokens, void *y,
                            int64_t ldy, lora_dtype dtype, void *ws, size_t ws_bytes, hipStream_t stream);

/* Rotary positions.  The first rot_dim values of a head are rot_dim / 2
 * pairs: pair j is (j, j + rot_dim / 2), or with `interleaved` (2j, 2j + 1).
 * At position p pair (a, b) becomes
 *
 *     (m (a cos w - b sin w), m (b cos w + a sin w)),   w = p * freq[j], m = mscale
 *
 * or with `inverse` the same with -w (the gradient of the first form; for m =
 * 1 also its inverse).  The other values of a head are left as they are.
 * Angles, m cos w and m sin w are computed in float64, for any position and
 * angles up to 2^50, and rounded to float32; the rest in float32, rounded once. */
typedef struct {
  const double *freq;   /* [rot_dim / 2], radians per position */
  int32_t head_dim;     /* 1 .. LORA_MAX_HEAD_DIM */
  int32_t rot_dim;      /* even, 2 .. head_dim */
  int32_t interleaved;  /* 0 or 1 */
  float mscale;
} lora_rotary;

/* A tensor of heads: value i of head h of token t is at t * token + h * head
 * + i (element strides).  dst may be src (with the same strides: in place),
 * or memory that does not overlap it.  Strides are not negative, and those of
 * dst keep its values apart. */
typedef struct {
  const void *src;
  void *dst;
  int64_t src_token, src_head;
  int64_t dst_token, dst_head;
  int32_t n_heads;  /* 1 .. LORA_MAX_HEADS */
} lora_rotary_slice;

/* Rotates up to LORA_MAX_SLICES tensors (query and key heads) of the same
 * tokens in one launch.
 *   positions  [n_tokens] int32.  A token of a negative position is skipped:
 *              its values in dst are left as they were.
 *   slices     HOST array of n_slices
 * n_tokens == 0 launches nothing.  LORA_EINVAL: NULL, a bad dtype or flag,
 * pointers not aligned to their element, overlap (between slices too);
 * LORA_ESHAPE: sizes and strides that do not fit what is said above;
 * LORA_EUNSUPPORTED: head_dim > LORA_MAX_HEAD_DIM. */
lora_status lora_rotary_apply(const lora_rotary *rotary, const int32_t *positions, int32_t n_tokens, int32_t n_slices,
                              const lora_rotary_slice *slices, lora_dtype dtype, int32_t inverse, hipStream_t stream);

/* How the frequencies base^(-2j / rot_dim) are changed for contexts longer
 * than a model was trained on (`factor` times as long). */
typedef enum {
  LORA_ROTARY_PLAIN = 0,   /* unchanged */
  LORA_ROTARY_LINEAR = 1,  /* every frequency divided by factor */
  LORA_ROTARY_BASE = 2,    /* base * factor^(rot_dim / (rot_dim - 2)): the slowest pair slowed by factor, the fastest not */
  LORA_ROTARY_PARTS = 3    /* by the turns n = length * freq / (2 pi) of a pair over the trained length: unchanged for
                              n >= high, divided by factor for n <= low, linear in n between the two */
} lora_rotary_scaling;

/* Fills the HOST array freq [rot_dim / 2].  `factor` (> 0) is read by every
 * scaling but PLAIN; length, low and high (length > 0, 0 <= low < high) by
 * PARTS.  LORA_EINVAL: NULL or a bad scaling; LORA_ESHAPE: a rot_dim that is
 * odd or < 2 (for BASE: < 4), base or another number out of range or not
 * finite. */
lora_status lora_rotary_frequencies(lora_rotary_scaling scaling, double base, int32_t rot_dim, double factor,
                                    double length, double low, double high, double *freq);

#ifdef __cplusplus
}
#endif

#endif /* RANK_SGMV_BGMV_LORA_BASE_H */
