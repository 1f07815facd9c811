// Internal declarations of the base product, the row quantisation and the
// rotary kernels (include/lora_base.h).  Not part of the public ABI.
#pragma once

#include "lora_base.h"
#include "lora_internal.hpp"

namespace lora {

struct QuantArgs {
  const void *x;
  int8_t *q;
  float *scale;
  int64_t ldx, ldq;
  int rows, d;
};
hipError_t launch_quantize(const QuantArgs &a, int dtype, hipStream_t stream);

struct ProductArgs {
  const int8_t *q, *W;
  const float *q_scale, *w_scale, *bias;  // bias may be nullptr
  void *y;
  int64_t ldq, ldw, ldy;
  int T, d_in, d_out;
  int y_by;  // results pass the caches by (set at the launch)
};
hipError_t launch_product(const ProductArgs &a, int dtype, hipStream_t stream);

// The product's kernels, and which one a launch takes.
enum {
  PRODUCT_TILE = 0,       // tiles, in the order of their costs
  PRODUCT_FEW_LINES = 7,  // up to 16, 32 and 64 rows of whole 16-byte pieces
  PRODUCT_FEW = 10,       // up to 16 rows
  PRODUCT_ROWS_128 = 11,  // tiles of 128 x 128 and 64 x 64 through registers
  PRODUCT_ROWS_64 = 12,
  PRODUCT_ANY = 13,
  PRODUCT_KERNELS = 14
};
struct ProductChoice {
  int kernel;
  int first;  // not 0: so many rows in a launch of their own and the rest in another, each with a choice of its own
};
ProductChoice choose_product(const ProductArgs &a);

struct RotaryArgs {
  const double *freq;
  const int32_t *positions;
  int T, head_dim, rot_dim, interleaved;
  float mscale, sign;  // sign of the angle: 1, or -1 for the inverse
  int n_slices, n_heads;  // heads of all slices
  int by;                 // results pass the caches by (set at the launch)
  lora_rotary_slice s[LORA_MAX_SLICES];
};
hipError_t launch_rotary(const RotaryArgs &a, int dtype, hipStream_t stream);

}  // namespace lora
