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
