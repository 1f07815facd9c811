// The 8-bit base product y = (q W^T) scaled by token and channel.
//
// The channels are the rows of the matrix instruction's result and the tokens
// its columns, so that a lane holds four neighbouring channels of one token
// and stores them together.  Both operands have the sum's axis contiguous,
// which is the order in which v_mfma_i32_16x16x64_i8 takes them: a lane holds
// 16 consecutive values of one row.

#include "lora_base.hpp"
#include "lora_device.hpp"

namespace lora {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bias_of(const ProductArgs &a, int o) { return a.bias ? gload<float>(a.bias + o) : 0.f; }

// Up to four neighbouring channels of one token, from channel o on.
__device__ __forceinline__ void store_y(const ProductArgs &a, uint16_t *y, int o, const float *v) {
  uint16_t *p = y + o;
  if (o + 4 <= a.d_out && reinterpret_cast<uintptr_t>(p) % 8 == 0) {
    gstore(p, make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3])));
  } else {
    for (int i = 0; i < 4; ++i)
      if (o + i < a.d_out) gstore(p + i, f_to_bf(v[i]));
  }
}
__device__ __forceinline__ void store_y(const ProductArgs &a, float *y, int o, const float *v) {
  float *p = y + o;
  if (o + 4 <= a.d_out && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    gstore(p, make_float4(v[0], v[1], v[2], v[3]));
  } else {
    for (int i = 0; i < 4; ++i)
      if (o + i < a.d_out) gstore(p + i, v[i]);
  }
}

// 16 bytes from p, of which the first n (any whole number) are there: the rest are zeros.
__device__ __forceinline__ i32x4 load16(const int8_t *p, int n) {
  typedef int i32x4u __attribute__((ext_vector_type(4), aligned(1)));
  if (n >= 16) return *(const LORA_GLOBAL i32x4u *)p;
  union {
    i32x4 v;
    int8_t b[16];
  } u;
  u.v = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) u.b[i] = *(const LORA_GLOBAL int8_t *)(p + i);
  return u.v;
}

// Any sizes, strides and alignment.  64 tokens x 64 channels, 64 values of the
// sum's axis a step, four waves of 32 x 32.  Rows of the LDS tiles are 80
// bytes apart: eight lanes that read neighbouring rows meet different banks.
constexpr int kAnyTile = 64, kAnyPitch = 80;
template <typename E>
__global__ __launch_bounds__(256) void product_any_kernel(ProductArgs a) {
  __shared__ __align__(16) int8_t lx[kAnyTile * kAnyPitch], lw[kAnyTile * kAnyPitch];
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int o0 = blockIdx.x * kAnyTile;
  const int64_t t0 = int64_t(blockIdx.y) * kAnyTile;
  const int row = tid / 4, chunk = tid % 4 * 16;
  const bool has_x = t0 + row < a.T, has_w = o0 + row < a.d_out;
  const int8_t *px = a.q + (t0 + row) * a.ldq, *pw = a.W + int64_t(o0 + row) * a.ldw;
  const int wo = wave / 2 * 32, wt = wave % 2 * 32;
  i32x4 acc[2][2] = {};
  for (int k = 0; k < a.d_in; k += 64) {
    const int n = a.d_in - k - chunk;
    const i32x4 vx = load16(px + k + chunk, has_x ? n : 0), vw = load16(pw + k + chunk, has_w ? n : 0);
    __syncthreads();
    *reinterpret_cast<i32x4 *>(lx + row * kAnyPitch + chunk) = vx;
    *reinterpret_cast<i32x4 *>(lw + row * kAnyPitch + chunk) = vw;
    __syncthreads();
    i32x4 fw[2], fx[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fw[i] = *reinterpret_cast<const i32x4 *>(lw + (wo + i * 16 + lane % 16) * kAnyPitch + lane / 16 * 16);
      fx[i] = *reinterpret_cast<const i32x4 *>(lx + (wt + i * 16 + lane % 16) * kAnyPitch + lane / 16 * 16);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], fx[j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int64_t t = t0 + wt + j * 16 + lane % 16;
    if (t >= a.T) continue;
    const float sx = gload<float>(a.q_scale + t);
    E *y = static_cast<E *>(a.y) + t * a.ldy;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int o = o0 + wo + i * 16 + lane / 16 * 4;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = min(o + e, a.d_out - 1);
        v[e] = float(acc[i][j][e]) * sx * gload<float>(a.w_scale + c) + bias_of(a, c);
      }
      store_y(a, y, o, v);
    }
  }
}

}  // namespace

hipError_t launch_product(const ProductArgs &a, int dtype, hipStream_t stream) {
  const dim3 grid((a.d_out + kAnyTile - 1) / kAnyTile, (a.T + kAnyTile - 1) / kAnyTile);
  if (dtype == LORA_BF16)
    product_any_kernel<uint16_t><<<grid, 256, 0, stream>>>(a);
  else
    product_any_kernel<float><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace lora
