// Rows in 8 bits: a = max |x|, scale = a / 127, q = rint(127 x / a).
//
// The maximum is taken over the bits of |x| as whole numbers, which order like
// the values they stand for, with infinity and NaN above every finite one: one
// integer maximum finds both the row's scale and whether it has one.

#include "lora_base.hpp"
#include "lora_device.hpp"

namespace lora {
namespace {

constexpr int kQuantThreads = 256;
constexpr uint32_t kInfBits = 0x7f800000u;

template <typename E> __device__ __forceinline__ float load_f(const E *p);
template <> __device__ __forceinline__ float load_f<uint16_t>(const uint16_t *p) { return bf_to_f(gload<uint16_t>(p)); }
template <> __device__ __forceinline__ float load_f<float>(const float *p) { return gload<float>(p); }

// What a row's elements are multiplied with, from the bits of its maximum.
struct RowScale {
  float pre;    // a power of two that keeps 127 / a finite for a tiny maximum (exact for such rows)
  float r;      // 127 / (a pre)
  float scale;  // a / 127
  double a;     // a pre
  __device__ __forceinline__ explicit RowScale(uint32_t bits) {
    const float m = __uint_as_float(bits);
    const bool some = bits != 0 && bits < kInfBits;
    pre = m < 0x1p-64f ? 0x1p64f : 1.f;
    const float s = m * pre;
    a = double(s);
    r = some ? 127.f / s : 0.f;
    scale = bits < kInfBits ? m / 127.f : __uint_as_float(0x7fc00000u);
  }
};

// rint(127 x / a).  x r is off by at most three roundings, 127 * 3 * 2^-24 =
// 2.3e-5; where it is that near to a half the quotient is taken in float64:
// 127 x is exact there, a true half comes out as one, and a quotient of two
// 24-bit numbers that is no half is at least 2^-33 away from it.
__device__ __forceinline__ int quantize(float x, const RowScale &s) {
  const float xs = x * s.pre;
  const float t = s.r == 0.f ? 0.f : xs * s.r;
  float k = rintf(t);
  if (fabsf(t - k) > 0.49997f) k = float(rint(127.0 * double(xs) / s.a));
  return int(k);
}

template <typename E>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(QuantArgs a) {
  __shared__ uint32_t part[kQuantThreads / 64];
  const int64_t row = blockIdx.x;
  const E *x = static_cast<const E *>(a.x) + row * a.ldx;
  int8_t *q = a.q + row * a.ldq;
  uint32_t m = 0;
  for (int c = threadIdx.x; c < a.d; c += kQuantThreads) m = max(m, __float_as_uint(load_f(x + c)) & 0x7fffffffu);
  for (int o = 32; o > 0; o >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), o)));
  if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / 64; ++w) m = max(m, part[w]);
  const RowScale s(m);
  for (int c = threadIdx.x; c < a.d; c += kQuantThreads) q[c] = int8_t(quantize(load_f(x + c), s));
  if (threadIdx.x == 0) a.scale[row] = s.scale;
}

}  // namespace

hipError_t launch_quantize(const QuantArgs &a, int dtype, hipStream_t stream) {
  if (dtype == LORA_BF16)
    quantize_rows_kernel<uint16_t><<<a.rows, kQuantThreads, 0, stream>>>(a);
  else
    quantize_rows_kernel<float><<<a.rows, kQuantThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace lora
