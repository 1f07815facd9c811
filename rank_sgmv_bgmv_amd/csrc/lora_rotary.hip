// Rotary positions: the pairs of each head turned by position * frequency.
//
// Angles are float64 products, reduced to a fraction of a turn there, so that
// a position of millions keeps an error of 2^-26 turns; sine and cosine of the
// fraction are float32.  One table of rot_dim / 2 of them serves all heads of a
// token, in LDS.

#include "lora_base.hpp"
#include "lora_device.hpp"

namespace lora {
namespace {

constexpr int kRotaryThreads = 256;

template <typename E> __device__ __forceinline__ float load_f(const E *p);
template <> __device__ __forceinline__ float load_f<uint16_t>(const uint16_t *p) { return bf_to_f(gload<uint16_t>(p)); }
template <> __device__ __forceinline__ float load_f<float>(const float *p) { return gload<float>(p); }
__device__ __forceinline__ void store_f(uint16_t *p, float v) { gstore(p, f_to_bf(v)); }
__device__ __forceinline__ void store_f(float *p, float v) { gstore(p, v); }

// (m cos, m sin) of position * frequency, the sine with the direction's sign.
__device__ __forceinline__ float2 turn(int pos, double freq, float m, float sign) {
  const double turns = double(pos) * freq * 0.15915494309189533576888;  // 1 / (2 pi)
  const float f = float(turns - rint(turns));
  float sn, cs;
  sincospif(2.f * f, &sn, &cs);
  return make_float2(m * cs, m * sign * sn);
}

template <typename E>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(RotaryArgs a) {
  __shared__ float2 cs[LORA_MAX_HEAD_DIM / 2];
  const int64_t t = blockIdx.x;
  const int pos = gload<int>(a.positions + t);
  if (pos < 0) return;
  const int half = a.rot_dim / 2, rest = a.head_dim - a.rot_dim;
  for (int j = threadIdx.x; j < half; j += kRotaryThreads) cs[j] = turn(pos, gload<double>(a.freq + j), a.mscale, a.sign);
  __syncthreads();
  for (int s = 0; s < a.n_slices; ++s) {
    const lora_rotary_slice &v = a.s[s];
    const E *src = static_cast<const E *>(v.src) + t * v.src_token;
    E *dst = static_cast<E *>(v.dst) + t * v.dst_token;
    for (int i = threadIdx.x; i < v.n_heads * half; i += kRotaryThreads) {
      const int h = i / half, j = i % half;
      const int p0 = a.interleaved ? 2 * j : j, p1 = a.interleaved ? 2 * j + 1 : j + half;
      const E *x = src + h * v.src_head;
      E *y = dst + h * v.dst_head;
      const float x0 = load_f(x + p0), x1 = load_f(x + p1);
      store_f(y + p0, x0 * cs[j].x - x1 * cs[j].y);
      store_f(y + p1, x1 * cs[j].x + x0 * cs[j].y);
    }
    if (v.src != v.dst)
      for (int i = threadIdx.x; i < v.n_heads * rest; i += kRotaryThreads) {
        const int h = i / rest, j = a.rot_dim + i % rest;
        gstore(dst + h * v.dst_head + j, gload<E>(src + h * v.src_head + j));
      }
  }
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, int dtype, hipStream_t stream) {
  if (dtype == LORA_BF16)
    rotary_kernel<uint16_t><<<a.T, kRotaryThreads, 0, stream>>>(a);
  else
    rotary_kernel<float><<<a.T, kRotaryThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace lora
