// Rows of bf16 or fp32 in registers and their 8-bit form: a = max |x|, scale = a
// / 127, q = rint(127 x / a).  Shared by the kernels that quantise what they read
// or compute.
#pragma once

#include "lora_device.hpp"

namespace lora {

constexpr uint32_t kInfBits = 0x7f800000u;

// 16 bytes of a row as floats, at any alignment (global accesses of any
// alignment are in order on this hardware; an aligned one costs the same).
template <typename E> struct RowVec;
template <> struct RowVec<uint16_t> {
  static constexpr int kN = 8;
  typedef uint32_t U __attribute__((ext_vector_type(4), aligned(2)));
  typedef uint32_t Q __attribute__((ext_vector_type(2), aligned(1)));
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const { return i % 2 ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]); }
};
template <> struct RowVec<float> {
  static constexpr int kN = 4;
  typedef uint32_t U __attribute__((ext_vector_type(4), aligned(4)));
  typedef uint32_t Q __attribute__((aligned(1)));
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const { return __uint_as_float(w[i]); }
};

// The vector at p, of which n (1 or more) elements are there: the rest are zeros.
template <typename E>
__device__ __forceinline__ RowVec<E> load_vec(const E *p, int n) {
  typedef typename RowVec<E>::U U;
  RowVec<E> v;
  if (n >= RowVec<E>::kN) {
    const U u = *(const LORA_GLOBAL U *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = u[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 4) {
        v.w[i] = i < n ? __float_as_uint(gload<float>(p + i)) : 0u;
      } else {
        v.w[i] = 2 * i < n ? uint32_t(gload<uint16_t>(p + 2 * i)) : 0u;
        if (2 * i + 1 < n) v.w[i] |= uint32_t(gload<uint16_t>(p + 2 * i + 1)) << 16;
      }
    }
  }
  return v;
}

template <typename E>
__device__ __forceinline__ uint32_t max_bits(const RowVec<E> &v, uint32_t m) {
#pragma unroll
  for (int i = 0; i < RowVec<E>::kN; ++i) m = max(m, __float_as_uint(v.get(i)) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t m) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), o)));
  return m;
}

// What a row's elements are multiplied with, from the bits of its maximum.
struct RowScale {
  float a;      // the maximum, or 0 for a row that quantises to zeros
  float r;      // 127 / a; 0 for a maximum so small that it would not be finite
  float scale;  // a / 127
  // (limit: the bits of the first maximum that no row may have)
  __device__ __forceinline__ explicit RowScale(uint32_t bits, uint32_t limit = kInfBits) {
    a = bits < limit ? __uint_as_float(bits) : 0.f;
    r = a > 0x1p-100f ? 127.f / a : 0.f;
    scale = bits < limit ? a / 127.f : __uint_as_float(0x7fc00000u);
  }
};

// rint(127 x / a) of a vector's elements, as bytes.  x r is off by at most
// three roundings, 127 * 3 * 2^-24 = 2.3e-5; where one of them is that near to
// a half (and in rows of tiny values) the quotients are taken in float64: 127 x
// is exact there, a true half comes out as one, and a quotient of two 24-bit
// numbers that is no half is at least 2^-33 away from it.
template <typename E>
__device__ __forceinline__ void store_vec(int8_t *q, const RowVec<E> &v, const RowScale &s, int n) {
  constexpr int kN = RowVec<E>::kN;
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number, in the low bits
  uint32_t k[kN];
  float far = s.r > 0.f ? 0.f : 1.f;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const float t = v.get(i) * s.r, u = t + kRound;
    k[i] = __float_as_uint(u);
    far = fmaxf(far, fabsf(t - (u - kRound)));
  }
  if (far > 0.49997f) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      k[i] = s.a > 0.f ? uint32_t(int(rint(127.0 * double(v.get(i)) / double(s.a)))) : 0u;
  }
  uint32_t w[kN / 4];
#pragma unroll
  for (int i = 0; i < kN / 4; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(k[4 * i + 1], k[4 * i], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(k[4 * i + 3], k[4 * i + 2], 0x0c0c0400u);
    w[i] = lo | hi << 16;
  }
  if (n >= kN) {
    if constexpr (kN == 8) {
      const typename RowVec<E>::Q u = {w[0], w[1]};
      *(LORA_GLOBAL typename RowVec<E>::Q *)q = u;
    } else {
      *(LORA_GLOBAL typename RowVec<E>::Q *)q = w[0];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < n) *(LORA_GLOBAL int8_t *)(q + i) = int8_t(w[i / 4] >> (i % 4 * 8));
  }
}

}  // namespace lora
