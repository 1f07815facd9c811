// Rows in 8 bits: a = max |x|, scale = a / 127, q = rint(127 x / a).
//
// The maximum is taken over the bits of |x| as whole numbers, which order like
// the values they stand for, with infinity and NaN above every finite one: one
// integer maximum finds both the row's scale and whether it has one.
//
// Bound by memory: a row is read once, kept in registers between the maximum
// and the rounding, and written once in 8 bits.  Rows of up to 4 vectors a lane
// of one wave have a wave each (no barrier), longer ones a workgroup, and rows
// beyond 16 vectors a lane are read twice, the second time from cache.

#include "lora_base.hpp"
#include "lora_device.hpp"

namespace lora {
namespace {

constexpr int kQuantThreads = 256;
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
  __device__ __forceinline__ explicit RowScale(uint32_t bits) {
    a = bits < kInfBits ? __uint_as_float(bits) : 0.f;
    r = a > 0x1p-100f ? 127.f / a : 0.f;
    scale = bits < kInfBits ? a / 127.f : __uint_as_float(0x7fc00000u);
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

// W waves a row, VPL vectors a lane.
template <typename E, int W, int VPL>
__global__ __launch_bounds__(kQuantThreads) void quantize_rows_kernel(QuantArgs a) {
  constexpr int kN = RowVec<E>::kN, kLanes = 64 * W, kRows = kQuantThreads / kLanes;
  __shared__ uint32_t part[2][kQuantThreads / 64];
  const int lane = threadIdx.x % kLanes;
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * kRows; row0 < a.rows; row0 += int64_t(gridDim.x) * kRows, turn ^= 1) {
    const int64_t row = row0 + (W == 1 ? uniform(threadIdx.x / kLanes) : 0);
    if (row >= a.rows) return;  // one wave a row: no barrier is missed
    const E *x = static_cast<const E *>(a.x) + row * a.ldx;
    int8_t *q = a.q + row * a.ldq;
    RowVec<E> v[VPL];
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = (k * kLanes + lane) * kN;
      if (c < a.d) v[k] = load_vec(x + c, a.d - c);
      else v[k] = RowVec<E>{{0u, 0u, 0u, 0u}};
    }
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < VPL; ++k) m = max_bits(v[k], m);
    m = wave_max(m);
    if constexpr (W > 1) {
      // two sets in turn: the next row's parts never meet a wave that still reads this row's
      if (lane % 64 == 0) part[turn][lane / 64] = m;
      lds_barrier();
#pragma unroll
      for (int w = 0; w < W; ++w) m = max(m, part[turn][w]);
    }
    const RowScale s(m);
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = (k * kLanes + lane) * kN;
      if (c < a.d) store_vec(q + c, v[k], s, a.d - c);
    }
    if (lane == 0) gstore(a.scale + row, s.scale);
  }
}

// Rows of any length, read twice.
template <typename E>
__global__ __launch_bounds__(kQuantThreads) void quantize_long_rows_kernel(QuantArgs a) {
  constexpr int kN = RowVec<E>::kN, kStep = kQuantThreads * kN;
  __shared__ uint32_t part[2][kQuantThreads / 64];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const E *x = static_cast<const E *>(a.x) + row * a.ldx;
    int8_t *q = a.q + row * a.ldq;
    uint32_t m = 0;
    for (int64_t c = threadIdx.x * kN; c < a.d; c += kStep) m = max_bits(load_vec(x + c, int(a.d - c)), m);
    m = wave_max(m);
    if (threadIdx.x % 64 == 0) part[turn][threadIdx.x / 64] = m;
    lds_barrier();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 64; ++w) m = max(m, part[turn][w]);
    const RowScale s(m);
    for (int64_t c = threadIdx.x * kN; c < a.d; c += kStep) store_vec(q + c, load_vec(x + c, int(a.d - c)), s, int(a.d - c));
    if (threadIdx.x == 0) gstore(a.scale + row, s.scale);
  }
}

template <typename E>
hipError_t launch_typed(const QuantArgs &a, hipStream_t stream) {
  constexpr int kN = RowVec<E>::kN;
  const int vecs = (a.d - 1) / kN + 1;
  // a grid of a few workgroups for each place on the chip; rows beyond it in turn
  const auto grid = [&](int rows) { return dim3(uint32_t(a.rows < (1 << 16) * rows ? (a.rows - 1) / rows + 1 : 1 << 16)); };
  const dim3 waves = grid(kQuantThreads / 64), groups = grid(1);
  if (vecs <= 64 * 4) {
    switch ((vecs - 1) / 64 + 1) {
      case 1: quantize_rows_kernel<E, 1, 1><<<waves, kQuantThreads, 0, stream>>>(a); break;
      case 2: quantize_rows_kernel<E, 1, 2><<<waves, kQuantThreads, 0, stream>>>(a); break;
      case 3: quantize_rows_kernel<E, 1, 3><<<waves, kQuantThreads, 0, stream>>>(a); break;
      default: quantize_rows_kernel<E, 1, 4><<<waves, kQuantThreads, 0, stream>>>(a); break;
    }
  } else if (vecs <= kQuantThreads * 2) {
    quantize_rows_kernel<E, 4, 2><<<groups, kQuantThreads, 0, stream>>>(a);
  } else if (vecs <= kQuantThreads * 4) {
    quantize_rows_kernel<E, 4, 4><<<groups, kQuantThreads, 0, stream>>>(a);
  } else if (vecs <= kQuantThreads * 8) {
    quantize_rows_kernel<E, 4, 8><<<groups, kQuantThreads, 0, stream>>>(a);
  } else if (vecs <= kQuantThreads * 16) {
    quantize_rows_kernel<E, 4, 16><<<groups, kQuantThreads, 0, stream>>>(a);
  } else {
    quantize_long_rows_kernel<E><<<groups, kQuantThreads, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const QuantArgs &a, int dtype, hipStream_t stream) {
  return dtype == LORA_BF16 ? launch_typed<uint16_t>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace lora
