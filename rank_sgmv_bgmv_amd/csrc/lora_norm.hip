// Root-mean-square norm with the residual's addition before it and the 8-bit
// form of its result behind it: h = x + r, y = h w / sqrt(mean h^2 + eps), and
// a = max |y|, scale = a / 127, q = rint(127 y / a).
//
// A row is read once and stays in registers: as h until its mean is known, as y
// until its maximum is.  Both sums over a row run over the lanes in the same
// order whatever the batch, so a row's bits are its own.
//
// The mean, its root and y are float64.  Float32 sums would put y off by some
// 2^-23, and where that crosses the border between two values of the output's
// type the 8-bit values that follow move by whole steps; in float64 they are
// what the formula says.  The arithmetic hides behind the memory accesses: some
// 12 float64 operations a value of 9 bytes, at 64 of them a clock and CU.
//
// Bound by memory: 16997 rows of 4096 bf16 values with everything asked for are
// 627 MB and take 126 us, 5.0 TB/s.  64 such rows take 5.8 us, the length of one
// row: loads, two sums over four waves, stores.

#include "lora_layer.hpp"
#include "lora_rows.hpp"

namespace lora {
namespace {

template <typename E>
__device__ __forceinline__ void put_pair(RowVec<E> &v, int i, float a, float b) {
  if constexpr (sizeof(E) == 4) v.w[i] = __float_as_uint(a), v.w[i + 1] = __float_as_uint(b);
  else v.w[i / 2] = pack_bf2(a, b);
}

// The first n elements of v at p, at any alignment of elements.
template <typename E>
__device__ __forceinline__ void store_row_vec(E *p, const RowVec<E> &v, int n) {
  if (n >= RowVec<E>::kN) {
    const typename RowVec<E>::U u = {v.w[0], v.w[1], v.w[2], v.w[3]};
    *(LORA_GLOBAL typename RowVec<E>::U *)p = u;
  } else {
#pragma unroll
    for (int i = 0; i < RowVec<E>::kN; ++i)
      if (i < n) {
        if constexpr (sizeof(E) == 4) gstore(p + i, v.w[i]);
        else gstore(p + i, uint16_t(v.w[i / 2] >> (i % 2 * 16)));
      }
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// TH threads a row, VPL vectors a lane, kRows rows a workgroup.
template <typename E, int TH, int VPL>
__global__ __launch_bounds__(TH < 256 ? 256 : TH) void norm_kernel(NormArgs a) {
  constexpr int kN = RowVec<E>::kN, kThreads = TH < 256 ? 256 : TH, kRows = kThreads / TH, kWaves = TH / 64;
  __shared__ double sums[2][kThreads / 64];
  __shared__ uint32_t tops[2][kThreads / 64];
  const int lane = threadIdx.x % TH;
  int turn = 0;
  for (int64_t row0 = int64_t(blockIdx.x) * kRows; row0 < a.rows; row0 += int64_t(gridDim.x) * kRows, turn ^= 1) {
    const int64_t row = row0 + (kRows > 1 ? uniform(threadIdx.x / TH) : 0);
    if (row >= a.rows) return;  // one wave a row: no barrier is missed
    const E *x = static_cast<const E *>(a.x) + row * a.ldx;
    const E *r = static_cast<const E *>(a.residual) + row * a.ldr;
    E *total = static_cast<E *>(a.total) + row * a.ldt;
    RowVec<E> v[VPL];
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = (k * TH + lane) * kN;
      v[k] = c < a.d ? load_vec(x + c, a.d - c) : RowVec<E>{{0u, 0u, 0u, 0u}};
    }
    if (a.residual) {
      RowVec<E> u[VPL];
#pragma unroll
      for (int k = 0; k < VPL; ++k) {
        const int c = (k * TH + lane) * kN;
        u[k] = c < a.d ? load_vec(r + c, a.d - c) : RowVec<E>{{0u, 0u, 0u, 0u}};
      }
#pragma unroll
      for (int k = 0; k < VPL; ++k) {
#pragma unroll
        for (int i = 0; i < kN; i += 2)
          put_pair(v[k], i, v[k].get(i) + u[k].get(i), v[k].get(i + 1) + u[k].get(i + 1));
        const int c = (k * TH + lane) * kN;
        if (a.total && c < a.d) store_row_vec(total + c, v[k], a.d - c);
      }
    }
    double sum = 0;
#pragma unroll
    for (int k = 0; k < VPL; ++k)
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const double h = v[k].get(i);
        sum = fma(h, h, sum);
      }
    sum = wave_sum(sum);
    if constexpr (kWaves > 1) {
      // two sets in turn: the next row's parts never meet a wave that still reads this row's
      if (lane % 64 == 0) sums[turn][lane / 64] = sum;
      lds_barrier();
      sum = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sum += sums[turn][w];
    }
    const double root = 1.0 / sqrt(sum / a.d + a.eps);
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = (k * TH + lane) * kN;
      if (c < a.d) {
        float w[kN];
#pragma unroll
        for (int i = 0; i < kN; i += 4) {
          const RowVec<float> g = c + i < a.d ? load_vec(a.weight + c + i, a.d - c - i) : RowVec<float>{{0u, 0u, 0u, 0u}};
#pragma unroll
          for (int j = 0; j < 4; ++j) w[i + j] = g.get(j);
        }
#pragma unroll
        for (int i = 0; i < kN; i += 2)
          put_pair(v[k], i, float(v[k].get(i) * root * double(w[i])), float(v[k].get(i + 1) * root * double(w[i + 1])));
        if (c + kN > a.d) {
          // (past the row's end 0 * root may be NaN)
#pragma unroll
          for (int i = 0; i < kN; i += 2)
            put_pair(v[k], i, c + i < a.d ? v[k].get(i) : 0.f, c + i + 1 < a.d ? v[k].get(i + 1) : 0.f);
        }
        if (a.y) store_row_vec(static_cast<E *>(a.y) + row * a.ldy + c, v[k], a.d - c);
        top = max_bits(v[k], top);
      }
    }
    if (!a.q) continue;
    top = wave_max(top);
    if constexpr (kWaves > 1) {
      if (lane % 64 == 0) tops[turn][lane / 64] = top;
      lds_barrier();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = max(top, tops[turn][w]);
    }
    const RowScale s(top);
#pragma unroll
    for (int k = 0; k < VPL; ++k) {
      const int c = (k * TH + lane) * kN;
      if (c < a.d) store_vec(a.q + row * a.ldq + c, v[k], s, a.d - c);
    }
    if (lane == 0) gstore(a.scale + row, s.scale);
  }
}

template <typename E>
hipError_t launch_typed(const NormArgs &a, hipStream_t stream) {
  const int vecs = (a.d - 1) / RowVec<E>::kN + 1;
  const auto grid = [&](int rows) { return dim3(uint32_t(a.rows < (1 << 16) * rows ? (a.rows - 1) / rows + 1 : 1 << 16)); };
  if (vecs <= 64) norm_kernel<E, 64, 1><<<grid(4), 256, 0, stream>>>(a);
  else if (vecs <= 128) norm_kernel<E, 64, 2><<<grid(4), 256, 0, stream>>>(a);
  else if (vecs <= 256) norm_kernel<E, 256, 1><<<grid(1), 256, 0, stream>>>(a);
  else if (vecs <= 512) norm_kernel<E, 256, 2><<<grid(1), 256, 0, stream>>>(a);
  else if (vecs <= 1024) norm_kernel<E, 256, 4><<<grid(1), 256, 0, stream>>>(a);
  else if (vecs <= 2048) norm_kernel<E, 256, 8><<<grid(1), 256, 0, stream>>>(a);
  else if (vecs <= 4096) norm_kernel<E, 1024, 4><<<grid(1), 1024, 0, stream>>>(a);
  else if (vecs <= 8192) norm_kernel<E, 1024, 8><<<grid(1), 1024, 0, stream>>>(a);
  else norm_kernel<E, 1024, 16><<<grid(1), 1024, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs &a, int dtype, hipStream_t stream) {
  return dtype == LORA_BF16 ? launch_typed<uint16_t>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace lora
