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
#include "lora_rows.hpp"

namespace lora {
namespace {

constexpr int kQuantThreads = 256;

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
