// The 8-bit cache: heads of keys and values quantised into slots of its pages,
// and read back.
//
// A head is a row of its own: a = max |x|, scale = a / 127, q = rint(127 x / a),
// by the same code as lora_quantize_rows.  kLanes lanes, a vector each, take a
// head; nothing crosses more than a wave.  Bound by memory: each value is read
// and written once.

#include "lora_layer.hpp"
#include "lora_rows.hpp"

namespace lora {
namespace {

constexpr int kCacheThreads = 256;
constexpr uint32_t kMostBits = 0x5f800000u;  // 2^64: heads with values from there on are kept as NaN

// Where row `row` of the launch lies: rows are (token, k or v, head), the head the fastest.
struct CacheRow {
  int64_t token;
  int head, value;  // value: 0 of the keys, 1 of the values
  __device__ __forceinline__ CacheRow(const CacheArgs &a, int64_t row) {
    const int per = 2 * a.c.n_heads;
    token = row / per;
    const int rest = int(row - token * per);
    value = rest >= a.c.n_heads;
    head = rest - (value ? a.c.n_heads : 0);
  }
  // the head in the tensors of the call, and in the cache
  template <typename E>
  __device__ __forceinline__ E *outside(const CacheArgs &a) const {
    const lora_heads &h = value ? a.v : a.k;
    return static_cast<E *>(h.data) + token * h.token + head * h.head;
  }
  __device__ __forceinline__ int8_t *inside(const CacheArgs &a, int slot) const {
    const int64_t page = slot >> a.page_bits, at = (int64_t(head) << a.page_bits) + (slot & ((1 << a.page_bits) - 1));
    return (value ? a.c.v + page * a.c.v_page : a.c.k + page * a.c.k_page) + at * a.pitch;
  }
  __device__ __forceinline__ float *scale(const CacheArgs &a, int slot) const {
    const int64_t page = slot >> a.page_bits, at = (int64_t(head) << a.page_bits) + (slot & ((1 << a.page_bits) - 1));
    return (value ? a.c.v_scale + page * a.c.v_scale_page : a.c.k_scale + page * a.c.k_scale_page) + at;
  }
};

__device__ __forceinline__ bool in_cache(const CacheArgs &a, int slot) {
  return slot >= 0 && (slot >> a.page_bits) < a.c.n_pages;
}

template <typename E, int kLanes>
__global__ __launch_bounds__(kCacheThreads) void cache_write_kernel(CacheArgs a) {
  constexpr int kN = RowVec<E>::kN, kRows = kCacheThreads / kLanes;
  const int lane = threadIdx.x % kLanes, c = lane * kN;
  const int64_t rows = int64_t(a.T) * 2 * a.c.n_heads;
  for (int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes; row < rows; row += int64_t(gridDim.x) * kRows) {
    const CacheRow at(a, row);
    const int slot = gload<int>(a.slots + at.token);
    RowVec<E> v = {{0u, 0u, 0u, 0u}};
    if (c < a.c.head_dim) v = load_vec(at.outside<const E>(a) + c, a.c.head_dim - c);
    uint32_t m = max_bits(v, 0u);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), o)));
    if (!in_cache(a, slot)) continue;
    const RowScale s(m, kMostBits);
    if (c < a.pitch) store_vec(at.inside(a, slot) + c, v, s, kN);
    if (lane == 0) gstore(at.scale(a, slot), s.scale);
  }
}

template <typename E, int kLanes>
__global__ __launch_bounds__(kCacheThreads) void cache_read_kernel(CacheArgs a) {
  constexpr int kN = RowVec<E>::kN, kRows = kCacheThreads / kLanes;
  const int lane = threadIdx.x % kLanes, c = lane * kN;
  const int64_t rows = int64_t(a.T) * 2 * a.c.n_heads;
  for (int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes; row < rows; row += int64_t(gridDim.x) * kRows) {
    const CacheRow at(a, row);
    const int slot = gload<int>(a.slots + at.token);
    if (!in_cache(a, slot) || c >= a.c.head_dim) continue;
    const float scale = gload<float>(at.scale(a, slot));
    const int8_t *p = at.inside(a, slot) + c;
    uint32_t w[kN / 4];
    if constexpr (kN == 8) {
      const uint2 u = gload<uint2>(p);
      w[0] = u.x, w[1] = u.y;
    } else {
      w[0] = gload<uint32_t>(p);
    }
    float f[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = float(int8_t(w[i / 4] >> (i % 4 * 8))) * scale;
    E *to = at.outside<E>(a) + c;
    const int n = a.c.head_dim - c;
    if (n >= kN) {
      typename RowVec<E>::U u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kN == 8) u[i] = pack_bf2(f[2 * i], f[2 * i + 1]);
        else u[i] = __float_as_uint(f[i]);
      }
      *(LORA_GLOBAL typename RowVec<E>::U *)to = u;
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i < n) {
          if constexpr (kN == 8) gstore(to + i, f_to_bf(f[i]));
          else gstore(to + i, f[i]);
        }
    }
  }
}

template <typename E, bool kWrite, int kLanes>
void launch_lanes(const CacheArgs &a, hipStream_t stream) {
  const int64_t rows = int64_t(a.T) * 2 * a.c.n_heads, groups = (rows - 1) / (kCacheThreads / kLanes) + 1;
  const dim3 grid(uint32_t(groups < (1 << 18) ? groups : 1 << 18));
  if constexpr (kWrite) cache_write_kernel<E, kLanes><<<grid, kCacheThreads, 0, stream>>>(a);
  else cache_read_kernel<E, kLanes><<<grid, kCacheThreads, 0, stream>>>(a);
}

template <typename E, bool kWrite>
hipError_t launch_typed(const CacheArgs &a, hipStream_t stream) {
  switch ((a.pitch - 1) / RowVec<E>::kN / 8) {  // vectors of a head, in eighths
    case 0: launch_lanes<E, kWrite, 8>(a, stream); break;
    case 1: launch_lanes<E, kWrite, 16>(a, stream); break;
    case 2:
    case 3: launch_lanes<E, kWrite, 32>(a, stream); break;
    default: launch_lanes<E, kWrite, 64>(a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(const CacheArgs &a, int dtype, hipStream_t stream) {
  return dtype == LORA_BF16 ? launch_typed<uint16_t, true>(a, stream) : launch_typed<float, true>(a, stream);
}
hipError_t launch_cache_read(const CacheArgs &a, int dtype, hipStream_t stream) {
  return dtype == LORA_BF16 ? launch_typed<uint16_t, false>(a, stream) : launch_typed<float, false>(a, stream);
}

}  // namespace lora
