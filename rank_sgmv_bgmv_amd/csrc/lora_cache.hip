// The 8-bit cache: heads of keys and values quantised into slots of its pages,
// and read back.
//
// A head is a row of its own: a = max |x|, scale = a / 127, q = rint(127 x / a),
// by the same code as lora_quantize_rows.  kLanes neighbouring lanes take a head,
// up to kVecs vectors each, and nothing crosses more than them.
//
// Each value is read and written once: 16997 tokens of 8 + 8 bf16 heads of 128
// are 106 MB, 21 us at the rate of a large copy.  Writing them takes 30 us and
// reading them back 18.5; half the vectors a lane, so twice the lanes that
// compute addresses and scales, took 39 and 22: instructions bound the first.
// 64 tokens take 4 and 3 us, the length of one chain of loads.

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
    token = int64_t(a.T) * per <= 0x7fffffff ? int64_t(uint32_t(row) / uint32_t(per)) : row / per;
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

// The largest over the kLanes neighbouring lanes of a row (8, 16 or 32), by moves within the register file.
template <int kLanes>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
#define LORA_DPP(how) v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), how, 0xf, 0xf, false)))
  LORA_DPP(0xb1);   // neighbours
  LORA_DPP(0x4e);   // pairs of a quad
  LORA_DPP(0x141);  // mirrored halves of a row of 16
  if constexpr (kLanes > 8) LORA_DPP(0x140);  // mirrored rows of 16
#undef LORA_DPP
  if constexpr (kLanes > 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(uint32_t(s[0]), uint32_t(s[1]));
  }
  return v;
}

template <typename E, int kLanes, int kVecs>
__global__ __launch_bounds__(kCacheThreads) void cache_write_kernel(CacheArgs a) {
  constexpr int kN = RowVec<E>::kN, kRows = kCacheThreads / kLanes;
  const int lane = threadIdx.x % kLanes;
  const int64_t rows = int64_t(a.T) * 2 * a.c.n_heads;
  for (int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes; row < rows; row += int64_t(gridDim.x) * kRows) {
    const CacheRow at(a, row);
    const int slot = gload<int>(a.slots + at.token);
    const E *from = at.outside<const E>(a);
    RowVec<E> v[kVecs];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * kLanes + lane) * kN;
      v[k] = c < a.c.head_dim ? load_vec(from + c, a.c.head_dim - c) : RowVec<E>{{0u, 0u, 0u, 0u}};
      m = max_bits(v[k], m);
    }
    m = lanes_max<kLanes>(m);
    if (!in_cache(a, slot)) continue;
    const RowScale s(m, kMostBits);
    int8_t *to = at.inside(a, slot);
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * kLanes + lane) * kN;
      if (c < a.pitch) store_vec(to + c, v[k], s, kN);
    }
    if (lane == 0) gstore(at.scale(a, slot), s.scale);
  }
}

template <typename E, int kLanes, int kVecs>
__global__ __launch_bounds__(kCacheThreads) void cache_read_kernel(CacheArgs a) {
  constexpr int kN = RowVec<E>::kN, kRows = kCacheThreads / kLanes;
  const int lane = threadIdx.x % kLanes;
  const int64_t rows = int64_t(a.T) * 2 * a.c.n_heads;
  for (int64_t row = int64_t(blockIdx.x) * kRows + threadIdx.x / kLanes; row < rows; row += int64_t(gridDim.x) * kRows) {
    const CacheRow at(a, row);
    const int slot = gload<int>(a.slots + at.token);
    if (!in_cache(a, slot)) continue;
    const float scale = gload<float>(at.scale(a, slot));
    const int8_t *from = at.inside(a, slot);
    uint32_t w[kVecs][kN / 4];
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int8_t *p = from + min((k * kLanes + lane) * kN, a.pitch - kN);
      if constexpr (kN == 8) {
        const uint2 u = gload<uint2>(p);
        w[k][0] = u.x, w[k][1] = u.y;
      } else {
        w[k][0] = gload<uint32_t>(p);
      }
    }
#pragma unroll
    for (int k = 0; k < kVecs; ++k) {
      const int c = (k * kLanes + lane) * kN, n = a.c.head_dim - c;
      float f[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) f[i] = float(int8_t(w[k][i / 4] >> (i % 4 * 8))) * scale;
      E *to = at.outside<E>(a) + c;
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
}

template <typename E, bool kWrite, int kLanes, int kVecs>
void launch_lanes(const CacheArgs &a, hipStream_t stream) {
  const int64_t rows = int64_t(a.T) * 2 * a.c.n_heads, groups = (rows - 1) / (kCacheThreads / kLanes) + 1;
  const dim3 grid(uint32_t(groups < (1 << 18) ? groups : 1 << 18));
  if constexpr (kWrite) cache_write_kernel<E, kLanes, kVecs><<<grid, kCacheThreads, 0, stream>>>(a);
  else cache_read_kernel<E, kLanes, kVecs><<<grid, kCacheThreads, 0, stream>>>(a);
}

template <typename E, bool kWrite>
hipError_t launch_typed(const CacheArgs &a, hipStream_t stream) {
  // two vectors a lane wherever eight lanes have them
  const int vecs = (a.pitch - 1) / RowVec<E>::kN + 1;
  if (vecs <= 8) launch_lanes<E, kWrite, 8, 1>(a, stream);
  else if (vecs <= 16) launch_lanes<E, kWrite, 8, 2>(a, stream);
  else if (vecs <= 32) launch_lanes<E, kWrite, 16, 2>(a, stream);
  else launch_lanes<E, kWrite, 32, 2>(a, stream);
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
