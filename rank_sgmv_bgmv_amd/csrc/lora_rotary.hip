// Rotary positions: the pairs of each head turned by position * frequency.
//
// Angles are float64 products, reduced to a part of a quarter turn there, so that
// the largest positions keep theirs, and so are sine and cosine, rounded once.
// One table of rot_dim / 2 of them serves all heads of a token, in LDS.
//
// Bound by memory: every value is read and written once, 16 bytes a lane.  A
// workgroup takes kTokens tokens (one when there are few: then the heads are
// split over workgroups too) and a lane one 16-byte column of a head, for every
// slots-th head of each of them.  17k tokens of 40 bf16 heads of 128 take 64.5
// us (5.4 TB/s, as a large copy), with 70 of the 128 turned, whose partners come
// through LDS, 69; 64 tokens 3.2 us, a launch.

#include "lora_base.hpp"
#include "lora_device.hpp"

namespace lora {
namespace {

constexpr int kRotaryThreads = 256;

// Where a value's partner in its pair lies.
enum {
  ROT_HALVES = 0,  // half a rotation further on, in whole vectors: a lane takes both vectors
  ROT_NEXT = 1,    // beside it, in the same vector
  ROT_ANY = 2      // half a rotation away, inside other vectors: found in LDS
};

// (m cos, m sin) of position * frequency, the sine with the direction's sign.
// The angle is n quarter turns and w, |w| <= pi / 4.  The float64 products keep
// what they round off, so w is right for every position (angles up to 2^50).  The
// Taylor series of sine to w^9 and of cosine to w^10 end 2e-9 and 1e-10 away, a
// thirtieth of the rounding to float32 that follows, the only one that counts.
// In float32 the series lost twice as much, and took as long (17k tokens of 40
// heads of 128 64 us, 64 tokens 3.2; of one head of 64 12.2 us against 12.5).
__device__ __forceinline__ float2 turn(int pos, double freq, float m, float sign) {
#pragma clang fp contract(off)  // h is a rounded product: no sum may take it in unrounded
  constexpr double kHigh = 0.63661977236758134, kLow = -3.9357353350364972e-17;  // 2 / pi
  constexpr double kQuarter = 1.5707963267948966, kRound = 0x1.8p52;  // adding kRound rounds to a whole number, in the low bits
  const double p = double(pos), a = p * freq, a_low = fma(p, freq, -a);
  const double h = a * kHigh, h_low = fma(a, kHigh, -h) + fma(a, kLow, a_low * kHigh);
  const double u = h + kRound;
  const uint32_t n = uint32_t(__double_as_longlong(u));
  const double w = ((h - (u - kRound)) + h_low) * kQuarter, w2 = w * w;
  double s = fma(w2, 1.0 / 362880, -1.0 / 5040), c = fma(w2, -1.0 / 3628800, 1.0 / 40320);
  s = fma(w2, s, 1.0 / 120), c = fma(w2, c, -1.0 / 720);
  s = fma(w2, s, -1.0 / 6), c = fma(w2, c, 1.0 / 24);
  s = fma(w * w2, s, w), c = fma(w2, fma(w2, c, -0.5), 1.0);
  const float x = float(m * (n & 1 ? s : c)), y = sign * float(m * (n & 1 ? c : s));
  return make_float2((n + 1) & 2 ? -x : x, n & 2 ? -y : y);
}

// 16 bytes of a head, at any alignment of its elements.
template <typename E> struct HeadVec {
  static constexpr int kN = 16 / int(sizeof(E));
  uint32_t w[4];
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(E) == 4) return __uint_as_float(w[i]);
    else return i % 2 ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]);
  }
  // v[i] in the place of every element for which turned(i) holds
  template <typename F>
  __device__ __forceinline__ void put(const float *v, F turned) {
#pragma unroll
    for (int i = 0; i < kN; i += 4 / int(sizeof(E))) {
      if constexpr (sizeof(E) == 4) {
        w[i] = turned(i) ? __float_as_uint(v[i]) : w[i];
      } else {
        const uint32_t u = pack_bf2(v[i], v[i + 1]);
        const uint32_t keep = (turned(i) ? 0u : 0xffffu) | (turned(i + 1) ? 0u : 0xffff0000u);
        w[i / 2] = (w[i / 2] & keep) | (u & ~keep);
      }
    }
  }
};
template <typename E> struct Unaligned;
template <> struct Unaligned<uint16_t> { typedef uint32_t U __attribute__((ext_vector_type(4), aligned(2))); };
template <> struct Unaligned<float> { typedef uint32_t U __attribute__((ext_vector_type(4), aligned(4))); };

// The vector at p, of which n elements are there.
template <typename E>
__device__ __forceinline__ HeadVec<E> load_head(const E *p, int n) {
  HeadVec<E> v = {{0u, 0u, 0u, 0u}};
  if (n >= HeadVec<E>::kN) {
    const typename Unaligned<E>::U u = *(const LORA_GLOBAL typename Unaligned<E>::U *)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.w[i] = u[i];
  } else {
#pragma unroll
    for (int i = 0; i < HeadVec<E>::kN; ++i)
      if (i < n) {
        if constexpr (sizeof(E) == 4) v.w[i] = gload<uint32_t>(p + i);
        else v.w[i / 2] |= uint32_t(gload<uint16_t>(p + i)) << (i % 2 * 16);
      }
  }
  return v;
}
template <typename E>
__device__ __forceinline__ void store_head(E *p, const HeadVec<E> &v, int n, int by) {
  if (n >= HeadVec<E>::kN) {
    const typename Unaligned<E>::U u = {v.w[0], v.w[1], v.w[2], v.w[3]};
    LORA_GLOBAL typename Unaligned<E>::U *to = (LORA_GLOBAL typename Unaligned<E>::U *)p;
    if (by) {
      // (the compiler would make one of the two stores, and that an ordinary one)
      asm volatile("");
      __builtin_nontemporal_store(u, to);
      asm volatile("");
    } else {
      *to = u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < HeadVec<E>::kN; ++i)
      if (i < n) {
        if constexpr (sizeof(E) == 4) gstore(p + i, v.w[i]);
        else gstore(p + i, uint16_t(v.w[i / 2] >> (i % 2 * 16)));
      }
  }
}

// Dynamic LDS: the table [kTokens][rot_dim / 2], and for ROT_ANY a head for
// each slot, cols * 16 bytes.
template <typename E, int MODE, int kTokens>
__global__ __launch_bounds__(kRotaryThreads) void rotary_kernel(RotaryArgs a, int cols, int head_groups) {
  constexpr int kN = HeadVec<E>::kN;
  extern __shared__ __align__(16) char lds[];
  float2 *table = reinterpret_cast<float2 *>(lds);
  const int half = a.rot_dim / 2, D = a.head_dim;
  char *rows = lds + (kTokens * half * int(sizeof(float2)) + 15) / 16 * 16;
  const int slots = kRotaryThreads / cols, slot = threadIdx.x / cols, col = threadIdx.x % cols;
  const int64_t t0 = int64_t(blockIdx.x / head_groups) * kTokens;
  const int first = int(blockIdx.x % head_groups) * slots + slot, step = head_groups * slots;

  int pos[kTokens];
#pragma unroll
  for (int t = 0; t < kTokens; ++t) pos[t] = t0 + t < a.T ? gload<int>(a.positions + t0 + t) : -1;

  // where this lane's vectors lie in a head, and how much of them is there
  const bool pair = MODE == ROT_HALVES && col < half / kN;
  const int i0 = MODE == ROT_HALVES && !pair ? a.rot_dim + (col - half / kN) * kN : col * kN;
  const int n0 = D - i0;

  HeadVec<E> x0[kTokens], x1[kTokens];
  E *dst = nullptr;
  int64_t dst_token = 0;
  auto load = [&](int g) {
    // the slice of head g (few slices: a walk over all of them)
    const E *src = nullptr;
    int64_t src_token = 0;
    int start = 0;
    for (int s = 0; s < a.n_slices; ++s) {
      const lora_rotary_slice &v = a.s[s];
      if (g >= start) {
        src = static_cast<const E *>(v.src) + (g - start) * v.src_head;
        dst = static_cast<E *>(v.dst) + (g - start) * v.dst_head;
        src_token = v.src_token;
        dst_token = v.dst_token;
      }
      start += v.n_heads;
    }
#pragma unroll
    for (int t = 0; t < kTokens; ++t)
      if (pos[t] >= 0) {
        const E *p = src + (t0 + t) * src_token + i0;
        x0[t] = load_head(p, n0);
        if (pair) x1[t] = load_head(p + half, kN);
      }
  };
  const bool mine = slot < slots;
  // the first heads are on their way while the table is made
  if (mine && first < a.n_heads) load(first);
  for (int k = threadIdx.x; k < kTokens * half; k += kRotaryThreads) {
    const int t = kTokens == 1 ? 0 : k / half;
    int p = pos[0];
#pragma unroll
    for (int u = 1; u < kTokens; ++u) p = t == u ? pos[u] : p;
    table[k] = turn(max(p, 0), gload<double>(a.freq + (k - t * half)), a.mscale, a.sign);
  }
  lds_barrier();

  // all lanes of a workgroup go round as often as its first, which has the most heads
  for (int g = first; g - slot < a.n_heads; g += step) {
    const bool live = mine && g < a.n_heads;
    if (live && g != first) load(g);
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      const float2 *cs = table + t * half;
      if constexpr (MODE == ROT_ANY) {
        // the barriers are all lanes'
        if (t > 0 || g != first) lds_barrier();
        if (live && pos[t] >= 0)
          *reinterpret_cast<uint4 *>(rows + (slot * cols + col) * 16) = 
              make_uint4(x0[t].w[0], x0[t].w[1], x0[t].w[2], x0[t].w[3]);
        lds_barrier();
      }
      if (!live || pos[t] < 0) continue;
      E *p = dst + (t0 + t) * dst_token + i0;
      if (MODE == ROT_HALVES && pair) {
        float y0[kN], y1[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const float2 r = cs[i0 + i];
          const float u = x0[t].get(i), v = x1[t].get(i);
          y0[i] = u * r.x - v * r.y;
          y1[i] = v * r.x + u * r.y;
        }
        const auto all = [](int) { return true; };
        x0[t].put(y0, all);
        x1[t].put(y1, all);
        store_head(p + half, x1[t], kN, a.by);
      } else if (MODE == ROT_NEXT) {
        float y[kN];
#pragma unroll
        for (int i = 0; i < kN; i += 2) {
          const float2 r = cs[min((i0 + i) / 2, half - 1)];
          const float u = x0[t].get(i), v = x0[t].get(i + 1);
          y[i] = u * r.x - v * r.y;
          y[i + 1] = v * r.x + u * r.y;
        }
        x0[t].put(y, [&](int i) { return i0 + i < a.rot_dim; });
      } else if (MODE == ROT_ANY) {
        const E *row = reinterpret_cast<const E *>(rows + slot * cols * 16);
        float y[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int at = min(i0 + i, a.rot_dim - 1);
          const bool low = at < half;
          const float2 r = cs[low ? at : at - half];
          const E other = row[low ? at + half : at - half];
          float v;
          if constexpr (sizeof(E) == 4) v = other;
          else v = bf_to_f(other);
          y[i] = x0[t].get(i) * r.x + v * (low ? -r.y : r.y);
        }
        x0[t].put(y, [&](int i) { return i0 + i < a.rot_dim; });
      }
      store_head(p, x0[t], n0, a.by);
    }
  }
}

template <typename E, int MODE>
hipError_t launch_mode(const RotaryArgs &a, bool copy_rest, hipStream_t stream) {
  constexpr int kN = HeadVec<E>::kN;
  const int half = a.rot_dim / 2, rest = a.head_dim - a.rot_dim;
  // columns of a head that the call has to visit; in place those of the pairs
  int cols;
  if (MODE == ROT_HALVES) cols = half / kN + (copy_rest ? (rest + kN - 1) / kN : 0);
  else cols = ((copy_rest ? a.head_dim : a.rot_dim) + kN - 1) / kN;
  const int slots = kRotaryThreads / cols;
  const size_t rows = MODE == ROT_ANY ? size_t(slots) * cols * 16 : 0;
  // Few tokens: one a workgroup, and as many workgroups a token as its heads
  // fill.  Many: two, which share the table's work and have twice the loads in
  // flight.  40 bf16 heads of 128: 1000 tokens take 7.6 us with one and 8.0
  // with two, 2304 take 12.6 and 11.6, 16997 take 69 and 67 (72 with four).
  constexpr int kMany = 2;
  if (a.T >= 1536) {
    const size_t smem = (size_t(kMany) * half * sizeof(float2) + 15) / 16 * 16 + rows;
    rotary_kernel<E, MODE, kMany><<<dim3(uint32_t((a.T - 1) / kMany + 1)), kRotaryThreads, smem, stream>>>(a, cols, 1);
  } else {
    const size_t smem = (size_t(half) * sizeof(float2) + 15) / 16 * 16 + rows;
    const int groups = min((a.n_heads - 1) / slots + 1, 256);
    rotary_kernel<E, MODE, 1><<<dim3(uint32_t(a.T) * uint32_t(groups)), kRotaryThreads, smem, stream>>>(a, cols, groups);
  }
  return hipGetLastError();
}

template <typename E>
hipError_t launch_typed(const RotaryArgs &args, hipStream_t stream) {
  RotaryArgs a = args;
  // Values pass L2 by where a lane's neighbours write whole lines: 17k tokens of
  // 40 bf16 heads of 128 take 67 -> 64.5 us, of 10 fp32 ones 35.6 -> 29.0, 1000
  // tokens 7.8 -> 6.4; fewer or in place the same.  Heads of 80, halves of 80
  // bytes, would go from 28.7 to 39.3, and heads that begin inside a line alike.
  const int piece = (a.interleaved || a.rot_dim / 2 % HeadVec<E>::kN ? a.head_dim : a.rot_dim / 2) * int(sizeof(E));
  bool copy_rest = false;
  a.by = piece % 128 == 0;
  for (int s = 0; s < a.n_slices; ++s) {
    const lora_rotary_slice &v = a.s[s];
    copy_rest = copy_rest || v.src != v.dst;
    a.by = a.by && reinterpret_cast<uintptr_t>(v.dst) % 128 == 0 && v.dst_token * int(sizeof(E)) % 128 == 0 &&
           v.dst_head * int(sizeof(E)) % 128 == 0;
  }
  if (a.interleaved) return launch_mode<E, ROT_NEXT>(a, copy_rest, stream);
  if (a.rot_dim / 2 % HeadVec<E>::kN == 0) return launch_mode<E, ROT_HALVES>(a, copy_rest, stream);
  return launch_mode<E, ROT_ANY>(a, copy_rest, stream);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &args, int dtype, hipStream_t stream) {
  // a grid holds so many tokens; the rest in further launches
  constexpr int kMost = 1 << 24;
  const int64_t eb = dtype == LORA_BF16 ? 2 : 4;
  for (int64_t t = 0; t < args.T; t += kMost) {
    RotaryArgs a = args;
    a.positions += t;
    a.T = int(args.T - t < kMost ? args.T - t : kMost);
    for (int s = 0; s < a.n_slices; ++s) {
      a.s[s].src = static_cast<const char *>(a.s[s].src) + t * a.s[s].src_token * eb;
      a.s[s].dst = static_cast<char *>(a.s[s].dst) + t * a.s[s].dst_token * eb;
    }
    const hipError_t e = dtype == LORA_BF16 ? launch_typed<uint16_t>(a, stream) : launch_typed<float>(a, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace lora
