// The 8-bit base product y = (q W^T) scaled by token and channel.
//
// The channels are the rows of the matrix instruction's result and the tokens
// its columns, so that a lane holds four neighbouring channels of one token
// and stores them together.  Both operands have the sum's axis contiguous,
// which is the order in which v_mfma_i32_16x16x64_i8 takes them: a lane holds
// 16 consecutive values of one row.

#include <algorithm>
#include <type_traits>

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

// 16 bytes at any alignment: the five whole words around them (load), then
// moved down to their first byte (get).  One 16-byte load at an odd address
// takes the memory pipeline several times as long: 8 rows of 4095 through 4096
// channels 9.2 us this way and 15.3 that way.  No word is read that holds none
// of the bytes.
struct Words {
  i32x4 u;
  uint32_t e;
  __device__ __forceinline__ void load(const int8_t *p) {
    typedef int U __attribute__((ext_vector_type(4), aligned(4)));
    const uint32_t odd = uint32_t(reinterpret_cast<uintptr_t>(p)) & 3;
    u = *(const LORA_GLOBAL U *)(p - odd);
    e = *(const LORA_GLOBAL uint32_t *)(p - odd + (odd ? 16 : 12));
  }
  __device__ __forceinline__ i32x4 get(const int8_t *p) const {
    const uint32_t odd = uint32_t(reinterpret_cast<uintptr_t>(p));  // its last two bits count
    return i32x4{int(__builtin_amdgcn_alignbyte(u[1], u[0], odd)), int(__builtin_amdgcn_alignbyte(u[2], u[1], odd)),
                 int(__builtin_amdgcn_alignbyte(u[3], u[2], odd)), int(__builtin_amdgcn_alignbyte(e, u[3], odd))};
  }
};
__device__ __forceinline__ i32x4 load16(const int8_t *p) {
  Words w;
  w.load(p);
  return w.get(p);
}
// v moved down by `bytes` (16 or more: zeros).
__device__ __forceinline__ i32x4 move_down(const i32x4 &v, int bytes) {
  const int bits = min(bytes, 16) * 8, b = bits & 63;
  const uint64_t lo = uint32_t(v[0]) | uint64_t(uint32_t(v[1])) << 32, hi = uint32_t(v[2]) | uint64_t(uint32_t(v[3])) << 32;
  const uint64_t down = b ? hi << (64 - b) : 0;
  const uint64_t l = bits < 64 ? lo >> b | down : bits < 128 ? hi >> b : 0, h = bits < 64 ? hi >> b : 0;
  return i32x4{int(uint32_t(l)), int(uint32_t(l >> 32)), int(uint32_t(h)), int(uint32_t(h >> 32))};
}
// The 16 bytes at k of a row of d_in (16 or more) bytes, zeros past its end:
// read from further ahead where they would pass it, and moved down.
__device__ __forceinline__ int start_of(int k, int d_in) { return min(k, d_in - 16); }
__device__ __forceinline__ i32x4 load16_end(const int8_t *row, int k, int d_in) {
  const int start = start_of(k, d_in);
  return move_down(load16(row + start), k - start);
}

// 16 bytes of results, as aligned as one of them.
template <typename E> struct ResultVec;
template <> struct ResultVec<uint16_t> { typedef uint32_t U __attribute__((ext_vector_type(4), aligned(2))); };
template <> struct ResultVec<float> { typedef uint32_t U __attribute__((ext_vector_type(4), aligned(4))); };

// The first n elements of a vector to y; with BY, past the caches.
template <bool BY, typename E>
__device__ __forceinline__ void store_vec(E *y, const uint4 &v, int n) {
  typedef typename ResultVec<E>::U U;
  constexpr int kN = 16 / int(sizeof(E));
  if (n >= kN) {
    const U u = {v.x, v.y, v.z, v.w};
    LORA_GLOBAL U *p = (LORA_GLOBAL U *)y;
    if constexpr (BY)
      __builtin_nontemporal_store(u, p);
    else
      *p = u;
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i < n) {
        if constexpr (sizeof(E) == 2) gstore(y + i, uint16_t(w[i / 2] >> (i % 2 * 16)));
        else gstore(y + i, __uint_as_float(w[i]));
      }
  }
}

// 16 bytes from p, of which the first n (any whole number) are there: the rest are zeros.
__device__ __forceinline__ i32x4 load16(const int8_t *p, int n) {
  if (n >= 16) return load16(p);
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

// ------------------------------------------------- copies to LDS and waits --
// The sum's axis goes through LDS in stages of 128 values.  A row of a stage is
// 128 bytes, eight 16-byte pieces; piece c of row r lies at place c ^ (r & 7),
// so that eight lanes reading one piece of neighbouring rows meet every bank
// once.  A copy (eight rows) writes LDS in lane order, so the lanes take their
// global pieces in that order instead.
constexpr int kStage = 128;

// 16 bytes a lane from base + off straight to LDS at `lds` (wave-uniform) + 16 lane.
__device__ __forceinline__ void copy_to_lds(const int8_t *base, uint32_t off, uint32_t lds) {
  __builtin_amdgcn_global_load_lds((const LORA_GLOBAL void *)((const LORA_GLOBAL char *)base + off),
                                   (__attribute__((address_space(3))) void *)(uintptr_t)lds, 16, 0, 0);
}
// Waits as the compiler counts them (after one it adds none of its own for
// what came before), and the workgroup's barrier, which no memory access of
// the code around it crosses.
template <int kCopies>  // of this wave's copies, all but the last kCopies have landed
__device__ __forceinline__ void wait_copies() {
  static_assert(kCopies < 64, "");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (kCopies & 15) | (kCopies >> 4) << 14);
}
// At most `stages` stages of kCopies copies still on their way (a wave-uniform number; kMost at most).
template <int kCopies, int kMost>
__device__ __forceinline__ void wait_stages(int stages) {
  if constexpr (kMost == 0) {
    wait_copies<0>();
  } else {
    if (stages >= kMost)
      wait_copies<kCopies * kMost>();
    else
      wait_stages<kCopies, kMost - 1>(stages);
  }
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xc07f); }  // lgkmcnt(0)
__device__ __forceinline__ void meet() { asm volatile("s_barrier" ::: "memory"); }

// --------------------------------------------------------------- few rows --
//
// Up to 16 tokens and rows of any alignment: bound by reading the weights once.
// A workgroup takes 16 channels and all tokens, its eight waves an eighth of the
// sum's axis each, so that a weight of 4096 channels fills the chip and a CU has
// 16 waves of loads on their way.  Operands go straight to registers, four
// 64-value steps at a time while the four before are multiplied; only the last
// steps look where the rows end.  The waves' sums meet in LDS.  One row through
// 4096 x 4096 takes 5.4 us when rows are a multiple of 16 bytes, 7.6 when they
// are of 4095.
constexpr int kFewWaves = 8, kFewSteps = 4;

// The sums of 16 channels and 16 tokens, added over the waves, to y.
template <typename E>
__device__ __forceinline__ void store_few(const ProductArgs &a, const i32x4 *part, int stride, int o0, int t0) {
  const int lane = threadIdx.x % 64, t = t0 + lane % 16, o = o0 + lane / 16 * 4;
  i32x4 sum = part[lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) sum += part[w * stride + lane];
  if (t >= a.T || o >= a.d_out) return;
  const float sx = gload<float>(a.q_scale + t);
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = min(o + e, a.d_out - 1);
    v[e] = float(sum[e]) * sx * gload<float>(a.w_scale + c) + bias_of(a, c);
  }
  store_y(a, static_cast<E *>(a.y) + t * a.ldy, o, v);
}

template <typename E>
__global__ __launch_bounds__(64 * kFewWaves, 2) void product_few_kernel(ProductArgs a) {
  __shared__ i32x4 part[kFewWaves * 64];
  const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const int steps = (a.d_in + 63) / 64, each = (steps + kFewWaves - 1) / kFewWaves;
  const int begin = wave * each, end = min(begin + each, steps), whole = min(end, a.d_in / 64);
  const int o0 = blockIdx.x * 16, piece = lane / 16 * 16;
  // rows past the end: the last row again
  const int8_t *pw = a.W + int64_t(min(o0 + lane % 16, a.d_out - 1)) * a.ldw;
  const int8_t *px = a.q + int64_t(min(lane % 16, a.T - 1)) * a.ldq;
  i32x4 acc = {};
  i32x4 w[2][kFewSteps], x[2][kFewSteps];
  auto load = [&](int step, int set) {
#pragma unroll
    for (int u = 0; u < kFewSteps; ++u) {
      w[set][u] = load16(pw + piece + (step + u) * 64);
      x[set][u] = load16(px + piece + (step + u) * 64);
    }
  };
  auto multiply_set = [&](int set) {
#pragma unroll
    for (int u = 0; u < kFewSteps; ++u) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[set][u], x[set][u], acc, 0, 0, 0);
  };
  int k = begin;
  if (k + kFewSteps <= whole) {
    load(k, 0);
    for (; k + 3 * kFewSteps <= whole; k += 2 * kFewSteps) {
      load(k + kFewSteps, 1);
      multiply_set(0);
      load(k + 2 * kFewSteps, 0);
      multiply_set(1);
    }
    const bool two = k + 2 * kFewSteps <= whole;
    if (two) load(k + kFewSteps, 1);
    multiply_set(0);
    if (two) multiply_set(1);
    k += two ? 2 * kFewSteps : kFewSteps;
  }
  for (; k < end; ++k)
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(load16_end(pw, k * 64 + piece, a.d_in), load16_end(px, k * 64 + piece, a.d_in),
                                                acc, 0, 0, 0);
  part[wave * 64 + lane] = acc;
  lds_barrier();
  if (wave == 0) store_few<E>(a, part, 64, o0, 0);
}

template <typename E>
hipError_t launch_few(const ProductArgs &a, hipStream_t stream) {
  product_few_kernel<E><<<dim3(uint32_t((a.d_out - 1) / 16 + 1)), 64 * kFewWaves, 0, stream>>>(a);
  return hipGetLastError();
}

// Up to NT * 16 tokens and rows of whole 16-byte pieces.  Read as above, 64
// lanes would take 16 bytes of each of 16 rows, neighbours never side by side,
// at a quarter of the cache's rate: that is fine for the weights, read once, but
// with 64 rows q is four times their bytes (64 rows through 4096 x 4096: 11.9
// us).  Here each wave copies its stages to its own part of LDS in whole
// lines, one stage ahead, and needs no barrier before the sums meet: 7.9 us; 1
// row through 4096 x 1024 3.9 us instead of 4.8.
template <int NT>
struct FewShape {
  static constexpr int kRows = 16 + NT * 16, kCopies = kRows / 8, kBytes = kRows * kStage;  // of a wave's stage
  static constexpr int kLds = kFewWaves * 2 * kBytes;  // the sums take the same place afterwards
  static_assert(kLds <= kMaxLdsBytes && kFewWaves * NT * 1024 <= kLds && NT <= kFewWaves, "");
};
template <typename E, int NT>
__global__ __launch_bounds__(64 * kFewWaves, 2) void product_few_lines_kernel(ProductArgs a) {
  typedef FewShape<NT> S;
  extern __shared__ __align__(16) int8_t lds[];
  const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64);
  const int stages = (a.d_in + kStage - 1) / kStage, each = (stages + kFewWaves - 1) / kFewWaves;
  const int begin = wave * each, end = min(begin + each, stages);
  const int piece = (lane % 8) ^ (lane / 8), o0 = blockIdx.x * 16;
  int8_t *mine = lds + wave * 2 * S::kBytes;
  const uint32_t lds0 = uint32_t(uintptr_t((__attribute__((address_space(3))) int8_t *)mine));
  const int8_t *W = a.W + int64_t(o0) * a.ldw;
  uint32_t off[S::kCopies];  // two of W, then q's; rows past the end: the last row again
#pragma unroll
  for (int i = 0; i < S::kCopies; ++i)
    off[i] = (i < 2 ? uint32_t(min(i * 8 + lane / 8, a.d_out - 1 - o0)) * uint32_t(a.ldw)
                    : uint32_t(min((i - 2) * 8 + lane / 8, a.T - 1)) * uint32_t(a.ldq)) +
             piece * 16;
  auto copy = [&](int stage) {
    // pieces past the end of the rows are not read: the stage's first piece stands in (and is masked below)
    const uint32_t back = stage * kStage + piece * 16 < a.d_in ? 0u : piece * 16u;
#pragma unroll
    for (int i = 0; i < S::kCopies; ++i)
      copy_to_lds((i < 2 ? W : a.q) + stage * kStage, off[i] - back, lds0 + (stage & 1) * S::kBytes + i * 1024);
  };
  i32x4 acc[NT] = {};
  if (begin < end) copy(begin);
  if (begin + 1 < end) copy(begin + 1);
  for (int i = begin; i < end; ++i) {
    if (i + 1 < end)
      wait_copies<S::kCopies>();
    else
      wait_copies<0>();
    __builtin_amdgcn_sched_barrier(0);
    const int8_t *p = mine + (i & 1) * S::kBytes + lane % 16 * kStage;
    i32x4 w[2], x[2][NT];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int at = ((s * 4 + lane / 16) ^ (lane & 7)) * 16;
      w[s] = *reinterpret_cast<const i32x4 *>(p + at);
#pragma unroll
      for (int j = 0; j < NT; ++j) x[s][j] = *reinterpret_cast<const i32x4 *>(p + (16 + j * 16) * kStage + at);
    }
    wait_lds();  // the stage is read: its place may be written
    __builtin_amdgcn_sched_barrier(0);
    if (i + 2 < end) copy(i + 2);
    if (i == stages - 1) {
      // past the end of the sum's axis the weights count as zero
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool in = i * kStage + s * 64 + lane / 16 * 16 < a.d_in;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[s][e] = in ? w[s][e] : 0;
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s], x[s][j], acc[j], 0, 0, 0);
  }
  i32x4 *part = reinterpret_cast<i32x4 *>(lds);
  lds_barrier();  // every wave is done with its stages
#pragma unroll
  for (int j = 0; j < NT; ++j) part[(wave * NT + j) * 64 + lane] = acc[j];
  lds_barrier();
  if (wave < NT) store_few<E>(a, part + wave * 64, NT * 64, o0, wave * 16);
}

template <typename E, int NT>
hipError_t launch_few_lines(const ProductArgs &a, hipStream_t stream) {
  typedef FewShape<NT> S;
  const auto kernel = product_few_lines_kernel<E, NT>;
  static const bool ready = raise_lds_limit(reinterpret_cast<const void *>(kernel), S::kLds);
  (void)ready;
  kernel<<<dim3(uint32_t((a.d_out - 1) / 16 + 1)), 64 * kFewWaves, S::kLds, stream>>>(a);
  return hipGetLastError();
}

// ------------------------------------------------------------ large tiles --
//
// WM x WN waves of MT x NT blocks of v_mfma_i32_16x16x64_i8: MT * WM * 16
// channels x NT * WN * 16 tokens, with ST stages in LDS: stage i + ST is on its
// way while stages i + 1 .. lie ready or arrive and i is multiplied.  Within a
// stage the operands of one 64-value step are read from LDS while the step
// before is multiplied, across stages too, so the matrix unit waits for nothing
// but the one barrier of a stage.
//
// What bounds large tiles is power: four waves on every CU that only multiply
// random 8-bit numbers run at 1.79 GHz (3.68 POP/s) with 16 x 16 blocks and at
// 1.44 GHz (2.97 POP/s) with 32 x 32 ones, which move twice the sums.  So 16 x 16
// blocks, and the largest tile that fits the registers, which reads the fewest
// operands from LDS for each product: 256 x 256 by eight waves (2 x 4, 128 x 64
// each).  A stage of it is 2048 clocks of products; it takes 2444 when all
// operands are in L2 (four waves of 128 x 128, which read a third less from LDS
// but cannot fill each other's gaps: 2655) and about 2750 from memory, at 1.85
// GHz.  8192^3: 397 us, 2.77 POP/s; 16384 rows through 4096 x 4096: 207 us, 2.7
// POP/s, the rest being the tiles' first stages and stores (4 of 52 us a tile).
// c += a b^T on a 16 x 16 block, c kept where it is: given the choice, the
// compiler writes the sums elsewhere and moves 200 registers back each stage.
// It sees no matrix instruction here, so the waits that it would insert stand
// at the places that need them (settle, settled).
__device__ __forceinline__ void multiply(i32x4 &c, const i32x4 &a, const i32x4 &b) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
}
// Between vector instructions that write operands and the products that read them (2 wait states).
__device__ __forceinline__ void settle() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 3");
  __builtin_amdgcn_sched_barrier(0);
}
// Between the last products and reads of their sums (at most 19 wait states).
template <int M, int N>
__device__ __forceinline__ void settled(i32x4 (&c)[M][N]) {
  asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
  for (int m = 0; m < M; ++m)
#pragma unroll
    for (int j = 0; j < N; ++j) asm volatile("" : "+v"(c[m][j]));
}

template <typename E, int MT, int NT, int WM, int WN, int ST>
struct TileShape {
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int kO = MT * 16 * WM, kT = NT * 16 * WN;  // channels and tokens of a tile
  static constexpr int kCopyO = kO / 8 / kWaves, kCopyT = kT / 8 / kWaves;  // copies of a wave a stage
  static constexpr int kBytes = (kO + kT) * kStage;  // one stage
  static constexpr int kScales = ST * kBytes;  // then the scales and biases
  static constexpr int kLds = kScales + (2 * kO + kT) * 4;
  static_assert(MT % 2 == 0 && kLds <= kMaxLdsBytes, "");
  static_assert(ST >= 2 && (ST & (ST - 1)) == 0, "stages are found by their number's low bits");
  static_assert(kO % (8 * kWaves) == 0 && kT % (8 * kWaves) == 0, "every wave copies the same");
};

template <typename E, int MT, int NT, int WM, int WN, int ST, bool LINES>
__global__ __launch_bounds__(64 * WM * WN, 2) void product_tile_kernel(ProductArgs a, int tiles_o, int tiles_t) {
  typedef TileShape<E, MT, NT, WM, WN, ST> S;
  extern __shared__ __align__(16) int8_t lds[];
  const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64);
  // Workgroups go to the XCDs in turn.  Each XCD takes a contiguous eighth of
  // the tiles, in blocks of four token tiles by all channel tiles, so that the
  // 32 tiles it works on at a time are about 4 x 8 and share their operands
  // in its L2.
  const uint32_t tiles = gridDim.x, xcd = blockIdx.x % 8;
  const uint32_t tile = xcd * (tiles / 8) + min(xcd, tiles % 8) + blockIdx.x / 8;
  constexpr uint32_t kGroup = 4;
  const uint32_t group = tile / (kGroup * tiles_o), in_group = tile % (kGroup * tiles_o);
  const uint32_t high = min(kGroup, tiles_t - group * kGroup);
  const int o0 = int(in_group / high) * S::kO;
  const int64_t t0 = int64_t(group * kGroup + in_group % high) * S::kT;
  const int n_o = min(S::kO, a.d_out - o0), n_t = int(min(int64_t(S::kT), a.T - t0));

  const int n = (a.d_in + kStage - 1) / kStage;
  // this lane's pieces of W and of q (rows past the end: the last row again)
  const int8_t *W = a.W + int64_t(o0) * a.ldw, *q = a.q + t0 * a.ldq;
  const int piece = (lane % 8) ^ (lane / 8);
  constexpr int kCopies = S::kCopyO + S::kCopyT;
  uint32_t off[kCopies];
#pragma unroll
  for (int i = 0; i < S::kCopyO; ++i)
    off[i] = uint32_t(min((wave * S::kCopyO + i) * 8 + lane / 8, n_o - 1)) * uint32_t(a.ldw) + piece * 16;
#pragma unroll
  for (int i = 0; i < S::kCopyT; ++i)
    off[S::kCopyO + i] = uint32_t(min((wave * S::kCopyT + i) * 8 + lane / 8, n_t - 1)) * uint32_t(a.ldq) + piece * 16;
  const uint32_t lds0 = uint32_t(uintptr_t((__attribute__((address_space(3))) int8_t *)lds));

  auto copy = [&](int i, int stage, uint32_t back) {
    const uint32_t at = lds0 + (stage & (ST - 1)) * S::kBytes;
    if (i < S::kCopyO)
      copy_to_lds(W + stage * kStage, off[i] - back, at + (wave * S::kCopyO + i) * 1024);
    else
      copy_to_lds(q + stage * kStage, off[i] - back, at + S::kO * kStage + (wave * S::kCopyT + i - S::kCopyO) * 1024);
  };
  // pieces past the end of the rows are not read: the stage's first piece stands in (and is masked below)
  auto back_of = [&](int stage) -> uint32_t { return stage * kStage + piece * 16 < a.d_in ? 0u : piece * 16u; };
  // Rows of any alignment go through registers: a stage's pieces are read a
  // stage before they are written to LDS, where they are moved to their place.
  Words held[LINES ? 1 : kCopies];
  auto row_of = [&](int i) { return (i < S::kCopyO ? W : q) + (off[i] - piece * 16); };
  auto fetch = [&](Words &w, int i, int stage, bool whole) {
    const int k = stage * kStage + piece * 16;
    w.load(row_of(i) + (whole ? k : start_of(k, a.d_in)));
  };
  auto put = [&](const Words &w, int i, int stage, bool whole) {
    const int at = (stage & (ST - 1)) * S::kBytes +
                   (i < S::kCopyO ? (wave * S::kCopyO + i) * 1024 : S::kO * kStage + (wave * S::kCopyT + i - S::kCopyO) * 1024);
    i32x4 *to = reinterpret_cast<i32x4 *>(lds + at + lane * 16);
    if (whole) {
      *to = w.get(row_of(i));  // a multiple of 16 further on
    } else {
      const int k = min(stage, n - 1) * kStage + piece * 16, start = start_of(k, a.d_in);
      *to = move_down(w.get(row_of(i) + start), k - start);
    }
  };

  const int wm = wave / WN, wn = wave % WN;
  const int8_t *lw = lds + (wm * MT * 16 + lane % 16) * kStage, *lx = lds + (S::kO + wn * NT * 16 + lane % 16) * kStage;
  i32x4 fw[2][MT], fx[2][NT];
  i32x4 acc[MT][NT] = {};
  auto place = [&](int stage, int s) { return (stage & (ST - 1)) * S::kBytes + (((s * 4 + lane / 16) ^ (lane & 7)) * 16); };
  auto read = [&](int k, int p, int s) {
    if (k < MT)
      fw[s][k] = *reinterpret_cast<const i32x4 *>(lw + p + k * 16 * kStage);
    else
      fx[s][k - MT] = *reinterpret_cast<const i32x4 *>(lx + p + (k - MT) * 16 * kStage);
  };

  float *s_o = reinterpret_cast<float *>(lds + S::kScales), *b_o = s_o + S::kO, *s_t = b_o + S::kO;
  float scale_o[S::kO / S::kThreads + 1], scale_t[S::kT / S::kThreads + 1], bias[S::kO / S::kThreads + 1];
#pragma unroll
  for (int i = 0; i * S::kThreads < S::kO; ++i) {
    const int o = o0 + min(tid + i * S::kThreads, n_o - 1);
    scale_o[i] = gload<float>(a.w_scale + o);
    bias[i] = bias_of(a, o);
  }
#pragma unroll
  for (int i = 0; i * S::kThreads < S::kT; ++i)
    scale_t[i] = gload<float>(a.q_scale + t0 + min(tid + i * S::kThreads, n_t - 1));
  if constexpr (LINES) {
    for (int st = 0; st < min(n, ST); ++st) {
      const uint32_t back = back_of(st);
#pragma unroll
      for (int i = 0; i < kCopies; ++i) copy(i, st, back);
    }
  } else {
    static_assert(LINES || ST == 2, "a third stage is in registers");
    Words first[kCopies];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) fetch(first[i], i, 0, false);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) fetch(held[i], i, min(1, n - 1), false);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) put(first[i], i, 0, false);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) put(held[i], i, 1, false);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) fetch(held[i], i, min(2, n - 1), false);
  }
#pragma unroll
  for (int i = 0; i * S::kThreads < S::kO; ++i)
    if (tid + i * S::kThreads < S::kO) s_o[tid + i * S::kThreads] = scale_o[i], b_o[tid + i * S::kThreads] = bias[i];
#pragma unroll
  for (int i = 0; i * S::kThreads < S::kT; ++i)
    if (tid + i * S::kThreads < S::kT) s_t[tid + i * S::kThreads] = scale_t[i];
  if constexpr (LINES) wait_stages<kCopies, ST - 1>(n - 1);
  wait_lds();
  meet();
#pragma unroll
  for (int k = 0; k < MT + NT; ++k) read(k, place(0, 0), 0);

  // A stage is two steps of 64 values.  The first step's products go with the
  // reads of the second's operands.  Then all waves meet: the stage has been
  // read by all, so the copies of stage i + ST may take its place, and stage i +
  // 1 has landed for all, so the second step's products go with the reads of
  // its first operands.  The order of issue is the order written.
  constexpr int kReads = MT + NT, kMul = MT * NT;
  constexpr int kCopyEach = kMul / 2 > kCopies ? kMul / 2 / kCopies : 1;
  constexpr int kReadAt = kMul / 2 + kReads <= kMul ? kMul / 2 : kMul - kReads;
  static_assert(kReads <= kMul && kCopies <= kMul, "a read or a copy goes with a product");
  auto stage = [&](int i, auto more, auto masked) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      wait_lds();
      if (s == 1 && !masked) {
        // what may still be on its way: the stages after the next one
        if constexpr (LINES && more)
          wait_copies<kCopies *(ST - 2)>();
        else if constexpr (LINES)
          wait_stages<kCopies, ST - 2>(n - 2 - i);
        meet();
      }
      const int p = place(s ? i + 1 : i, s ^ 1);
      const uint32_t back = LINES && more && s == 1 ? back_of(i + ST) : 0;
      if constexpr (LINES && masked) {
        // past the end of the sum's axis q counts as zero
        const bool in = i * kStage + s * 64 + lane / 16 * 16 < a.d_in;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) fx[s][j][e] = in ? fx[s][j][e] : 0;
        settle();
      }
#pragma unroll
      for (int t = 0; t < kMul; ++t) {
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (LINES) {
          if (more && s == 1 && t % kCopyEach == 0 && t / kCopyEach < kCopies) copy(t / kCopyEach, i + ST, back);
        } else if (!masked && s == 1 && t % kCopyEach == 0 && t / kCopyEach < kCopies) {
          const int c = t / kCopyEach;
          put(held[c], c, i + ST, more);
          fetch(held[c], c, more ? i + ST + 1 : min(i + ST + 1, n - 1), more);
        }
        if (s == 0 && t < kReads) read(t, p, 1);
        if (!masked && s == 1 && t >= kReadAt && t < kReadAt + kReads) read(t - kReadAt, p, 0);
        __builtin_amdgcn_sched_barrier(0);
        multiply(acc[t / NT][t % NT], fw[s][t / NT], fx[s][t % NT]);
      }
    }
  };
  int i = 0;
  // (in registers: `more` as long as the stage to be read is a whole one)
  for (; i < (LINES ? n - ST : n - ST - 2); ++i) stage(i, std::true_type{}, std::false_type{});
  for (; i < n - 1; ++i) stage(i, std::false_type{}, std::false_type{});
  stage(i, std::false_type{}, std::true_type{});
  settled(acc);

  // Results leave from registers.  A lane has four channels of a token in each
  // block, its neighbours 16 lanes on the next four: in bf16 two blocks change
  // places between such neighbours, so that each has eight of one block, and
  // a store is 16 bytes a lane and 64 a token.  Whole tiles go further: the lanes
  // of tokens 0..7 and 8..15 change their second halves, and a store writes a
  // line of 128 bytes of eight tokens (65536 rows through 1280 x 1280 114 -> 104
  // us, 16997 through 4096 x 4096 235 -> 226).  Elsewhere a token's stores follow
  // one another, so that its lines fill up in L2.
  constexpr int kVec = 16 / int(sizeof(E));
  float4 sw[MT], b[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int o = (wm * MT + m) * 16 + lane / 16 * 4;
    sw[m] = *reinterpret_cast<const float4 *>(s_o + o);
    b[m] = *reinterpret_cast<const float4 *>(b_o + o);
  }
  auto result = [&](int m, int j, float sx) -> uint4 {
    float v[kVec];
#pragma unroll
    for (int k = 0; k < kVec / 4; ++k) {
      const i32x4 &c = acc[m + k][j];
      v[k * 4] = float(c[0]) * sx * sw[m + k].x + b[m + k].x;
      v[k * 4 + 1] = float(c[1]) * sx * sw[m + k].y + b[m + k].y;
      v[k * 4 + 2] = float(c[2]) * sx * sw[m + k].z + b[m + k].z;
      v[k * 4 + 3] = float(c[3]) * sx * sw[m + k].w + b[m + k].w;
    }
    if constexpr (kVec == 8) {
      const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf2(v[0], v[1]), pack_bf2(v[4], v[5]), false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf2(v[2], v[3]), pack_bf2(v[6], v[7]), false, false);
      return make_uint4(lo[0], hi[0], lo[1], hi[1]);
    }
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  };
  const int o_lane = wm * MT * 16 + (kVec == 8 ? lane / 16 % 2 * 16 + lane / 32 * 8 : lane / 16 * 4);
  constexpr int kStep = kVec / 4, kLine = 2 * kStep;  // blocks of 64 bytes of a token, and of 128
  // Block m of token block j (and kStep - 1 more), 64 bytes a token.
  auto store_half = [&](int m, int j, float sx, auto by) {
    E *y = static_cast<E *>(a.y) + (t0 + (wn * NT + j) * 16 + lane % 16) * a.ldy + o0;
    store_vec<decltype(by)::value>(y + o_lane + m * 16, result(m, j, sx), kVec);
  };
  // ... and as many again, a line of eight tokens to each store.
  const bool low = lane % 16 < 8;
  auto store_line = [&](int m, int j, float sx, auto by) {
    E *y = static_cast<E *>(a.y) + (t0 + (wn * NT + j) * 16 + lane % 8) * a.ldy + o0 + o_lane + (low ? 0 : kStep * 16);
    const uint4 p = result(m, j, sx), q = result(m + kStep, j, sx);
    auto move = [&](uint32_t of_p, uint32_t of_q) {
      return uint32_t(__builtin_amdgcn_update_dpp(0, int(low ? of_q : of_p), 0x128, 0xf, 0xf, false));  // row_ror:8
    };
    const uint4 x = make_uint4(move(p.x, q.x), move(p.y, q.y), move(p.z, q.z), move(p.w, q.w));
    store_vec<decltype(by)::value>(
        y + m * 16, make_uint4(low ? p.x : x.x, low ? p.y : x.y, low ? p.z : x.z, low ? p.w : x.w), kVec);
    store_vec<decltype(by)::value>(
        y + 8 * a.ldy + m * 16, make_uint4(low ? x.x : q.x, low ? x.y : q.y, low ? x.z : q.z, low ? x.w : q.w), kVec);
  };
  // The blocks of a whole tile.  Where a wave's are no whole number of lines, one
  // line is half its and half the next wave's.  The halves of a 192-channel tile
  // still go past L2 with the rest, although memory then writes 1.04 to 1.1 times
  // the results: 37709 rows through 384 x 576 17.9 us, 58400 through 1024 x 384
  // 28.8; all as half lines, 1.3 times the results, 19.8 and 31.1; these halves
  // through L2, not a byte too many, 17.6 and 32.3 (and 16741 through 128 x 576
  // 7.9 against 7.1).  A 64-channel tile has nothing but halves: through L2, at
  // the same time, 64 rows through 4096 x 14336 write 1792 KiB, not 2290.
  auto store_whole = [&](auto first_half, auto by) {
    constexpr bool kOdd = MT % kLine != 0, kFirst = kOdd && decltype(first_half)::value;
    constexpr std::integral_constant<bool, decltype(by)::value && (MT > kStep)> by_half{};
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float sx = s_t[(wn * NT + j) * 16 + lane % 16];
      if constexpr (kFirst) store_half(0, j, sx, by_half);
#pragma unroll
      for (int m = kFirst ? kStep : 0; m + kLine <= MT; m += kLine) store_line(m, j, sx, by);
      if constexpr (kOdd && !kFirst) store_half(MT - kStep, j, sx, by_half);
    }
  };
  auto store_part = [&] {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int tt = (wn * NT + j) * 16 + lane % 16;
      const float sx = s_t[tt];
      E *y = static_cast<E *>(a.y) + (t0 + tt) * a.ldy + o0;
#pragma unroll
      for (int m = 0; m < MT; m += kStep) {
        const int oo = o_lane + m * 16;
        const uint4 out = result(m, j, sx);
        if (tt < n_t && oo < n_o) store_vec<false>(y + oo, out, n_o - oo);
      }
    }
  };
  if (n_o < S::kO || n_t < S::kT) {
    store_part();
    return;
  }
  auto store = [&](auto by) {
    if (MT % kLine != 0 && wm % 2 != 0)
      store_whole(std::true_type{}, by);
    else
      store_whole(std::false_type{}, by);
  };
  if (a.y_by) {
    asm volatile("");
    store(std::true_type{});
    asm volatile("");  // the compiler would make one of this and what follows, with ordinary stores
  } else {
    store(std::false_type{});
  }
}

template <typename E, int MT, int NT, int WM, int WN, int ST, bool LINES = true>
hipError_t launch_tiles(const ProductArgs &a, hipStream_t stream) {
  typedef TileShape<E, MT, NT, WM, WN, ST> S;
  const auto kernel = product_tile_kernel<E, MT, NT, WM, WN, ST, LINES>;
  static const bool ready = raise_lds_limit(reinterpret_cast<const void *>(kernel), S::kLds);
  (void)ready;
  const int tiles_o = (a.d_out + S::kO - 1) / S::kO;
  const int tiles_t = (a.T - 1) / S::kT + 1;
  const int64_t tiles = int64_t(tiles_o) * tiles_t;
  kernel<<<dim3(uint32_t(tiles)), S::kThreads, S::kLds, stream>>>(a, tiles_o, tiles_t);
  return hipGetLastError();
}

// The tile shapes and what a tile of n stages costs, in microseconds: when its
// CU has no other tile, and when the CU is full (so many tiles at once).  Large
// tiles move the fewest bytes for each product, small ones fill more CUs.
// Measured, with the shapes in their order here:
//                              256x256 192x256 128x128 128x128 128x64 64x64 128x160
//   512 rows,  4096 -> 4096       39.8    34.0    22.7    18.1   13.0  16.2    24.0
//   512 rows,  4096 -> 14336      40.4    34.0    28.9    34.8   43.1  44.5    35.7
//   2304 rows, 4096 -> 4096       40.6    35.6    49.3    50.5   55.2  58.2    37.5
//   2304 rows, 14336 -> 4096       157     141     175     157    173   202     121
//   2304 rows, 4096 -> 14336       100     113     118     142    178   202     125
//   16997 rows, 4096 -> 4096       239     242     258     299    376   424     251
struct TileCost {
  int o, t, at_once;
  float alone, full, once;  // per stage, per stage with a full CU, per tile
};
constexpr TileCost kTileCosts[] = {
    {256, 256, 1, 1.10f, 1.45f, 6.0f}, {192, 256, 1, 0.88f, 1.20f, 5.0f}, {128, 128, 2, 0.60f, 0.82f, 3.2f},
    {128, 128, 1, 0.48f, 0.48f, 3.0f}, {128, 64, 1, 0.33f, 0.33f, 2.5f},  {64, 64, 2, 0.19f, 0.45f, 3.0f},
    {128, 160, 2, 0.75f, 1.13f, 3.2f},
};

// The shape of the least cost, among those whose bit is set in `among`.
int choose_tile(const ProductArgs &a, unsigned among, double &least) {
  const int64_t cus = cu_count(), n = (a.d_in + kStage - 1) / kStage;
  int best = -1;
  for (int k = 0; k < int(sizeof(kTileCosts) / sizeof(kTileCosts[0])); ++k) {
    if (!(among >> k & 1)) continue;
    const TileCost &c = kTileCosts[k];
    const int64_t tiles = int64_t((a.d_out - 1) / c.o + 1) * ((a.T - 1) / c.t + 1);
    const int64_t rounds = tiles / (cus * c.at_once), rest = tiles % (cus * c.at_once);
    double us = rounds * double(n * c.full + c.once);
    // one to a CU, tiles slow down with the number of CUs at work (power)
    const double busy = c.at_once == 1 ? double(rest) / cus : rest > cus;
    if (rest) us += n * (c.alone + (c.full - c.alone) * busy) + c.once;
    if (best < 0 || us < least) best = k, least = us;
  }
  return best;
}

// The rows of whole rounds of one of the two large shapes, if these and the
// rest, in a launch of its own (2 us), cost 7% less than `least` or better (the
// costs are good to some 5%); else 0.
int split_rows(const ProductArgs &a, double least) {
  const int64_t cus = cu_count(), n = (a.d_in + kStage - 1) / kStage;
  int first = 0;
  least *= 0.93;
  for (int k = 0; k < 2; ++k) {
    const TileCost &c = kTileCosts[k];
    const int64_t across = (a.d_out - 1) / c.o + 1, down = (a.T - 1) / c.t + 1;
    const int64_t rounds = across * down / cus, rows = rounds * cus / across * c.t;
    if (rounds == 0 || rows == 0 || rows >= a.T) continue;
    ProductArgs rest = a;
    rest.T = a.T - int(rows);
    double us = 0;
    choose_tile(rest, ~0u, us);
    us += rounds * double(n * c.full + c.once) + 2;
    if (us < least) least = us, first = int(rows);
  }
  return first;
}

// What the kernel for few rows costs, likewise: a wave's stages, in as many
// rounds as its workgroups fill the chip (two on a CU up to 16 rows).  64 rows
// through 4096 x 4096 take 7.9 us with it and 9.3 with 64 x 64 tiles, through
// 14336 x 4096 22.7 and 36.8, through 4096 x 14336, whose channels make it read
// the rows 896 times, 29.5 and 17.5.
double cost_of_few(const ProductArgs &a) {
  const int each = ((a.d_in + kStage - 1) / kStage + kFewWaves - 1) / kFewWaves, nt = (a.T + 15) / 16;
  const double stage = nt <= 1 ? 0.75 : nt <= 2 ? 0.9 : 1.3, at_once = nt <= 1 ? 2 : 1;
  return std::max(1.0, ((a.d_out - 1) / 16 + 1) / (at_once * cu_count())) * (2.2 + stage * each);
}

template <typename E>
hipError_t launch_typed(const ProductArgs &a, hipStream_t stream) {
  const ProductChoice c = choose_product(a);
  if (c.first > 0) {
    ProductArgs b = a;
    b.T = c.first;
    hipError_t e = launch_typed<E>(b, stream);
    if (e != hipSuccess) return e;
    b = a;
    b.q += c.first * b.ldq;
    b.q_scale += c.first;
    b.y = static_cast<E *>(b.y) + c.first * b.ldy;
    b.T -= c.first;
    return launch_typed<E>(b, stream);
  }
  switch (c.kernel) {
    case PRODUCT_TILE: return launch_tiles<E, 8, 4, 2, 4, 2>(a, stream);
    case PRODUCT_TILE + 1: return launch_tiles<E, 6, 4, 2, 4, 2>(a, stream);
    case PRODUCT_TILE + 2: return launch_tiles<E, 4, 4, 2, 2, 2>(a, stream);
    case PRODUCT_TILE + 3: return launch_tiles<E, 4, 4, 2, 2, 4>(a, stream);
    case PRODUCT_TILE + 4: return launch_tiles<E, 4, 2, 2, 2, 4>(a, stream);
    case PRODUCT_TILE + 5: return launch_tiles<E, 2, 2, 2, 2, 4>(a, stream);
    case PRODUCT_TILE + 6: return launch_tiles<E, 4, 5, 2, 2, 2>(a, stream);
    case PRODUCT_FEW_LINES: return launch_few_lines<E, 1>(a, stream);
    case PRODUCT_FEW_LINES + 1: return launch_few_lines<E, 2>(a, stream);
    case PRODUCT_FEW_LINES + 2: return launch_few_lines<E, 4>(a, stream);
    case PRODUCT_FEW: return launch_few<E>(a, stream);
    case PRODUCT_ROWS_128: return launch_tiles<E, 4, 4, 2, 2, 2, false>(a, stream);
    case PRODUCT_ROWS_64: return launch_tiles<E, 2, 2, 2, 2, 2, false>(a, stream);
    default: break;
  }
  const dim3 grid((a.d_out + kAnyTile - 1) / kAnyTile, (a.T + kAnyTile - 1) / kAnyTile);
  product_any_kernel<E><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

ProductChoice choose_product(const ProductArgs &a) {
  const bool lines = aligned16(a.q) && aligned16(a.W) && a.ldq % 16 == 0 && a.ldw % 16 == 0 && a.d_in % 16 == 0;
  const bool near = a.ldq <= (1 << 22) && a.ldw <= (1 << 22);  // a tile's rows within 32-bit offsets
  double us = 0;
  if (near && lines) {
    const int tile = choose_tile(a, ~0u, us);
    // Whole rounds of one shape first and the rest, which would leave most CUs
    // idle in a last round, by itself: 16997 rows through 4096 x 4096, 4.2
    // rounds of 256 x 256 tiles, 228 us instead of 243, through 4096 x 1024 62
    // instead of 71.
    const int first = split_rows(a, us);
    if (first > 0) return {PRODUCT_TILE + tile, first};
    if (a.T <= 64 && cost_of_few(a) < us) return {PRODUCT_FEW_LINES + (a.T <= 16 ? 0 : a.T <= 32 ? 1 : 2), 0};
    return {PRODUCT_TILE + tile, 0};
  }
  if (a.d_in >= 16 && a.T <= 16) return {PRODUCT_FEW, 0};
  if (a.d_in >= 16 && near) return {choose_tile(a, 1u << 2 | 1u << 5, us) == 2 ? PRODUCT_ROWS_128 : PRODUCT_ROWS_64, 0};
  return {PRODUCT_ANY, 0};
}

hipError_t launch_product(const ProductArgs &args, int dtype, hipStream_t stream) {
  // what a launch may hold, at one thread for every 16 results at least
  constexpr int kMostT = 1 << 18, kMostO = 1 << 17;
  const int64_t eb = dtype == LORA_BF16 ? 2 : 4;
  // Results pass L2 by where every row begins on a whole line, and the operands
  // that other tiles share stay in: 65536 rows through 1280 x 1280 128 -> 105 us,
  // through 640 x 128 26 -> 20, 2304 rows through 14336 x 4096 112 -> 105, 1024
  // rows through 4096 x 4096 19.8 -> 19.0; fewer take the same.  Rows that begin
  // inside a line would go out in parts (65536 x 1280 through 1283 channels 168
  // -> 202).
  const int y_by = reinterpret_cast<uintptr_t>(args.y) % 128 == 0 && args.ldy * eb % 128 == 0;
  for (int64_t t = 0; t < args.T; t += kMostT)
    for (int64_t o = 0; o < args.d_out; o += kMostO) {
      ProductArgs a = args;
      a.y_by = y_by;
      a.q += t * a.ldq;
      a.q_scale += t;
      a.W += o * a.ldw;
      a.w_scale += o;
      if (a.bias) a.bias += o;
      a.y = static_cast<char *>(a.y) + (t * a.ldy + o) * eb;
      a.T = int(std::min<int64_t>(kMostT, args.T - t));
      a.d_out = int(std::min<int64_t>(kMostO, args.d_out - o));
      const hipError_t e = dtype == LORA_BF16 ? launch_typed<uint16_t>(a, stream) : launch_typed<float>(a, stream);
      if (e != hipSuccess) return e;
    }
  return hipSuccess;
}

}  // namespace lora
