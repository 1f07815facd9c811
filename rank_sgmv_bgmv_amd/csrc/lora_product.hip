// The 8-bit base product y = (q W^T) scaled by token and channel.
//
// The channels are the rows of the matrix instruction's result and the tokens
// its columns, so that a lane holds four neighbouring channels of one token
// and stores them together.  Both operands have the sum's axis contiguous,
// which is the order in which v_mfma_i32_16x16x64_i8 takes them: a lane holds
// 16 consecutive values of one row.

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

// 16 bytes from p, of which the first n (any whole number) are there: the rest are zeros.
__device__ __forceinline__ i32x4 load16(const int8_t *p, int n) {
  typedef int i32x4u __attribute__((ext_vector_type(4), aligned(1)));
  if (n >= 16) return *(const LORA_GLOBAL i32x4u *)p;
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

// ------------------------------------------------------------ large tiles --
//
// MT * 64 channels x NT * 64 tokens by four waves (2 x 2, each MT x NT blocks
// of v_mfma_i32_32x32x32_i8).  The sum's axis goes in stages of 128 values,
// copied to LDS without passing registers, two stages in LDS: stage i + 2 is on
// its way while stage i + 1 lies ready and i is multiplied.  Within a stage
// the operands of one 32-value step are read from LDS while the step before
// is multiplied, across stages too, so the matrix unit waits for nothing but
// the one barrier of a stage.
//
// A row of a stage is 128 bytes, eight 16-byte pieces; piece c of row r lies
// at place c ^ (r & 7), so that eight lanes reading one piece of neighbouring
// rows meet every bank once.  The copy writes LDS in lane order, so the lanes
// take their global pieces in that order instead.
typedef int i32x16 __attribute__((ext_vector_type(16)));
constexpr int kStage = 128;

// 16 bytes a lane from base + off straight to LDS at `lds` (wave-uniform) + 16 lane.
__device__ __forceinline__ void copy_to_lds(const int8_t *base, uint32_t off, uint32_t lds) {
  __builtin_amdgcn_global_load_lds((const LORA_GLOBAL void *)((const LORA_GLOBAL char *)base + off),
                                   (__attribute__((address_space(3))) void *)(uintptr_t)lds, 16, 0, 0);
}
// Every copy of this wave has landed and every LDS read has returned, for all waves.
__device__ __forceinline__ void stage_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <typename E, int MT, int NT>
struct TileShape {
  static constexpr int kO = MT * 64, kT = NT * 64;   // channels and tokens of a tile
  static constexpr int kBytes = (kO + kT) * kStage;  // one stage
  // results on their way out: up to 256 bytes of channels of each of a wave's tokens
  static constexpr int kOutM = MT * 32 * int(sizeof(E)) <= 256 ? MT : 256 / (32 * int(sizeof(E)));
  static constexpr int kOutRow = kOutM * 32 * int(sizeof(E)), kOutPitch = kOutRow + 16;
  static constexpr int kOut = 4 * NT * 32 * kOutPitch;
  static constexpr int kScales = 2 * kBytes > kOut ? 2 * kBytes : kOut;  // then the scales and biases
  static constexpr int kLds = kScales + (2 * kO + kT) * 4;
  static_assert(MT % kOutM == 0 && kLds <= kMaxLdsBytes, "");
};

template <typename E, int MT, int NT>
__global__ __launch_bounds__(256, 1) void product_tile_kernel(ProductArgs a, int tiles_o) {
  typedef TileShape<E, MT, NT> S;
  extern __shared__ __align__(16) int8_t lds[];
  const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64);
  const int o0 = int(blockIdx.x) % tiles_o * S::kO;
  const int64_t t0 = int64_t(int(blockIdx.x) / tiles_o) * S::kT;
  const int n_o = min(S::kO, a.d_out - o0), n_t = int(min(int64_t(S::kT), a.T - t0));

  // this lane's pieces: 2 MT rows of W and 2 NT of q a stage (rows past the end: the last row again)
  const int8_t *W = a.W + int64_t(o0) * a.ldw, *q = a.q + t0 * a.ldq;
  const int piece = (lane % 8) ^ (lane / 8);
  uint32_t off[2 * (MT + NT)];
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i)
    off[i] = uint32_t(min((wave * 2 * MT + i) * 8 + lane / 8, n_o - 1)) * uint32_t(a.ldw) + piece * 16;
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i)
    off[2 * MT + i] = uint32_t(min((wave * 2 * NT + i) * 8 + lane / 8, n_t - 1)) * uint32_t(a.ldq) + piece * 16;
  const uint32_t lds0 = uint32_t(uintptr_t((__attribute__((address_space(3))) int8_t *)lds));

  auto copy = [&](int i, int stage, uint32_t back) {
    const uint32_t at = lds0 + (stage & 1) * S::kBytes;
    if (i < 2 * MT)
      copy_to_lds(W + stage * kStage, off[i] - back, at + (wave * 2 * MT + i) * 1024);
    else
      copy_to_lds(q + stage * kStage, off[i] - back, at + S::kO * kStage + (wave * 2 * NT + i - 2 * MT) * 1024);
  };
  // pieces past the end of the rows are not read: the stage's first piece stands in (and is masked below)
  auto back_of = [&](int stage) -> uint32_t { return stage * kStage + piece * 16 < a.d_in ? 0u : piece * 16u; };

  const int wm = wave / 2, wn = wave % 2;
  const int8_t *lw = lds + (wm * MT * 32 + lane % 32) * kStage, *lx = lds + (S::kO + wn * NT * 32 + lane % 32) * kStage;
  i32x4 fw[2][MT], fx[2][NT];
  i32x16 acc[MT][NT] = {};
  auto read = [&](int stage, int s, int set) {
    const int p = (stage & 1) * S::kBytes + (((s * 2 + lane / 32) ^ (lane & 7)) * 16);
#pragma unroll
    for (int i = 0; i < MT; ++i) fw[set][i] = *reinterpret_cast<const i32x4 *>(lw + p + i * 32 * kStage);
#pragma unroll
    for (int j = 0; j < NT; ++j) fx[set][j] = *reinterpret_cast<const i32x4 *>(lx + p + j * 32 * kStage);
  };

  const int n = (a.d_in + kStage - 1) / kStage;
  for (int st = 0; st < min(n, 2); ++st) {
    const uint32_t back = back_of(st);
#pragma unroll
    for (int i = 0; i < 2 * (MT + NT); ++i) copy(i, st, back);
  }
  float *s_o = reinterpret_cast<float *>(lds + S::kScales), *b_o = s_o + S::kO, *s_t = b_o + S::kO;
  for (int i = tid; i < S::kO; i += 256) {
    const int o = o0 + min(i, n_o - 1);
    s_o[i] = gload<float>(a.w_scale + o);
    b_o[i] = bias_of(a, o);
  }
  for (int i = tid; i < S::kT; i += 256) s_t[i] = gload<float>(a.q_scale + t0 + min(i, n_t - 1));
  stage_barrier();
  read(0, 0, 0);

  auto stage = [&](int i, auto more, auto masked) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      uint32_t back = 0;
      if (s == 3) {
        stage_barrier();
        if constexpr (more) back = back_of(i + 2);
      }
      read(s == 3 ? i + 1 : i, (s + 1) & 3, (s + 1) & 1);
      if constexpr (masked) {
        // past the end of the sum's axis q counts as zero
        const bool in = i * kStage + s * 32 + lane / 32 * 16 < a.d_in;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) fx[s & 1][j][e] = in ? fx[s & 1][j][e] : 0;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          if constexpr (more) {
            constexpr int kCopies = 2 * (MT + NT), kMul = MT * NT;
            if (s == 3)
              for (int c = (m * NT + j) * kCopies / kMul; c < (m * NT + j + 1) * kCopies / kMul; ++c) copy(c, i + 2, back);
          }
          acc[m][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[s & 1][m], fx[s & 1][j], acc[m][j], 0, 0, 0);
        }
      // the order of issue: LDS reads spread over the products, then the copies
      constexpr int kReads = MT + NT, kMul = MT * NT, kCopies = 2 * kReads;
      static_assert(kReads <= kMul, "a read goes with a product");
#pragma unroll
      for (int k = 0; k < kReads; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(8, 1, 0);
      }
      if (more && s == 3) {
#pragma unroll
        for (int k = 0; k < kMul - kReads; ++k) {
          __builtin_amdgcn_sched_group_barrier(0x20, kCopies / (kMul - kReads), 0);
          __builtin_amdgcn_sched_group_barrier(8, 1, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int i = 0;
  for (; i < n - 2; ++i) stage(i, std::true_type{}, std::false_type{});
  for (; i < n - 1; ++i) stage(i, std::false_type{}, std::false_type{});
  stage(i, std::false_type{}, std::true_type{});

  // Results through LDS, so that a token's channels leave in whole lines.  Each
  // wave has its own place there, which it writes and reads in order: no
  // barrier after the first, and stores stay in flight.
  stage_barrier();
  int8_t *mine = lds + wave * NT * 32 * S::kOutPitch;
  constexpr int kVec = 16 / int(sizeof(E)), kPer = S::kOutRow / 16;  // 16-byte vectors of a token's row
  const bool whole = a.y_vec && n_o == S::kO && n_t == S::kT;
  float sx[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) sx[j] = s_t[wn * NT * 32 + j * 32 + lane % 32];
#pragma unroll
  for (int m0 = 0; m0 < MT; m0 += S::kOutM) {
    float4 sw[S::kOutM * 4], b[S::kOutM * 4];
#pragma unroll
    for (int k = 0; k < S::kOutM * 4; ++k) {
      const int o = wm * MT * 32 + m0 * 32 + k * 8 + lane / 32 * 4;
      sw[k] = *reinterpret_cast<const float4 *>(s_o + o);
      b[k] = *reinterpret_cast<const float4 *>(b_o + o);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < S::kOutM * 4; ++k) {
        const i32x16 &c = acc[m0 + k / 4][j];
        const int g = k % 4 * 4;
        const float v0 = float(c[g]) * sx[j] * sw[k].x + b[k].x, v1 = float(c[g + 1]) * sx[j] * sw[k].y + b[k].y;
        const float v2 = float(c[g + 2]) * sx[j] * sw[k].z + b[k].z, v3 = float(c[g + 3]) * sx[j] * sw[k].w + b[k].w;
        int8_t *p = mine + (j * 32 + lane % 32) * S::kOutPitch + (k * 8 + lane / 32 * 4) * int(sizeof(E));
        if constexpr (sizeof(E) == 2)
          *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf2(v0, v1), pack_bf2(v2, v3));
        else
          *reinterpret_cast<float4 *>(p) = make_float4(v0, v1, v2, v3);
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    const int tt = wn * NT * 32, oo = wm * MT * 32 + m0 * 32;
    E *y = static_cast<E *>(a.y) + (t0 + tt) * a.ldy + o0 + oo;
    if (whole) {
      constexpr int kBatch = 8;
      static_assert(NT * 32 * kPer % (64 * kBatch) == 0, "");
#pragma unroll 1
      for (int v = lane; v < NT * 32 * kPer; v += 64 * kBatch) {
        uint4 r[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
          r[k] = *reinterpret_cast<const uint4 *>(mine + (v + k * 64) / kPer * S::kOutPitch + (v + k * 64) % kPer * 16);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) gstore(y + (v + k * 64) / kPer * a.ldy + (v + k * 64) % kPer * kVec, r[k]);
      }
    } else {
      for (int v = lane; v < NT * 32 * kPer; v += 64) {
        const int r = v / kPer, c = v % kPer * kVec;
        if (tt + r >= n_t || oo + c >= n_o) continue;
        const int8_t *p = mine + r * S::kOutPitch + c * int(sizeof(E));
        if (oo + c + kVec <= n_o && a.y_vec) {
          gstore(y + r * a.ldy + c, *reinterpret_cast<const uint4 *>(p));
        } else {
          for (int e = 0; e < kVec; ++e)
            if (oo + c + e < n_o) gstore(y + r * a.ldy + c + e, reinterpret_cast<const E *>(p)[e]);
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <typename E, int MT, int NT>
hipError_t launch_tiles(const ProductArgs &a, hipStream_t stream) {
  typedef TileShape<E, MT, NT> S;
  static const bool ready = raise_lds_limit(reinterpret_cast<const void *>(product_tile_kernel<E, MT, NT>), S::kLds);
  (void)ready;
  const int tiles_o = (a.d_out + S::kO - 1) / S::kO;
  const int64_t tiles = int64_t(tiles_o) * ((a.T + S::kT - 1) / S::kT);
  product_tile_kernel<E, MT, NT><<<dim3(uint32_t(tiles)), 256, S::kLds, stream>>>(a, tiles_o);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_typed(const ProductArgs &args, hipStream_t stream) {
  ProductArgs a = args;
  a.y_vec = aligned16(a.y) && a.ldy * int64_t(sizeof(E)) % 16 == 0;
  const bool lines = aligned16(a.q) && aligned16(a.W) && a.ldq % 16 == 0 && a.ldw % 16 == 0 && a.d_in % 16 == 0 &&
                     a.ldq <= (1 << 22) && a.ldw <= (1 << 22);
  if (lines && a.T > 128) return launch_tiles<E, 4, 4>(a, stream);
  const dim3 grid((a.d_out + kAnyTile - 1) / kAnyTile, (a.T + kAnyTile - 1) / kAnyTile);
  product_any_kernel<E><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_product(const ProductArgs &a, int dtype, hipStream_t stream) {
  return dtype == LORA_BF16 ? launch_typed<uint16_t>(a, stream) : launch_typed<float>(a, stream);
}

}  // namespace lora
