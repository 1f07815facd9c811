// Device helpers shared by the attention kernels: 8-bit values as float16,
// swaps between the quarters of a wave, the walk over a plan's items, masks.
#pragma once

#include "lora_device.hpp"
#include "lora_layer.hpp"

namespace lora {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr uint32_t kNoScale = 0x7f800000u;  // from these bits on: infinite, NaN or negative

constexpr float kNoScore = -3.0e38f;  // the running maximum before the first key
// The largest weight of a row is 2^kHeadroom when its maximum is taken, and no more than 2^(kHeadroom + kSlack) before
// the maximum is taken anew, so that float16 holds it.  Weights that are 2^-(14 + kHeadroom) of the largest and less are
// held to a fixed 2^-(25 + kHeadroom) of it.  A slack of 7 takes a maximum anew 3 or 4 times a row instead of at every
// new one; float32 calls, whose second float16 number begins 2^-11 lower, have the headroom instead.
// The kernel for few rows follows every new maximum and has the float32 headroom in both types.
template <bool F32> constexpr float kHeadroom = F32 ? 14.f : 8.f;
template <bool F32> constexpr float kSlack = F32 ? 1.f : 7.f;
// Kernels that sum weights after their rounding do so in tiles whose value exponent is no more than this below the largest
// of the tiles before: what a key's weight can lose there is 2^-(25 + kHeadroom - kLowTile) of a row's sum, 2^-29.  (A tile
// of zeros, whose exponent is -60, behind one of ordinary values would lose all of it.)  Where all tiles of a prompt but the
// first take the other way, 16384 tokens take 1600 us for 1240.
constexpr int kLowTile = 4;

// Two bytes of u (8-bit values plus 128, so 0 .. 255) as float16, (u - 128) /
// 512 each.  The bytes are taken as the float16 numbers u * 2^-24 that their
// bits are; one fused multiply-add moves and shifts them, with no rounding.
__device__ __forceinline__ f16x2 bytes_to_f16(uint32_t halves) {
  const f16x2 up = {_Float16(32768.f), _Float16(32768.f)}, off = {_Float16(-0.25f), _Float16(-0.25f)};
  return __builtin_elementwise_fma(__builtin_bit_cast(f16x2, halves), up, off);
}
constexpr uint32_t kByteBias = 0x80808080u;
constexpr float kByteScale = 512.f;

// Two floats as float16, to the nearest.
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const f32x2 f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, f16x2));
}

// acc + a.lo + a.hi
__device__ __forceinline__ float sum_f16(uint32_t a, float acc) {
  const f16x2 ones = {_Float16(1.f), _Float16(1.f)};
  return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), ones, acc, false);
}

__device__ __forceinline__ f16x8 frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint4 u = make_uint4(a, b, c, d);
  return __builtin_bit_cast(f16x8, u);
}

// over the lanes l, l ^ 32 (and the four l ^ 16, l ^ 32, l ^ 48)
__device__ __forceinline__ float half_max(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float half_sum(float v) {
  const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
__device__ __forceinline__ float quarters_max(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return half_max(fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1])));
}
__device__ __forceinline__ float quarters_sum(float v) {
  const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return half_sum(__uint_as_float(s[0]) + __uint_as_float(s[1]));
}

// The largest over the wave, of the bits of floats that are not negative too.
__device__ __forceinline__ uint32_t wave_max_bits(uint32_t v) {
#define LORA_ROR(n) v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x120 + (n), 0xf, 0xf, false)))
  LORA_ROR(1);
  LORA_ROR(2);
  LORA_ROR(4);
  LORA_ROR(8);
#undef LORA_ROR
  const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(uint32_t(s[0]), uint32_t(s[1]));
  const auto t = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(uint32_t(t[0]), uint32_t(t[1]));
}

// An exponent e with |v| in [2^(e-1), 2^e), held to -60 .. 100: what tiles are scaled by on their way to float16.
constexpr int kLeastExponent = -60;
__device__ __forceinline__ int tile_exponent(float v) {
  return v > 0.f ? min(max(__builtin_amdgcn_frexp_expf(v), kLeastExponent), 100) : kLeastExponent;
}

// Scales of a tile that are much less than its largest lose bits to it, which a row may not even see: in such a tile each
// key has an exponent of its own.  Keys lose none down to 2^-kSpreadK (an 8-bit value over 2^13 is a normal float16
// number); of values, what is left of a weight's range is smaller by as much, and one that is zero leaves none where its
// key takes most of the weight.  bfloat16 has less to lose; where every tile is such a one, a prompt of 16384 takes 2070 us
// for 1300, drafts 490 for 319, single tokens what they take else.
constexpr int kSpreadK = 12;
template <bool F32> constexpr int kSpreadV = F32 ? 4 : 8;

// Scores beyond this, where float32 has steps of 1/8 and more: a weight is then 2 to the difference of two rounded numbers,
// which may lie above or below what the headroom is for by some steps.  The product with the scales is rounded before the
// maximum is taken off it, so that the largest score keeps a weight, and weights are held to what float16 holds.
constexpr float kFarScore = 0x1p20f, kMostWeight = 15.f;  // (2^kMostWeight)
// a * b, rounded (not part of a fused multiply-add)
__device__ __forceinline__ float product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}
// s - less, no more than most (NaN stays)
__device__ __forceinline__ float far_score(float s, float less, float most) {
  const float x = s - less;
  return x > most ? most : x;
}

// The plan made for this call.
__device__ __forceinline__ bool plan_matches(const AttnArgs &a) {
  bool ok = true;
#pragma unroll
  for (int i = 0; i < A_KEYS; i += 4) {
    const int4 w = gload<int4>(a.plan + A_KEY + i);
    ok = ok && w.x == a.key[i] && w.y == a.key[i + 1] && w.z == a.key[i + 2] && w.w == a.key[i + 3];
  }
  return uniform(ok);
}

// A uniform value of which the compiler knows nothing: what depends on it is computed where it is used, and not kept in
// registers from before the loop over the items.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+s"(v));
  return v;
}

// Item `item` of a kind: its unit and which piece of it.
__device__ __forceinline__ int2 load_item(const AttnArgs &a, int kind, uint32_t item) {
  return gload<int2>(reinterpret_cast<const char *>(a.plan) + a.s.item[kind] + size_t(item) * 8);
}

__device__ __forceinline__ AttnUnit load_unit(const AttnArgs &a, int kind, int m) {
  const char *at = reinterpret_cast<const char *>(a.plan) + a.s.unit[kind] + size_t(m) * sizeof(AttnUnit);
  const int4 w0 = gload<int4>(at), w1 = gload<int4>(at + 16), w2 = gload<int4>(at + 32);
  AttnUnit u;
  u.q0 = uniform(w0.x), u.n = uniform(w0.y), u.len = uniform(w0.z), u.row0 = uniform(w0.w);
  u.rows = uniform(w1.x), u.seq = uniform(w1.y), u.ntiles = uniform(w1.z), u.sink_tiles = uniform(w1.w);
  u.main = uniform(w2.x), u.nsplit = uniform(w2.y), u.slot = uniform(w2.z);
  return u;
}

// Piece `part` of a unit: its tiles v0 .. v1 - 1.
__device__ __forceinline__ void piece_tiles(const AttnUnit &u, int part, int &v0, int &v1) {
  v0 = int(int64_t(u.ntiles) * part / u.nsplit);
  v1 = int(int64_t(u.ntiles) * (part + 1) / u.nsplit);
}

// The keys that a unit's rows see, one or another of them: lo .. hi - 1, and below hi the first keys of the sequence.
// Scales of others, which a former request may have left or nobody may ever have written, are not used for anything.
struct UnitKeys {
  int lo, hi;
  // (first, last: the first and last query)
  __device__ __forceinline__ void set(const AttnArgs &a, const AttnUnit &u, int first, int last) {
    const int context = u.len - u.n, p = context + (a.tree ? 0 : first);
    lo = p >= a.window ? p - a.window + 1 : 0;
    hi = a.tree ? u.len : min(u.len, context + last + 1);
  }
  // whether one of the keys key .. key + more is seen
  __device__ __forceinline__ bool seen(const AttnArgs &a, int key, int more = 0) const {
    return (key < hi) & ((key + more >= lo) | (key < a.sinks));
  }
};

// Which page a block of 16 keys lies in; -1 where no row sees its keys, or in no page of the cache.  (No lane branches here,
// nor elsewhere while a kernel's operands are in registers: where lanes come back from one, the compiler has put copies of
// registers before the instruction that brings them back, and what the other lanes held was lost.)
__device__ __forceinline__ int block_page(const AttnArgs &a, const AttnUnit &u, const UnitKeys &keys, int key, bool there) {
  there = there & keys.seen(a, key, 15);
  const int p = gload<int>(a.pages + int64_t(u.seq) * a.ld_pages + (there ? key >> a.page_bits : 0));
  return (there & (p >= 0) & (p < a.c.n_pages)) ? p : -1;
}

__device__ __forceinline__ int tile_key(const AttnUnit &u, int v) {
  return (v < u.sink_tiles ? v : u.main + v - u.sink_tiles) * kKeyTile;
}

// The first n bits: none for a negative n, all from 64 on.
__device__ __forceinline__ uint64_t bits_below(int n) {
  const uint64_t some = ~uint64_t(0) >> ((64 - min(max(n, 0), 64)) & 63);
  return n > 0 ? some : 0;
}

// What a row sees: keys up to its position within the window, the first ones, and of a tree's drafted tokens those of its mask.
struct RowSight {
  int pos, first_end;  // position; the end of the first keys that stay visible
  uint64_t mask;       // the drafted tokens of a tree
  // (no lane branches, as for the queries: rows that are not there read the first one's mask)
  __device__ __forceinline__ void set(const AttnArgs &a, const AttnUnit &u, int row) {
    const bool live = row < u.row0 + u.rows;
    const int i = (live ? row : u.row0) / a.s.group, context = u.len - u.n;
    int at = context + i;
    mask = 0;
    if (a.tree) {
      mask = gload<uint64_t>(a.tree + u.q0 + i) & (~uint64_t(0) >> (LORA_MAX_TREE - u.n));
      at = context + __popcll(mask & ((uint64_t(1) << i) - 1));
      mask = live ? mask : 0;
    }
    pos = live ? at : -1;
    first_end = min(a.sinks, pos + 1);
  }
  // The keys of a tile that it sees, a bit each.  hidden: the blocks of 16 that nobody sees.
  __device__ __forceinline__ uint64_t seen(const AttnArgs &a, const AttnUnit &u, int key, uint32_t hidden) const {
    const int lo = pos >= a.window ? pos - a.window + 1 : 0, context = u.len - u.n;
    uint64_t keys = (bits_below(pos + 1 - key) & ~bits_below(lo - key)) | bits_below(first_end - key);
    if (a.tree && key + kKeyTile > context) {
      const int c = context - key;  // less than 64
      const uint64_t drafts = c >= 0 ? mask << (c & 63) : mask >> (-c & 63);
      keys = (keys & bits_below(c)) | ((c > -64 ? drafts : 0) & ~bits_below(c));
    }
#pragma unroll
    for (int b = 0; b < 4; ++b) keys &= hidden >> b & 1 ? ~(uint64_t(0xffff) << 16 * b) : ~uint64_t(0);
    return keys;
  }
};

// Whether every row at positions lo .. hi sees all of a tile.
__device__ __forceinline__ bool all_seen(const AttnArgs &a, const AttnUnit &u, int key, int lo, int hi) {
  const int last = key + kKeyTile - 1;
  return last <= (a.tree ? u.len - u.n - 1 : lo) && (hi - key < a.window || last < a.sinks);
}

template <typename E>
__device__ __forceinline__ float to_float(E v) {
  if constexpr (sizeof(E) == 4) return v;
  else return bf_to_f(v);
}

// What is kept of the keys of a tile that have exponents of their own: those of K and of V, less the tile's.
__device__ __forceinline__ uint32_t pack_exponents(int k, int v) { return uint32_t(k & 0xffff) | uint32_t(v) << 16; }
__device__ __forceinline__ int k_exponent(uint32_t e) { return int(int16_t(e)); }
__device__ __forceinline__ int v_exponent(uint32_t e) { return int(e) >> 16; }

// A lane's products of such a tile become scores plus exponents of V (less the tile's).  e: the tile's, groups of four keys
// a lane, two groups apart.
__device__ __forceinline__ void scale_apart(f32x16 (&s)[2], float factor, const uint4 *e) {
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const uint4 w = e[2 * n];
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s[n / 4][n % 4 * 4 + i] = fmaf(s[n / 4][n % 4 * 4 + i], ldexpf(factor, k_exponent(x[i])), float(v_exponent(x[i])));
  }
}

// A lane's part of a tile's sum of 2^(score - M): its weights 2^(s factor - less), of which the exponents of V are taken off
// again, so that they err as the outputs' do.  apart: s is what scale_apart made of it.
__device__ __forceinline__ float sum_exact(const f32x16 (&s)[2], float factor, float less, int e_v, bool apart, const uint4 *e) {
  float sum = 0.f;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    uint32_t x[4] = {0u, 0u, 0u, 0u};
    if (apart) {
      const uint4 w = e[2 * n];
      x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sum += ldexpf(__builtin_amdgcn_exp2f(fmaf(s[n / 4][n % 4 * 4 + i], factor, -less)), -e_v - v_exponent(x[i]));
  }
  return sum;
}

// Values d0 .. d0 + N - 1 of a query head, of the D that it has (zeros behind them, and in rows that are not `live`).  No
// lane branches: where there is nothing to read, the values at `safe`, a row of D, are read and not used.
template <typename E, int N>
__device__ __forceinline__ void load_query(const E *p, const E *safe, bool live, int d0, int D, float *f) {
  constexpr int kWide = 16 / sizeof(E);
  typedef uint32_t U __attribute__((ext_vector_type(4), aligned(2)));
  const int left = live ? D - d0 : 0;
  p += left > 0 ? d0 : 0;
  if (D % kWide == 0) {
#pragma unroll
    for (int i = 0; i < N; i += kWide) {
      const bool ok = i < left;
      const U u = *(const LORA_GLOBAL U *)(ok ? p + i : safe);
#pragma unroll
      for (int j = 0; j < kWide; ++j) {
        float x;
        if constexpr (sizeof(E) == 4) x = __uint_as_float(u[j]);
        else x = j % 2 ? bf_hi(u[j / 2]) : bf_lo(u[j / 2]);
        f[i + j] = ok ? x : 0.f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool ok = i < left;
      const float x = to_float(gload<E>(ok ? p + i : safe));
      f[i] = ok ? x : 0.f;
    }
  }
}

// Four output values at p, of which n are there.
template <typename E>
__device__ __forceinline__ void store_four(E *p, const float *f, int n) {
  if (n >= 4) {
    if constexpr (sizeof(E) == 2) {
      typedef uint32_t U __attribute__((ext_vector_type(2), aligned(2)));
      const U u = {pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3])};
      *(LORA_GLOBAL U *)p = u;
    } else {
      typedef float U __attribute__((ext_vector_type(4), aligned(4)));
      const U u = {f[0], f[1], f[2], f[3]};
      *(LORA_GLOBAL U *)p = u;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) {
        if constexpr (sizeof(E) == 2) gstore(p + j, f_to_bf(f[j]));
        else gstore(p + j, f[j]);
      }
  }
}

// Row `row` of a sequence in the query or output heads.
template <typename E>
__device__ __forceinline__ E *row_at(const AttnArgs &a, const lora_heads &h, const AttnUnit &u, int kv_head, int row) {
  const int i = row / a.s.group, g = row - i * a.s.group;
  return static_cast<E *>(h.data) + int64_t(u.q0 + i) * h.token + int64_t(kv_head * a.s.group + g) * h.head;
}

// Workgroups of a kind: cache heads x items, heads in turn, so that the units of a sequence that read the same keys come to
// one XCD where there are 8 heads.  No more than 2^20 or so, however many heads and sequences there may be: each takes
// items in turn.
inline dim3 item_grid(const AttnArgs &a, int kind) {
  const int most = (1 << 20) / a.s.kv_heads + 1, cap = most < 65535 ? most : 65535;
  return dim3(uint32_t(a.s.kv_heads), uint32_t(a.s.items[kind] < cap ? a.s.items[kind] : cap));
}

hipError_t launch_attention_few(const AttnArgs &a, int dtype, hipStream_t stream);
hipError_t launch_attention_many(const AttnArgs &a, int dtype, hipStream_t stream);
hipError_t launch_attention_exact(const AttnArgs &a, int dtype, hipStream_t stream);

}  // namespace lora
