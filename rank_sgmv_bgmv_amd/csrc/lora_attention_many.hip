// Attention of many bf16 rows over the 8-bit cache, heads of up to 128 (prompts,
// long drafts); the joining of cut units, for every kernel.
//
// A workgroup takes 32 rows a wave of a sequence's (query, query head) pairs for
// one cache head, and goes over their key tiles of 64.  A tile is widened to
// float16 once for all waves and laid in LDS, K as it is and V transposed: while
// one is used the next is converted and the one after it is on its way from
// memory.  Eight waves have four tiles in LDS and meet at a barrier every second
// tile (a prompt of 16384: 2.5% less than with two tiles and a barrier each), four
// waves two tiles, so that two workgroups find room in a CU.
//
//     S^T = K Q^T      32 x 32 x 16 products of float16: keys are rows, queries columns
//     O^T += V^T P^T   the same; P^T comes out of S^T in the lanes that need it
//
// V^T's keys stand in LDS in the order in which a lane holds its weights, so
// that an operand is 16 bytes in a row; pieces of 16 bytes are exchanged within
// rows so that neighbouring lanes meet different banks.
//
// The scales go into the float16 values, over a power of two common to a tile
// (eK, eV): one rounding of at most 2^-11 a value, as the weights have, and
// nothing is left to do per score but exp2.  With t = scale k.q log2 e + eV the
// weights are w = 2^(t - M), rounded to float16, and l = sum w 2^-eV takes them
// rounded, so that weights and sum err alike; where a tile's eV is so far below
// an earlier one's that they would lose more than that, l = sum 2^(t - M - eV)
// in float32.  M follows the running maximum only when that has risen by
// 2^kSlack.  In a tile whose scales lie far apart (kSpreadK, kSpreadV), the keys
// have eK and eV of their own, which meet the scores.
//
// A step computes the scores of the next tile between the weights of this one,
// and widens the tiles after them between the products with V, a piece after
// each pair of products.  A prompt of 16384, window 4096, 32 heads of 128 takes
// 1240 to 1360 us on one card or another, 9.6e11 operations at 0.74 POP/s where a
// large library product of float16 reaches 1.39.  Matrix units are busy 33% of
// the clocks, vector units 50%: the two waves of a SIMD run into the same kind of
// work and wait for each other.  What it spends, taken apart at 1400 us: without
// the products QK 236 us less, PV 226, exponentials 136, widening and loads 364.
// 32 drafts of 24 tokens after up to 16384 keys take 306 us, 0.42 POP/s: a
// quarter of their units' rows are empty, and 47 MB of pieces are written and
// joined.

#include "lora_attention.hpp"

namespace lora {
namespace {

// LDS by 32-bit addresses: generic pointers cost two registers and an addition an operand.
#define LORA_LDS __attribute__((address_space(3)))
template <typename T>
__device__ __forceinline__ T lds_get(int at) {
  typedef typename Raw<sizeof(T)>::type R;
  return __builtin_bit_cast(T, *(const LORA_LDS R *)uintptr_t(uint32_t(at)));
}
template <typename T>
__device__ __forceinline__ void lds_put(int at, const T &v) {
  typedef typename Raw<sizeof(T)>::type R;
  *(LORA_LDS R *)uintptr_t(uint32_t(at)) = __builtin_bit_cast(R, v);
}

// Holds the computation of x to this place: products and exponentials have no order of their own for the compiler, which
// would gather them.
template <typename T>
__device__ __forceinline__ void pin(T &x) {
  asm volatile("" : "+v"(x));
}

// NW waves; DP: the head padded.
template <int DP, int NW>
__global__ __launch_bounds__(64 * NW, 2) void attention_many_kernel(AttnArgs a) {
  typedef uint16_t E;
  constexpr int kThreads = 64 * NW, kSteps = DP / 16, kBlocks = DP / 32;
  constexpr int kChunks = DP / 8;               // 16-byte pieces of a K row
  constexpr int kMask = kChunks < 16 ? kChunks - 1 : 15;
  constexpr int kKUnits = 64 * DP / 16, kKPer = (kKUnits + kThreads - 1) / kThreads;
  constexpr int kVUnits = 16 * DP / 4, kVPer = (kVUnits + kThreads - 1) / kThreads;
  constexpr int kPages = 1024;                  // key blocks whose pages are looked up at once
  static_assert(kPages / 2 % kThreads == 0, "looked up by all threads, half of them at a time");
  // Tiles of V that are widened ahead of the one at work (of K one more), steps from one barrier to the next.
  constexpr int kLead = NW == 8 ? 2 : 1, kBufs = 2 * kLead;
  // LDS: K [kBufs][64][kChunks] and V^T [kBufs][DP][8] in pieces of 16 bytes; of 2 NW tiles the scales of K and V, [2 NW][64]
  // each, what else is known of them and (where they differ much) the keys' exponents; the pages of key blocks
  extern __shared__ __align__(1024) char lds[];
  // (addresses as whole numbers: an exclusive or of them is an address, with no base to be added behind it)
  const int base = int(uintptr_t((LORA_LDS char *)lds));
  constexpr int kRing = 2 * NW;
  constexpr int kV = kBufs * 64 * DP * 2, kKS = 2 * kV, kVS = kKS + kRing * 256, kMeta = kVS + kRing * 256, kExps = kMeta + kRing * 16, kList = kExps + kRing * 256;
  int *lds_pages = reinterpret_cast<int *>(lds + kList);
  const uint4 *exps = reinterpret_cast<const uint4 *>(lds + kExps) + threadIdx.x % 64 / 32;  // of a lane's keys

  if (!plan_matches(a)) {
    if (!a.s.few_blocks && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicAdd(a.plan + H_ERR, 1);  // (else counted there)
    return;
  }
  const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64), col = lane % 32, half = lane / 32;
  const int kv = a.s.kv_heads;
  const int n_items = uniform(gload<int>(a.plan + A_ITEMS + ATTN_MANY));

  for (int item = blockIdx.y; item < n_items; item += gridDim.y) {
    const int head = opaque(blockIdx.x), D = opaque(a.s.head_dim);
    const int2 im = load_item(a, ATTN_MANY, item);
    const AttnUnit u = load_unit(a, ATTN_MANY, uniform(im.x));
    int v0, v1;
    piece_tiles(u, uniform(im.y), v0, v1);

    // queries: lane (col, half) holds values 16 s + 8 half .. of row col of its wave
    const int row_first = u.row0 + wave * 32, row = row_first + col, row_end = u.row0 + u.rows;
    const bool idle = row_first >= row_end;
    f16x8 q[kSteps];
    RowSight sight;
    sight.set(a, u, row);
    float shift;
    {
      float f[kSteps][8];
      float top = 0.f;
      const bool live = row < row_end;
      const E *safe = row_at<const E>(a, a.q, u, head, u.row0), *p = row_at<const E>(a, a.q, u, head, live ? row : u.row0);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        load_query<E, 8>(p, safe, live, 16 * s + 8 * half, D, f[s]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = fabsf(f[s][i]);
          top = fmaxf(top, v < __uint_as_float(0x7f800000u) ? v : 0.f);
        }
      }
      top = half_max(top);  // (a power of two for each row: a large query takes no bits from others)
      const int x = top > 0.f ? min(15 - __builtin_amdgcn_frexp_expf(top), 100) : 0;
      shift = ldexpf(1.f, -x);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack_f16(ldexpf(f[s][2 * i], x), ldexpf(f[s][2 * i + 1], x));
        q[s] = frag(w[0], w[1], w[2], w[3]);
      }
    }
    const float score = a.scale * shift;
    UnitKeys keys;
    keys.set(a, u, u.row0 / a.s.group, (row_end - 1) / a.s.group);
    // positions of the wave's rows
    const int context = u.len - u.n;
    const int p_lo = a.tree ? context : context + row_first / a.s.group;
    const int p_hi = a.tree ? u.len - 1 : context + (min(row_first + 32, row_end) - 1) / a.s.group;

    f32x16 o[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[b][i] = 0.f;
    float M = kNoScore, l = 0.f;
    int e_most = -128;  // the largest eV of the piece's tiles so far
    bool far = false;   // scores are beyond kFarScore

    const int in_page = (1 << a.page_bits) - 1;
    auto fetch_pages = [&](int v, int n) {  // of tiles v .. v + n - 1, as far as there are, to their places in the list
      // (as many for every thread: no lane branch)
      for (int t = v; t < min(v + n, v1); t += kThreads / 4)
        lds_pages[((t - v0) * 4 + tid) % kPages] = block_page(a, u, keys, tile_key(u, t + tid / 4) + (tid % 4) * 16, t + tid / 4 < v1);
    };

    // The scales of a tile, a key a lane, are one wave's work: over a power of two that leaves them below 1 (fp32: those
    // of V), to LDS.  All waves do a tile each at once, NW tiles ahead, so that none waits for another.
    uint32_t sk = 0, sv = 0;
    auto load_scales = [&](int v) {
      const int page = max(lds_pages[((v - v0) * 4 + lane / 16) % kPages], 0);
      const int64_t slot = (int64_t(head) << a.page_bits) + ((tile_key(u, v) + lane) & in_page);
      if (v < v1) {
        sk = gload<uint32_t>(a.c.k_scale + page * a.c.k_scale_page + slot);
        sv = gload<uint32_t>(a.c.v_scale + page * a.c.v_scale_page + slot);
      }
    };
    auto put_scales = [&](int v) {
      const int at = (v - v0) % kRing;
      const bool paged = lds_pages[((v - v0) * 4 + lane / 16) % kPages] >= 0, there = paged & keys.seen(a, tile_key(u, v) + lane);
      sk = there ? sk : 0u, sv = there ? sv : 0u;
      const uint64_t seen = __ballot(paged), nan = __ballot(sv >= kNoScale);
      const uint32_t v_fine = sv >= kNoScale ? 0u : sv, k_fine = sk >= kNoScale ? 0u : sk;
      const int e_k = tile_exponent(__uint_as_float(wave_max_bits(k_fine))), e_v = tile_exponent(__uint_as_float(wave_max_bits(v_fine)));
      // (scales of V that are none become zeros: the rows that see the key get their NaN from its score)
      const float ks = sk >= kNoScale ? __builtin_nanf("") : __uint_as_float(sk);
      int x_k = e_k, x_v = e_v;
      const int own_k = tile_exponent(__uint_as_float(k_fine)), own_v = tile_exponent(__uint_as_float(v_fine));
      const bool apart = __any((k_fine && own_k < e_k - kSpreadK) || (there && own_v < e_v - kSpreadV<false>));
      if (apart) {
        x_k = own_k, x_v = own_v;
        reinterpret_cast<uint32_t *>(lds + kExps)[at * 64 + lane] = pack_exponents(x_k - e_k, x_v - e_v);
      }
      reinterpret_cast<float *>(lds + kKS)[at * 64 + lane] = ks * ldexpf(1.f, -x_k);
      reinterpret_cast<float *>(lds + kVS)[at * 64 + lane] = __uint_as_float(v_fine) * ldexpf(1.f, -x_v);
      const int hidden = (seen & 1 ? 0 : 1) | (seen >> 16 & 1 ? 0 : 2) | (seen >> 32 & 1 ? 0 : 4) | (seen >> 48 & 1 ? 0 : 8);
      // (all lanes the same)
      reinterpret_cast<int4 *>(lds + kMeta)[at] = make_int4((e_k + 128) | (e_v + 128) << 8 | hidden << 16 | int(apart) << 20, 0, int(nan), int(nan >> 32));
    };

    // Raw values of a tile of K and one of V on their way.  A wave's rows lie in one block of 16 keys.  What is past a
    // row's end, or in no page, is read from elsewhere in the cache: it meets zeros of the queries, or is not seen.
    uint4 k_raw[kKPer];
    uint32_t v_raw[kVPer][4];
    // A thread's units lie kThreads apart, whole blocks of 16 keys: what it reads and where it goes is the first unit's
    // but for a constant.
    constexpr int kKRows = kThreads / (DP / 16), kVQuads = kThreads / (DP / 4);
    static_assert((kKPer == 1 || kKRows % 16 == 0) && (kVPer == 1 || kVQuads % 4 == 0), "units of a thread whole blocks apart");
    const int k_row = tid / (DP / 16), k_byte = tid % (DP / 16) * 16, v_quad = tid / (DP / 4), v_byte = tid % (DP / 4) * 4;
    const uint32_t k_off = uint32_t(k_row % 16 * a.pitch + (k_byte < a.pitch ? k_byte : 0));
    const uint32_t v_off = uint32_t(v_quad % 4 * 4 * a.pitch + (v_byte < a.pitch ? v_byte : 0));
    const int k_to = base + (k_row * kChunks + (k_byte / 8 ^ (k_row & kMask))) * 16;
    // keys 4 quad .. of a 16-key block are places 8 (quad & 1) + 4 (quad >> 1) .. of its 16
    const int v_to = base + kV + v_byte * 128 + ((v_quad / 4 * 2 + (v_quad & 1)) ^ (v_byte & 4) ^ (v_byte / 4 & 7)) * 16 + (v_quad >> 1 & 1) * 8;
    auto block_at = [&](int v, int block, int page, const int8_t *values, int64_t page_bytes) {
      const int64_t slot = (int64_t(head) << a.page_bits) + ((tile_key(u, v) + block * 16) & in_page);
      return values + max(page, 0) * page_bytes + slot * a.pitch;
    };
    auto load_k = [&](int v, const int (&pages)[kKPer]) {
#pragma unroll
      for (int i = 0; i < kKPer; ++i) {
        const int first = i * kThreads + wave * 64;
        if (kKUnits % kThreads && first >= kKUnits) continue;
        k_raw[i] = gload_at<uint4>(block_at(v, first / (DP / 16) / 16, pages[i], a.c.k, a.c.k_page), k_off);
      }
    };
    auto load_v = [&](int v, const int (&pages)[kVPer]) {
#pragma unroll
      for (int i = 0; i < kVPer; ++i) {
        const int first = i * kThreads + wave * 64;
        if (kVUnits % kThreads && first >= kVUnits) continue;
        const int8_t *base = block_at(v, first / (DP / 4) / 4, pages[i], a.c.v, a.c.v_page);
#pragma unroll
        for (int j = 0; j < 4; ++j) v_raw[i][j] = gload_at<uint32_t>(base + j * a.pitch, v_off);
      }
    };
    // .. and widened into their buffers
    auto put_k = [&](int v) {
      int to = k_to + ((v - v0) & (kBufs - 1)) * (64 * DP * 2), from = base + kKS + ((v - v0) % kRing * 64 + k_row) * 4;
      pin(to);
      pin(from);
#pragma unroll
      for (int i = 0; i < kKPer; ++i) {
        if (kKUnits % kThreads && i * kThreads + wave * 64 >= kKUnits) continue;
        pin(k_raw[i].x), pin(k_raw[i].y), pin(k_raw[i].z), pin(k_raw[i].w);  // (else widened, and waited for, as soon as loaded)
        const uint32_t w[4] = {k_raw[i].x, k_raw[i].y, k_raw[i].z, k_raw[i].w};
        uint32_t h[8];
        const float f = lds_get<float>(from + i * kKRows * 4);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          h[j] = pack_f16(float(int8_t(w[j / 2] >> (j % 2 * 16))) * f, float(int8_t(w[j / 2] >> (j % 2 * 16 + 8))) * f);
        lds_put(to + i * kKRows * DP * 2, make_uint4(h[0], h[1], h[2], h[3]));
        lds_put((to ^ 16) + i * kKRows * DP * 2, make_uint4(h[4], h[5], h[6], h[7]));
      }
    };
    auto put_v = [&](int v, int j0, int j1) {  // columns j0 .. j1 - 1 of a lane's four
      int to = v_to + ((v - v0) & (kBufs - 1)) * (64 * DP * 2), from = base + kVS + ((v - v0) % kRing * 16 + v_quad) * 16;
      pin(to);
      pin(from);
#pragma unroll
      for (int i = 0; i < kVPer; ++i) {
        if (kVUnits % kThreads && i * kThreads + wave * 64 >= kVUnits) continue;
        const float4 f = lds_get<float4>(from + i * kVQuads * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) pin(v_raw[i][j]);
#pragma unroll
        for (int j = j0; j < j1; ++j) {
          const uint32_t lo = pack_f16(float(int8_t(v_raw[i][0] >> (8 * j))) * f.x, float(int8_t(v_raw[i][1] >> (8 * j))) * f.y);
          const uint32_t hi = pack_f16(float(int8_t(v_raw[i][2] >> (8 * j))) * f.z, float(int8_t(v_raw[i][3] >> (8 * j))) * f.w);
          lds_put((to ^ 16 * (j ^ i * (kVQuads / 2))) + 128 * j, make_uint2(lo, hi));
        }
      }
    };
    // Operands from LDS, kRead at a time, the next ones on their way while these are used.  Their places differ from a
    // lane's first by an exclusive or of a constant.
    constexpr int kRead = 2, kKGroups = 2 * kSteps / kRead, kVGroups = 4 * kBlocks / kRead;
    const int k_first = base + (col * kChunks + (half ^ (col & kMask))) * 16;
    const int v_first = base + kV + (col * 8 + (half ^ ((col ^ col >> 2) & 7))) * 16;
    auto read_k = [&](int at, int g, f16x8 (&f)[kRead]) {
#pragma unroll
      for (int j = 0; j < kRead; ++j) {
        const int kb = (kRead * g + j) / kSteps, st = (kRead * g + j) % kSteps;
        f[j] = lds_get<f16x8>((at ^ 32 * st) + kb * 32 * DP * 2);
      }
    };
    auto read_v = [&](int at, int g, f16x8 (&f)[kRead]) {
#pragma unroll
      for (int j = 0; j < kRead; ++j) {
        const int st = (kRead * g + j) / kBlocks, b = (kRead * g + j) % kBlocks;
        f[j] = lds_get<f16x8>((at ^ 32 * st) + b * 32 * 128);
      }
    };
    // The scores of K tile v, and between the groups of products what `between` does.  f: the first operands.
    auto first_k = [&](int v) {
      int at = k_first + ((v - v0) & (kBufs - 1)) * (64 * DP * 2);
      pin(at);  // (else the places of all operands are kept in registers)
      return at;
    };
    auto scores = [&](int at, f16x8 (&f)[2][kRead], f32x16 (&s)[2], auto between) {
#pragma unroll
      for (int g = 0; g < kKGroups; ++g) {
        if (g + 1 < kKGroups) read_k(at, g + 1, f[(g + 1) % 2]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < kRead; ++j) {
          const int kb = (kRead * g + j) / kSteps, st = (kRead * g + j) % kSteps;
          if (st == 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s[kb][i] = 0.f;
          }
          s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[g % 2][j], q[st], s[kb], 0, 0, 0);
        }
        pin(s[kRead * g / kSteps]);
        between(g);
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    // Tile v: its scores s become weights and outputs, those of v + 1 are computed, V of v + kLead and K of the one after are widened.
    // (In the last tiles what is read and put for the next ones is of no use, and does no harm.)  What a step begins with
    // is read from LDS before the barrier in front of it: what is known of its tile, and the pages of its loads.
    int4 meta;
    int page_k[kKPer], page_v[kVPer];
    auto look_ahead = [&](int v) {
      meta = reinterpret_cast<const int4 *>(lds + kMeta)[(v - v0) % kRing];
#pragma unroll
      for (int i = 0; i < kKPer; ++i) page_k[i] = lds_pages[((v + kLead + 2 - v0) * 4 + (i * kThreads + wave * 64) / (DP / 16) / 16) % kPages];
#pragma unroll
      for (int i = 0; i < kVPer; ++i) page_v[i] = lds_pages[((v + kLead + 1 - v0) * 4 + (i * kThreads + wave * 64) / (DP / 4) * 4 / 16) % kPages];
    };
    auto step = [&](int v, f32x16 (&s)[2], f32x16 (&s_next)[2]) {
      const int word = uniform(meta.x), e_k = (word & 255) - 128, e_v = (word >> 8 & 255) - 128, bad = word >> 16 & 15;
      const bool apart = word >> 20;
      const uint64_t nan = uint32_t(uniform(meta.z)) | uint64_t(uint32_t(uniform(meta.w))) << 32;
      const int key = tile_key(u, v);
      int pk[kKPer], pv[kVPer];
#pragma unroll
      for (int i = 0; i < kKPer; ++i) pk[i] = uniform(page_k[i]);
#pragma unroll
      for (int i = 0; i < kVPer; ++i) pv[i] = uniform(page_v[i]);
      if (!idle) {
        const int at_k = first_k(v + 1);
        f16x8 fk[2][kRead];
        read_k(at_k, 0, fk[0]);
        // (held away from zero, where a hidden key's score would be NaN; it is what scores near zero are multiplied with)
        float factor = fminf(fmaxf(ldexpf(score, e_k), 1e-37f), 1e37f);
        const bool whole = bad == 0 && !apart && nan == 0 && all_seen(a, u, key, p_lo, p_hi);
        if (!whole) {
          if (apart) {
            scale_apart(s, factor, exps + (v - v0) % kRing * 16);
            factor = 1.f;
          }
          // (a lane's keys are four of each eight)
          const uint64_t seen = sight.seen(a, u, key, bad) >> 4 * half, hit = nan >> 4 * half;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int at = i / 4 * 8 + i % 4;
            const float x = hit >> at & 1 ? __builtin_nanf("") : s[i / 16][i % 16];
            s[i / 16][i % 16] = seen >> at & 1 ? x : -__builtin_inff();
          }
        }
        float top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < 32; ++i) top = fmaxf(top, s[i / 16][i % 16]);
        const float most = half_max(top);
        top = most * factor + (float(e_v) - kHeadroom<false>);
        if (__any(top > M + kSlack<false>)) {
          if (fabsf(top) > kFarScore) top = product(most, factor) + (float(e_v) - kHeadroom<false>);
          const float m = fmaxf(M, top), fade = __builtin_amdgcn_exp2f(M - m);
          M = m;
          far = __any(fabsf(M) > kFarScore && M != kNoScore);
          l *= fade;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) o[b] *= fade;
        }
        float less = M - float(e_v);
        e_most = max(e_most, e_v);
        const bool low = apart || e_v < e_most - kLowTile;
        if (low || far) {
          if (far) {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i / 16][i % 16] = far_score(product(s[i / 16][i % 16], factor), less, kMostWeight);
            factor = 1.f, less = 0.f;
          }
          if (low) l += sum_exact(s, factor, less, e_v, apart, exps + (v - v0) % kRing * 16);
        }
        float sum = 0.f;
        uint32_t r[16];
        int at_v = v_first + ((v - v0) & (kBufs - 1)) * (64 * DP * 2);
        pin(at_v);
        f16x8 fv[2][kRead];
        scores(at_k, fk, s_next, [&](int g) {
          // weights of 8 / kKGroups groups of four keys; the sum takes them as the outputs do, rounded
#pragma unroll
          for (int n = g * 8 / kKGroups; n < (g + 1) * 8 / kKGroups; ++n) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_exp2f(fmaf(s[n / 4][n % 4 * 4 + i], factor, -less));
            r[2 * n] = pack_f16(p[0], p[1]), r[2 * n + 1] = pack_f16(p[2], p[3]);
            sum = sum_f16(r[2 * n + 1], sum_f16(r[2 * n], sum));
            pin(r[2 * n]), pin(r[2 * n + 1]);
          }
          if (g == kKGroups - 1) read_v(at_v, 0, fv[0]);
        });
        l = fmaf(sum, low ? 0.f : ldexpf(1.f, -e_v), l);
#pragma unroll
        for (int g = 0; g < kVGroups; ++g) {
          if (g + 1 < kVGroups) read_v(at_v, g + 1, fv[(g + 1) % 2]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < kRead; ++j) {
            const int st = (kRead * g + j) / kBlocks, b = (kRead * g + j) % kBlocks;
            o[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fv[g % 2][j], frag(r[4 * st], r[4 * st + 1], r[4 * st + 2], r[4 * st + 3]),
                                                          o[b], 0, 0, 0);
          }
#pragma unroll
          for (int j = 0; j < kRead; ++j) pin(o[(kRead * g + j) % kBlocks]);
          // the next tiles, in pieces between the products
          if (g == kVGroups / 8) put_v(v + kLead, 0, 2);
          if (g == kVGroups * 3 / 8) put_v(v + kLead, 2, 4);
          if (g == kVGroups * 5 / 8) put_k(v + kLead + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        put_v(v + kLead, 0, 4);
        put_k(v + kLead + 1);
      }
      if (v + kLead + 1 < v1) load_v(v + kLead + 1, pv);
      if (v + kLead + 2 < v1) load_k(v + kLead + 2, pk);
      if ((v - v0) % NW == 0) {
        put_scales(v + NW + wave);
        load_scales(v + 2 * NW + wave);
      }
      // half the list of pages anew, well before it is needed
      constexpr int kHalf = kPages / 8;
      const int next_half = (v - v0) / kHalf * kHalf + kHalf;
      if ((v - v0) % kHalf == kHalf / 2 && next_half >= 2 * kHalf && v0 + next_half < v1) fetch_pages(v0 + next_half, kHalf);
      look_ahead(v + 1);
      if (kLead == 1 || (v - v0) & 1) lds_barrier();
    };

    if (v0 < v1) {
      fetch_pages(v0, kPages / 4);
      lds_barrier();
      auto pages_of = [&](int v, int (&pk)[kKPer], int (&pv)[kVPer]) {
#pragma unroll
        for (int i = 0; i < kKPer; ++i) pk[i] = uniform(lds_pages[((v - v0) * 4 + (i * kThreads + wave * 64) / (DP / 16) / 16) % kPages]);
#pragma unroll
        for (int i = 0; i < kVPer; ++i) pv[i] = uniform(lds_pages[((v - v0) * 4 + (i * kThreads + wave * 64) / (DP / 4) * 4 / 16) % kPages]);
      };
      int pk[kKPer], pv[kVPer];
      pages_of(v0, pk, pv);
      load_k(v0, pk);
      load_v(v0, pv);
      load_scales(v0 + wave);
      put_scales(v0 + wave);
      load_scales(v0 + NW + wave);
      lds_barrier();
      put_k(v0);
      put_v(v0, 0, 4);
#pragma unroll
      for (int t = 1; t <= kLead; ++t)
        if (v0 + t < v1) {
          pages_of(v0 + t, pk, pv);
          load_k(v0 + t, pk);
          load_v(v0 + t, pv);
          put_k(v0 + t);
          if (t < kLead) put_v(v0 + t, 0, 4);
        }
      if (v0 + kLead + 1 < v1) {
        pages_of(v0 + kLead + 1, pk, pv);
        load_k(v0 + kLead + 1, pk);
      }
      lds_barrier();
      f32x16 s[2][2];
      look_ahead(v0);
      if (!idle) {
        f16x8 f[2][kRead];
        const int at = first_k(v0);
        read_k(at, 0, f[0]);
        scores(at, f, s[0], [](int) {});
      }
      lds_barrier();  // the first buffer's next tile comes within the loop
      for (int v = v0; v < v1; ++v) {
        step(v, s[0], s[1]);
        s[0][0] = s[1][0], s[0][1] = s[1][1];
      }
      if (kLead == 2 && (v1 - v0) & 1) lds_barrier();  // the next item writes what the last step read
    }

    // (V in float16 is value * scale / 2^eV)
    l = half_sum(l);
    if (row < row_end) {
      if (u.nsplit == 1) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        E *to = row_at<E>(a, a.out, u, head, row);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int d = b * 32 + g * 8 + half * 4;
            const float f[4] = {o[b][4 * g] * inv, o[b][4 * g + 1] * inv, o[b][4 * g + 2] * inv, o[b][4 * g + 3] * inv};
            store_four(to + d, f, D - d);
          }
      } else {
        const int64_t at = (int64_t(u.slot + uniform(im.y)) * kv + head) * a.s.many_rows + (row - u.row0);
        float *part = reinterpret_cast<float *>(a.ws + a.s.part[ATTN_MANY]) + at * DP;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            gstore(part + b * 32 + g * 8 + half * 4,
                   make_float4(o[b][4 * g], o[b][4 * g + 1], o[b][4 * g + 2], o[b][4 * g + 3]));
        if (half == 0) gstore(reinterpret_cast<float *>(a.ws + a.s.stat[ATTN_MANY]) + at * 2, make_float2(M, l));
      }
    }
  }
}

template <int DP, int NW>
hipError_t launch_many(const AttnArgs &a, hipStream_t stream) {
  const auto kernel = attention_many_kernel<DP, NW>;
  constexpr size_t smem = size_t(NW == 8 ? 4 : 2) * 64 * DP * 2 * 2 + 2 * NW * (512 + 16 + 256) + 4096;
  static const bool once = raise_lds_limit(reinterpret_cast<const void *>(kernel), smem);
  (void)once;
  kernel<<<item_grid(a, ATTN_MANY), 64 * NW, smem, stream>>>(a);
  return hipGetLastError();
}

constexpr int kJoinThreads = 256, kJoinRows = 16;

// out = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) l_i over the pieces of a cut unit, in their order; 16 rows of a cache
// head a workgroup, the cut units of few rows (`few` workgroups a head) and those of many in one launch.  Four pieces are
// on their way at once.
template <int DP, typename E>
__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(AttnArgs a, int few) {
  constexpr int kCols = DP / 16, kAtOnce = 4;
  const int head = blockIdx.x % a.s.kv_heads, at_x = blockIdx.x / a.s.kv_heads;
  const int kind = at_x < few ? ATTN_FEW : ATTN_MANY, x = at_x < few ? at_x : at_x - few;
  const int most_rows = kind == ATTN_FEW ? a.s.few_rows : a.s.many_rows, tiles = (most_rows + kJoinRows - 1) / kJoinRows;
  const int cut = x / tiles;
  int n = gload<int>(a.plan + A_CUT + kind);
  if (!plan_matches(a)) return;
  n = uniform(n);
  const int kv = a.s.kv_heads, D = a.s.head_dim;
  const int r = x % tiles * kJoinRows + threadIdx.x / 16, d0 = threadIdx.x % 16 * kCols;
  if (cut < n) {
    const int m = uniform(gload<int>(reinterpret_cast<const char *>(a.plan) + a.s.cutlist[kind] + size_t(cut) * 4));
    const AttnUnit u = load_unit(a, kind, m);
    if (r >= u.rows) return;
    const float *part = reinterpret_cast<const float *>(a.ws + a.s.part[kind]);
    const float *stat = reinterpret_cast<const float *>(a.ws + a.s.stat[kind]);
    float M = kNoScore, l = 0.f, y[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) y[c] = 0.f;
    for (int i0 = 0; i0 < u.nsplit; i0 += kAtOnce) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce][kCols / 4];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int64_t at = (int64_t(u.slot + min(i0 + i, u.nsplit - 1)) * kv + head) * most_rows + r;
        ml[i] = gload<float2>(stat + at * 2);
#pragma unroll
        for (int c = 0; c < kCols / 4; ++c) v[i][c] = gload<float4>(part + at * DP + d0 + 4 * c);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (i0 + i >= u.nsplit) break;
        const float top = fmaxf(M, ml[i].x), old = __builtin_amdgcn_exp2f(M - top), now = __builtin_amdgcn_exp2f(ml[i].x - top);
        M = top;
        l = l * old + ml[i].y * now;
#pragma unroll
        for (int c = 0; c < kCols / 4; ++c) {
          y[4 * c] = y[4 * c] * old + v[i][c].x * now, y[4 * c + 1] = y[4 * c + 1] * old + v[i][c].y * now;
          y[4 * c + 2] = y[4 * c + 2] * old + v[i][c].z * now, y[4 * c + 3] = y[4 * c + 3] * old + v[i][c].w * now;
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    E *to = row_at<E>(a, a.out, u, head, u.row0 + r) + d0;
#pragma unroll
    for (int c = 0; c < kCols; c += 4) {
      const float f[4] = {y[c] * inv, y[c + 1] * inv, y[c + 2] * inv, y[c + 3] * inv};
      store_four(to + c, f, D - d0 - c);
    }
  }
}

template <typename E>
hipError_t launch_join(const AttnArgs &a, hipStream_t stream) {
  const auto tiles = [&](int kind, int rows) { return a.s.cut[kind] * ((rows + kJoinRows - 1) / kJoinRows); };
  const int few = tiles(ATTN_FEW, a.s.few_rows), many = tiles(ATTN_MANY, a.s.many_rows);
  if (!few && !many) return hipSuccess;
  const dim3 grid((few + many) * a.s.kv_heads);  // no more than 16 times the target of pieces
  if (a.s.dp == 64) attention_join_kernel<64, E><<<grid, kJoinThreads, 0, stream>>>(a, few);
  else if (a.s.dp == 128) attention_join_kernel<128, E><<<grid, kJoinThreads, 0, stream>>>(a, few);
  else attention_join_kernel<256, E><<<grid, kJoinThreads, 0, stream>>>(a, few);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_many(const AttnArgs &a, int dtype, hipStream_t stream) {
  if (dtype != LORA_BF16 || a.s.dp > 128) return launch_attention_exact(a, dtype, stream);
  const bool wide = a.s.many_rows == 256;
  if (a.s.dp == 64) return wide ? launch_many<64, 8>(a, stream) : launch_many<64, 4>(a, stream);
  return wide ? launch_many<128, 8>(a, stream) : launch_many<128, 4>(a, stream);
}

hipError_t launch_attention(const AttnArgs &a, int dtype, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.s.few_blocks) e = launch_attention_few(a, dtype, stream);
  if (e == hipSuccess && a.s.many_rows) e = launch_attention_many(a, dtype, stream);
  if (e == hipSuccess) e = dtype == LORA_BF16 ? launch_join<uint16_t>(a, stream) : launch_join<float>(a, stream);
  return e;
}

}  // namespace lora
