// Attention of many rows over the 8-bit cache where the values of K and V stay
// exact (fp32) or a head is longer than 128.
//
// As the kernel for many bf16 rows: 32 rows a wave, four waves, key tiles of 64
// widened to float16 once for all of them and laid in LDS, two in turn.
//
//     S^T = K Q^T      32 x 32 x 16 products of float16: keys are rows, queries columns
//     O^T += V^T P^T   the same; P^T comes out of S^T in the lanes that need it
//
// For fp32 the 8-bit values are widened exactly, the scales meet scores and
// weights in float32, and queries and weights are two float16 numbers each, 22
// bits.  For bf16 the scales go into the float16 values, over a power of two
// common to a tile (eK, eV): one rounding of at most 2^-11 a value, as the weights
// have, and maximum and sum are those of that kernel; fp32 has them as the kernel
// for few rows.
//
// One workgroup a CU, so one wave a SIMD with all 512 registers: the accumulators
// stay in the upper half, where products read and write them (held to the lower
// half by the scheduling that serves the other kernel, 711 of a tile's 1147
// instructions were copies between the halves).  Products and the arithmetic
// between them take turns; nothing of the next tile's runs beside them.  48 rows
// of 32 sequences over 8192 keys each, 8 heads: of 128 in fp32 469 us, of 256 in
// bf16 1066, in fp32 1835 (both of these spill, 288 and 436 bytes a lane).

#include "lora_attention.hpp"

namespace lora {
namespace {

// Holds the computation of x to this place: products and exponentials have no order of their own for the compiler, which
// would gather them.
template <typename T>
__device__ __forceinline__ void pin(T &x) {
  asm volatile("" : "+v"(x));
}

// NW waves; DP: the head padded; F32: queries and outputs in float32.
template <int DP, int NW, bool F32>
__global__ __launch_bounds__(64 * NW, NW / 4) void attention_exact_kernel(AttnArgs a) {
  typedef std::conditional_t<F32, float, uint16_t> E;
  constexpr int kVD = DP == 256 ? 128 : DP;  // columns of V at a time
  constexpr int kThreads = 64 * NW, kSteps = DP / 16, kBlocks = kVD / 32, kTerms = F32 ? 2 : 1;
  constexpr int kChunks = DP / 8;               // 16-byte pieces of a K row
  constexpr int kMask = kChunks < 16 ? kChunks - 1 : 15;
  constexpr int kKUnits = 64 * DP / 16, kKPer = (kKUnits + kThreads - 1) / kThreads;
  constexpr int kVUnits = 16 * kVD / 4, kVPer = (kVUnits + kThreads - 1) / kThreads;
  constexpr int kPages = 1024;                  // key blocks whose pages are looked up at once
  static_assert(kPages / 2 % kThreads == 0, "looked up by all threads, half of them at a time");
  // LDS: K [2][64][kChunks] and V^T [2][kVD][8] in pieces of 16 bytes; of 2 NW tiles the scales of K and V, [2 NW][64]
  // each, what else is known of them and (where they differ much) the keys' exponents; the pages of key blocks
  extern __shared__ __align__(16) char lds[];
  constexpr int kRing = 2 * NW;
  constexpr int kV = 2 * 64 * DP * 2, kKS = kV + 2 * 64 * kVD * 2, kVS = kKS + kRing * 256, kMeta = kVS + kRing * 256, kExps = kMeta + kRing * 16, kList = kExps + kRing * 256;
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
    int d0 = 0;  // the columns of V at work
    const int2 im = load_item(a, ATTN_MANY, item);
    const AttnUnit u = load_unit(a, ATTN_MANY, uniform(im.x));
    int v0, v1;
    piece_tiles(u, uniform(im.y), v0, v1);

    // queries: lane (col, half) holds values 16 s + 8 half .. of row col of its wave
    const int row_first = u.row0 + wave * 32, row = row_first + col, row_end = u.row0 + u.rows;
    const bool idle = row_first >= row_end;
    f16x8 q[kTerms][kSteps];
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
        uint32_t w[kTerms][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y0 = ldexpf(f[s][2 * i], x), y1 = ldexpf(f[s][2 * i + 1], x);
          w[0][i] = pack_f16(y0, y1);
          if constexpr (F32) {
            const f16x2 r = __builtin_bit_cast(f16x2, w[0][i]);
            w[kTerms - 1][i] = pack_f16(y0 - float(r.x), y1 - float(r.y));
          }
        }
#pragma unroll
        for (int t = 0; t < kTerms; ++t) q[t][s] = frag(w[t][0], w[t][1], w[t][2], w[t][3]);
      }
    }
    const float score = a.scale * shift * (F32 ? kByteScale : 1.f);
    UnitKeys keys;
    keys.set(a, u, u.row0 / a.s.group, (row_end - 1) / a.s.group);
    // positions of the wave's rows
    const int context = u.len - u.n;
    const int p_lo = a.tree ? context : context + row_first / a.s.group;
    const int p_hi = a.tree ? u.len - 1 : context + (min(row_first + 32, row_end) - 1) / a.s.group;

    f32x16 o[kBlocks];
    float M, l;
    int e_most;  // the largest eV of the piece's tiles so far
    bool far;    // scores are beyond kFarScore

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
      const bool apart = __any((!F32 && k_fine && own_k < e_k - kSpreadK) || (there && own_v < e_v - kSpreadV<F32>));
      if (apart) {
        x_k = own_k, x_v = own_v;
        reinterpret_cast<uint32_t *>(lds + kExps)[at * 64 + lane] = pack_exponents(F32 ? 0 : x_k - e_k, x_v - e_v);
      }
      reinterpret_cast<float *>(lds + kKS)[at * 64 + lane] = F32 ? ks : ks * ldexpf(1.f, -x_k);
      reinterpret_cast<float *>(lds + kVS)[at * 64 + lane] = __uint_as_float(v_fine) * ldexpf(1.f, -x_v);
      const int hidden = (seen & 1 ? 0 : 1) | (seen >> 16 & 1 ? 0 : 2) | (seen >> 32 & 1 ? 0 : 4) | (seen >> 48 & 1 ? 0 : 8);
      // (all lanes the same)
      reinterpret_cast<int4 *>(lds + kMeta)[at] = make_int4((e_k + 128) | (e_v + 128) << 8 | hidden << 16 | int(apart) << 20, 0, int(nan), int(nan >> 32));
    };

    // Raw values of a tile of K and one of V on their way.  A wave's rows lie in one block of 16 keys.  What is past a
    // row's end, or in no page, is read from elsewhere in the cache: it meets zeros of the queries, or is not seen.
    uint4 k_raw[kKPer];
    uint32_t v_raw[kVPer][4];
    auto load_k = [&](int v) {
#pragma unroll
      for (int i = 0; i < kKPer; ++i) {
        const int first = i * kThreads + wave * 64;
        if (kKUnits % kThreads && first >= kKUnits) continue;
        const int n = first + lane, r = n / (DP / 16), byte = n % (DP / 16) * 16, block = first / (DP / 16) / 16;
        const int page = max(uniform(lds_pages[((v - v0) * 4 + block) % kPages]), 0);
        const int64_t slot = (int64_t(head) << a.page_bits) + ((tile_key(u, v) + block * 16) & in_page);
        k_raw[i] = gload_at<uint4>(a.c.k + page * a.c.k_page + slot * a.pitch,
                                   uint32_t(r % 16 * a.pitch + (byte < a.pitch ? byte : 0)));
      }
    };
    auto load_v = [&](int v) {
#pragma unroll
      for (int i = 0; i < kVPer; ++i) {
        const int first = i * kThreads + wave * 64;
        if (kVUnits % kThreads && first >= kVUnits) continue;
        const int n = first + lane, byte = d0 + n % (kVD / 4) * 4, r = n / (kVD / 4) * 4, block = first / (kVD / 4) * 4 / 16;
        const int page = max(uniform(lds_pages[((v - v0) * 4 + block) % kPages]), 0);
        const int64_t slot = (int64_t(head) << a.page_bits) + ((tile_key(u, v) + block * 16) & in_page);
        const int8_t *base = a.c.v + page * a.c.v_page + slot * a.pitch;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v_raw[i][j] = gload_at<uint32_t>(base + j * a.pitch, uint32_t(r % 16 * a.pitch + (byte < a.pitch ? byte : 0)));
      }
    };
    // .. and widened into their buffers
    auto put_k = [&](int v) {
#pragma unroll
      for (int i = 0; i < kKPer; ++i) {
        const int first = i * kThreads + wave * 64;
        if (kKUnits % kThreads && first >= kKUnits) continue;
        const int n = first + lane, r = n / (DP / 16), chunk = n % (DP / 16) * 2;
        const uint32_t w[4] = {k_raw[i].x, k_raw[i].y, k_raw[i].z, k_raw[i].w};
        uint32_t h[8];
        if constexpr (F32) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            h[j] = __builtin_bit_cast(uint32_t, bytes_to_f16(__builtin_amdgcn_perm(0u, w[j / 2] ^ kByteBias, j % 2 ? 0x0c030c02u : 0x0c010c00u)));
        } else {
          const float f = reinterpret_cast<const float *>(lds + kKS)[(v - v0) % kRing * 64 + r];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            h[j] = pack_f16(float(int8_t(w[j / 2] >> (j % 2 * 16))) * f, float(int8_t(w[j / 2] >> (j % 2 * 16 + 8))) * f);
        }
        const int to = (r * kChunks + (chunk ^ (r & kMask))) * 16 + ((v - v0) & 1) * (64 * DP * 2);
        *reinterpret_cast<uint4 *>(lds + to) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(lds + (to ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
      }
    };
    auto put_v = [&](int v, int j0, int j1) {  // columns j0 .. j1 - 1 of a lane's four
#pragma unroll
      for (int i = 0; i < kVPer; ++i) {
        const int first = i * kThreads + wave * 64;
        if (kVUnits % kThreads && first >= kVUnits) continue;
        const int n = first + lane, c = n % (kVD / 4), quad = n / (kVD / 4);
        const float4 f = reinterpret_cast<const float4 *>(lds + kVS)[(v - v0) % kRing * 16 + quad];
        // keys 4 quad .. of a 16-key block are places 8 (quad & 1) + 4 (quad >> 1) .. of its 16
        const int chunk = quad / 4 * 2 + (quad & 1), part = quad >> 1 & 1;
#pragma unroll
        for (int j = j0; j < j1; ++j) {
          uint32_t lo, hi;
          if constexpr (F32) {
            const uint32_t pick = 0x0c040c00u + 0x10001u * j;
            lo = __builtin_bit_cast(uint32_t, bytes_to_f16(__builtin_amdgcn_perm(v_raw[i][1] ^ kByteBias, v_raw[i][0] ^ kByteBias, pick)));
            hi = __builtin_bit_cast(uint32_t, bytes_to_f16(__builtin_amdgcn_perm(v_raw[i][3] ^ kByteBias, v_raw[i][2] ^ kByteBias, pick)));
          } else {
            lo = pack_f16(float(int8_t(v_raw[i][0] >> (8 * j))) * f.x, float(int8_t(v_raw[i][1] >> (8 * j))) * f.y);
            hi = pack_f16(float(int8_t(v_raw[i][2] >> (8 * j))) * f.z, float(int8_t(v_raw[i][3] >> (8 * j))) * f.w);
          }
          const int d = 4 * c + j;
          *reinterpret_cast<uint2 *>(lds + kV + (d * 8 + (chunk ^ ((d ^ d >> 2) & 7))) * 16 + part * 8 + ((v - v0) & 1) * (64 * kVD * 2)) =
              make_uint2(lo, hi);
        }
      }
    };
    // Operands from LDS, kRead at a time, the next ones on their way while these are used.  Their places differ from a
    // lane's first by an exclusive or of a constant.
    constexpr int kRead = 2, kKGroups = 2 * kSteps / kRead, kVGroups = 4 * kBlocks / kRead;
    const int k_first = (col * kChunks + (half ^ (col & kMask))) * 16;
    const int v_first = kV + (col * 8 + (half ^ ((col ^ col >> 2) & 7))) * 16;
    auto read_k = [&](int at, int g, f16x8 (&f)[kRead]) {
#pragma unroll
      for (int j = 0; j < kRead; ++j) {
        const int kb = (kRead * g + j) / kSteps, st = (kRead * g + j) % kSteps;
        f[j] = __builtin_bit_cast(f16x8, *reinterpret_cast<const uint4 *>(lds + (at ^ 32 * st) + kb * 32 * DP * 2));
      }
    };
    auto read_v = [&](int at, int g, f16x8 (&f)[kRead]) {
#pragma unroll
      for (int j = 0; j < kRead; ++j) {
        const int st = (kRead * g + j) / kBlocks, b = (kRead * g + j) % kBlocks;
        f[j] = __builtin_bit_cast(f16x8, *reinterpret_cast<const uint4 *>(lds + (at ^ 32 * st) + b * 32 * 128));
      }
    };
    // The scores of K tile v.
    auto scores = [&](int v, f32x16 (&s)[2]) {
      f16x8 f[2][kRead];
      int at = k_first + ((v - v0) & 1) * (64 * DP * 2);
      pin(at);  // (else the places of all operands are kept in registers)
      read_k(at, 0, f[0]);
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
#pragma unroll
          for (int t = 0; t < kTerms; ++t) s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f[g % 2][j], q[t][st], s[kb], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };

    // Tile v: its scores become weights and outputs, and tile v + 1 is widened.  (In the last tiles what is read and put for
    // the next ones is of no use, and does no harm.)
    auto step = [&](int v) {
      if (!idle) {
        f32x16 s[2];
        scores(v, s);
        const int key = tile_key(u, v), turn = (v - v0) % kRing;
        const int4 meta = reinterpret_cast<const int4 *>(lds + kMeta)[turn];
        const int word = uniform(meta.x), e_k = (word & 255) - 128, e_v = (word >> 8 & 255) - 128, bad = word >> 16 & 15;
        const bool apart = word >> 20;
        const uint64_t nan = uint32_t(uniform(meta.z)) | uint64_t(uint32_t(uniform(meta.w))) << 32;
        const bool whole = bad == 0 && !apart && nan == 0 && all_seen(a, u, key, p_lo, p_hi);
        if constexpr (F32) {
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float4 f = reinterpret_cast<const float4 *>(lds + kKS)[turn * 16 + kb * 8 + g * 2 + half];
              s[kb][4 * g] *= f.x, s[kb][4 * g + 1] *= f.y, s[kb][4 * g + 2] *= f.z, s[kb][4 * g + 3] *= f.w;
            }
        }
        // (held away from zero, where a hidden key's score would be NaN; it is what scores near zero are multiplied with)
        float factor = fminf(fmaxf(F32 ? score : ldexpf(score, e_k), 1e-37f), 1e37f);
        if (!whole) {
          if (apart) {
            scale_apart(s, factor, exps + turn * 16);
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
        top = most * factor + (float(e_v) - kHeadroom<F32>);
        if (__any(top > M + kSlack<F32>)) {
          if (fabsf(top) > kFarScore) top = product(most, factor) + (float(e_v) - kHeadroom<F32>);
          const float m = fmaxf(M, top), fade = __builtin_amdgcn_exp2f(M - m);
          M = m;
          far = __any(fabsf(M) > kFarScore && M != kNoScore);
          l *= fade;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) o[b] *= fade;
        }
        float less = M - float(e_v);
        e_most = max(e_most, e_v);
        const bool low = apart || (!F32 && e_v < e_most - kLowTile);
        if (low || far) {
          if (far) {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i / 16][i % 16] = far_score(product(s[i / 16][i % 16], factor), less, kMostWeight);
            factor = 1.f, less = 0.f;
          }
          if (low) l += sum_exact(s, factor, less, e_v, apart, exps + turn * 16);
        }
        float sum = 0.f;
        uint32_t r[kTerms][16];
#pragma unroll
        for (int n = 0; n < 8; ++n) {  // groups of four keys
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = __builtin_amdgcn_exp2f(fmaf(s[n / 4][n % 4 * 4 + i], factor, -less));
          if constexpr (F32) {
            sum += (p[0] + p[1]) + (p[2] + p[3]);
            const float4 f = reinterpret_cast<const float4 *>(lds + kVS)[turn * 16 + n * 2 + half];
            p[0] *= f.x, p[1] *= f.y, p[2] *= f.z, p[3] *= f.w;
          }
          r[0][2 * n] = pack_f16(p[0], p[1]), r[0][2 * n + 1] = pack_f16(p[2], p[3]);
          if constexpr (F32) {
            const f16x2 r0 = __builtin_bit_cast(f16x2, r[0][2 * n]), r1 = __builtin_bit_cast(f16x2, r[0][2 * n + 1]);
            r[kTerms - 1][2 * n] = pack_f16(p[0] - float(r0.x), p[1] - float(r0.y));
            r[kTerms - 1][2 * n + 1] = pack_f16(p[2] - float(r1.x), p[3] - float(r1.y));
          } else {
            // the sum takes the weights as the outputs do, rounded
            sum = sum_f16(r[0][2 * n + 1], sum_f16(r[0][2 * n], sum));
          }
#pragma unroll
          for (int t = 0; t < kTerms; ++t) pin(r[t][2 * n]), pin(r[t][2 * n + 1]);
        }
        l = fmaf(sum, low ? 0.f : ldexpf(1.f, -e_v), l);
        f16x8 f[2][kRead];
        int at = v_first + ((v - v0) & 1) * (64 * kVD * 2);
        pin(at);
        read_v(at, 0, f[0]);
#pragma unroll
        for (int g = 0; g < kVGroups; ++g) {
          if (g + 1 < kVGroups) read_v(at, g + 1, f[(g + 1) % 2]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < kRead; ++j) {
            const int st = (kRead * g + j) / kBlocks, b = (kRead * g + j) % kBlocks;
#pragma unroll
            for (int t = 0; t < kTerms; ++t)
              o[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                  f[g % 2][j], frag(r[t][4 * st], r[t][4 * st + 1], r[t][4 * st + 2], r[t][4 * st + 3]), o[b], 0, 0, 0);
          }
          // the next tiles, in pieces between the products
          if (g == kVGroups / 8) put_v(v + 1, 0, 2);
          if (g == kVGroups * 3 / 8) put_v(v + 1, 2, 4);
          if (g == kVGroups * 5 / 8) put_k(v + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        put_v(v + 1, 0, 4);
        put_k(v + 1);
      }
      if (v + 2 < v1) load_v(v + 2);
      if (v + 2 < v1) load_k(v + 2);
      if ((v - v0) % NW == 0) {
        put_scales(v + NW + wave);
        load_scales(v + 2 * NW + wave);
      }
      // half the list of pages anew, well before it is needed
      constexpr int kHalf = kPages / 8;
      const int next_half = (v - v0) / kHalf * kHalf + kHalf;
      if ((v - v0) % kHalf == kHalf / 2 && next_half >= 2 * kHalf && v0 + next_half < v1) fetch_pages(v0 + next_half, kHalf);
      lds_barrier();
    };

    // Heads beyond 128 go over their keys once for each half of the values, which leaves the outputs room in the registers;
    // the queries stay, so that the outputs may take their place in memory.
#pragma nounroll
    for (; d0 < DP; d0 += kVD) {
      M = kNoScore, l = 0.f, e_most = -128, far = false;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[b][i] = 0.f;
      if (v0 < v1) {
        fetch_pages(v0, kPages / 4);
        lds_barrier();
        load_k(v0);
        load_v(v0);
        load_scales(v0 + wave);
        put_scales(v0 + wave);
        load_scales(v0 + NW + wave);
        lds_barrier();
        put_k(v0);
        put_v(v0, 0, 4);
        if (v0 + 1 < v1) {
          load_k(v0 + 1);
          load_v(v0 + 1);
        }
        lds_barrier();
        for (int v = v0; v < v1; ++v) step(v);
      }

      // (V in float16 is value * scale / 2^eV; for fp32 value / 512 * scale / 2^eV)
      l = half_sum(l);
      const float up = F32 ? kByteScale : 1.f;
      if (row < row_end) {
        if (u.nsplit == 1) {
          const float inv = l == 0.f ? 0.f : up / l;
          E *to = row_at<E>(a, a.out, u, head, row);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const int d = d0 + b * 32 + g * 8 + half * 4;
              const float f[4] = {o[b][4 * g] * inv, o[b][4 * g + 1] * inv, o[b][4 * g + 2] * inv, o[b][4 * g + 3] * inv};
              store_four(to + d, f, D - d);
            }
        } else {
          const int64_t at = (int64_t(u.slot + uniform(im.y)) * kv + head) * a.s.many_rows + (row - u.row0);
          float *part = reinterpret_cast<float *>(a.ws + a.s.part[ATTN_MANY]) + at * DP + d0;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int g = 0; g < 4; ++g)
              gstore(part + b * 32 + g * 8 + half * 4,
                     make_float4(o[b][4 * g] * up, o[b][4 * g + 1] * up, o[b][4 * g + 2] * up, o[b][4 * g + 3] * up));
          if (half == 0 && d0 == 0) gstore(reinterpret_cast<float *>(a.ws + a.s.stat[ATTN_MANY]) + at * 2, make_float2(M, l));
        }
      }
    }
  }
}

template <int DP, int NW, bool F32>
hipError_t launch_exact(const AttnArgs &a, hipStream_t stream) {
  const auto kernel = attention_exact_kernel<DP, NW, F32>;
  constexpr size_t smem = size_t(2) * 64 * (DP + (DP == 256 ? 128 : DP)) * 2 + 2 * NW * (512 + 16 + 256) + 4096;
  static const bool once = raise_lds_limit(reinterpret_cast<const void *>(kernel), smem);
  (void)once;
  kernel<<<item_grid(a, ATTN_MANY), 64 * NW, smem, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_exact(const AttnArgs &a, int dtype, hipStream_t stream) {
  if (dtype == LORA_BF16) return launch_exact<256, 4, false>(a, stream);
  if (a.s.dp == 64) return launch_exact<64, 4, true>(a, stream);
  if (a.s.dp == 128) return launch_exact<128, 4, true>(a, stream);
  return launch_exact<256, 4, true>(a, stream);
}

}  // namespace lora
