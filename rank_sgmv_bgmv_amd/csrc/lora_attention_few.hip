// Attention of few rows over the 8-bit cache: single tokens, short drafts.
//
// A workgroup takes a piece of a sequence's keys for one cache head; its four
// waves take its tiles of 64 keys in turn and keep a softmax each (running
// maximum M, sum l, outputs O), which meet in LDS at the end.  Rows (queries
// times the query heads of the cache head) lie in kBlocks blocks of 16.
//
//     S^T = K Q^T      16 x 16 x 32 products of float16: keys are rows, queries columns
//     O^T += V^T P^T   the same; P^T comes out of S^T in the lanes that need it
//
// so nothing is exchanged between lanes but the maxima and sums of a column.
// Each lane loads K and V straight from the pages to registers: for K 16 bytes
// of a row (the order of the head's values is the same in Q, so any will do),
// for V the same few columns of 8 rows, whose bytes are paired into float16
// operands as they are widened, which transposes them.
//
// The 8-bit values are exact in float16, as are bf16 queries after a common
// power of two (fp32 ones are two float16 numbers, 22 bits).  Scales enter in
// float32: those of K multiply the scores, those of V, as m = scale / 2^e with e
// common to a tile, the weights.  With s = scale k.q log2 e and t = s + e the
// weights are w = 2^(t - M) m in float16, M the running maximum of t less 14, and
// l = sum 2^(t - M) 2^-e.  So a weight keeps 11 bits while it is above 2^-23 of
// the largest contribution, whatever the values' size down to scales of 2^-60
// (below, e stays): where those of a tile lie more than 2^4 apart, M takes
// each key's own e.
//
// Bound by memory: 64 requests of up to 32768 keys, 8 heads of 128, read 2.94 GB
// in 521 us, 5.6 TB/s, above the rate of a large copy (4.9); 256 requests with a
// window of 4096 take 383 us (5.8 TB/s).  Heads of 64 take 321 us (4.7 TB/s) for
// the 64 requests, of 256 1017 (5.7); in fp32, of 64 352 (4.3), of 128 652 (4.5)
// and of 256 1044 (5.6).  One request over 4097 keys takes 15.5 us, two launches
// whose loads wait for each other: plan, item, unit, pages, keys.  Two workgroups
// a CU (launch bounds) have the loads of a tile and of its follower on their way; a
// register more than 256 costs 5%, which is why what depends on the head is
// computed anew for each item.

#include "lora_attention.hpp"

namespace lora {
namespace {

constexpr int kFewThreads = 256, kFewWaves = 4;

// DP: the head padded, kBlocks: row blocks, F32: queries and outputs in float32.
template <int DP, int kBlocks, bool F32>
__global__ __launch_bounds__(kFewThreads, DP <= 128 && kBlocks == 1 && !F32 ? 2 : 1) void attention_few_kernel(AttnArgs a) {
  typedef std::conditional_t<F32, float, uint16_t> E;
  constexpr int kSteps = DP / 32;             // products of 32 over a head's values
  constexpr int kCols = DP / 16;              // V columns of a lane, and row blocks of V^T
  constexpr int kKB = DP / 64;                // 16-byte pieces of K of a lane and key block
  constexpr int kTerms = F32 ? 2 : 1;
  constexpr int kPart = kBlocks == 1 ? 4 : 2;  // key blocks of a softmax step
  constexpr int kRowPitch = DP + 4;           // floats: rows begin in other banks
  __shared__ float lds_o[kFewWaves][16][kRowPitch];
  __shared__ float lds_m[kFewWaves][kBlocks * 16], lds_l[kFewWaves][kBlocks * 16];

  // (what a workgroup begins with is read at once; its first item lies within the plan whatever that holds)
  int n_items = gload<int>(a.plan + A_ITEMS + ATTN_FEW);
  int2 im = load_item(a, ATTN_FEW, blockIdx.y);
  if (!plan_matches(a)) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicAdd(a.plan + H_ERR, 1);
    return;
  }
  const int lane = threadIdx.x % 64, wave = uniform(threadIdx.x / 64), col = lane % 16, quarter = lane / 16;
  const int kv = a.s.kv_heads;
  n_items = uniform(n_items);

  for (int item = blockIdx.y; item < n_items; item += gridDim.y) {
    const int head = opaque(blockIdx.x), D = opaque(a.s.head_dim);
    const AttnUnit u = load_unit(a, ATTN_FEW, uniform(im.x));
    int v0, v1;
    const int piece = uniform(im.y);
    piece_tiles(u, piece, v0, v1);
    const int blocks = (u.rows + 15) / 16;  // live row blocks

    // queries: lane (col, quarter) holds values quarter * DP / 4 .. of row col
    f16x8 q[kBlocks][kTerms][kSteps];
    RowSight sight[kBlocks];
    UnitKeys keys;
    keys.set(a, u, 0, u.n - 1);
    const int p_lo = u.len - u.n, p_hi = u.len - 1;  // positions of the rows
    float score[kBlocks];  // what a row's products are multiplied with: its queries are over a power of two, 2^-x
    {
      const E *safe = row_at<const E>(a, a.q, u, head, 0);
      float f[kBlocks][DP / 4];
      float top[kBlocks];
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        top[b] = 0.f;
        const int row = b * 16 + col;
        const bool live = row < u.rows;
        load_query<E, DP / 4>(row_at<const E>(a, a.q, u, head, live ? row : 0), safe, live, quarter * (DP / 4), D, f[b]);
#pragma unroll
        for (int i = 0; i < DP / 4; ++i) {
          const float v = fabsf(f[b][i]);
          top[b] = fmaxf(top[b], v < __uint_as_float(0x7f800000u) ? v : 0.f);
        }
        sight[b].set(a, u, row);
      }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        top[b] = quarters_max(top[b]);
        const int x = top[b] > 0.f ? min(15 - __builtin_amdgcn_frexp_expf(top[b]), 100) : 0;
        score[b] = a.scale * ldexpf(1.f, -x) * kByteScale;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          uint32_t w[kTerms][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float y0 = ldexpf(f[b][8 * s + 2 * i], x), y1 = ldexpf(f[b][8 * s + 2 * i + 1], x);
            w[0][i] = pack_f16(y0, y1);
            if constexpr (F32) {
              const f16x2 r = __builtin_bit_cast(f16x2, w[0][i]);
              w[kTerms - 1][i] = pack_f16(y0 - float(r.x), y1 - float(r.y));
            }
          }
#pragma unroll
          for (int t = 0; t < kTerms; ++t) q[b][t][s] = frag(w[t][0], w[t][1], w[t][2], w[t][3]);
        }
      }
    }

    f32x4 o[kBlocks][kCols];
    float M[kBlocks], l[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      M[b] = kNoScore, l[b] = 0.f;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[b][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    // the wave's tiles: v0 + wave, v0 + wave + 4, ..; the pages of 16 of them at a time, one key block a lane
    int ids = -1;
    uint4 k_raw[4][kKB];
    uint32_t v_raw[16][(kCols + 3) / 4];
    float ks[4][4], vs[4][4];
    uint32_t bad = 0;  // key blocks of the loaded tile whose keys are not seen
    auto load_ids = [&](int v) {
      const int mine = v + (lane / 4) * kFewWaves;
      ids = block_page(a, u, keys, tile_key(u, mine) + (lane % 4) * 16, mine < v1);
    };
    auto page_of = [&](int turn, int kb) { return __builtin_amdgcn_readlane(ids, (turn % 16) * 4 + kb); };
    // (what is past a row's end is read from its begin: it meets zeros of the queries, or makes outputs that are not there)
    auto load_k = [&](int v, int turn) {
      const int key = tile_key(u, v);
      bad = 0;
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        const int page = page_of(turn, kb);
        const int slot = (key + kb * 16) & ((1 << a.page_bits) - 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) ks[kb][i] = vs[kb][i] = 0.f;
#pragma unroll
        for (int i = 0; i < kKB; ++i) k_raw[kb][i] = make_uint4(0u, 0u, 0u, 0u);
        if (page < 0) {
          bad |= 1u << kb;
          continue;
        }
        const int64_t at = (int64_t(head) << a.page_bits) + slot;
        const int8_t *base = a.c.k + page * a.c.k_page + at * a.pitch;
#pragma unroll
        for (int i = 0; i < kKB; ++i) {
          const int byte = quarter * (DP / 4) + i * 16;
          k_raw[kb][i] = gload_at<uint4>(base, uint32_t(col * a.pitch + (byte < a.pitch ? byte : 0)));
        }
        const float4 k4 = gload_at<float4>(a.c.k_scale + page * a.c.k_scale_page + at, uint32_t(quarter * 16));
        const float4 v4 = gload_at<float4>(a.c.v_scale + page * a.c.v_scale_page + at, uint32_t(quarter * 16));
        ks[kb][0] = k4.x, ks[kb][1] = k4.y, ks[kb][2] = k4.z, ks[kb][3] = k4.w;
        vs[kb][0] = v4.x, vs[kb][1] = v4.y, vs[kb][2] = v4.z, vs[kb][3] = v4.w;
      }
    };
    const uint32_t v_off = uint32_t(4 * quarter * a.pitch + (col * kCols < a.pitch ? col * kCols : 0));
    auto load_v = [&](int v, int turn) {
      const int key = tile_key(u, v);
#pragma unroll
      for (int kb = 0; kb < 4; ++kb) {
        const int page = page_of(turn, kb);
        const int slot = (key + kb * 16) & ((1 << a.page_bits) - 1);
        const int8_t *base = a.c.v + max(page, 0) * a.c.v_page + ((int64_t(head) << a.page_bits) + slot) * a.pitch;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t *to = v_raw[4 * kb + i];
#pragma unroll
          for (int j = 0; j < (kCols + 3) / 4; ++j) to[j] = 0u;
          if (page >= 0) {
            if constexpr (kCols == 4) {
              to[0] = gload_at<uint32_t>(base + i * a.pitch, v_off);
            } else if constexpr (kCols == 8) {
              const uint2 w = gload_at<uint2>(base + i * a.pitch, v_off);
              to[0] = w.x, to[1] = w.y;
            } else {
              const uint4 w = gload_at<uint4>(base + i * a.pitch, v_off);
              to[0] = w.x, to[1] = w.y, to[2] = w.z, to[3] = w.w;
            }
          }
        }
      }
    };

    int turn = 0;
    if (v0 + wave < v1) {
      load_ids(v0 + wave);
      load_k(v0 + wave, 0);
      load_v(v0 + wave, 0);
    }
    for (int v = v0 + wave; v < v1; v += kFewWaves, ++turn) {
      const int key = tile_key(u, v);
      const bool whole = bad == 0 && all_seen(a, u, key, p_lo, p_hi);
      const uint32_t hidden = bad;
      const int next = v + kFewWaves;
      // the tile's exponent, and its scales
      float kf[4][4], vm[4][4];
      int e;
      uint32_t nans = 0;  // keys whose scales are none
      bool apart;         // keys have exponents of their own
      {
        // (the bits of floats that are not negative are in their order)
        uint32_t top = 0, most = 0, all_least = ~0u, least = ~0u;  // of V, of K, of V, of V's keys that are seen
        if (!whole) {
#pragma unroll
          for (int kb = 0; kb < 4; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool there = keys.seen(a, key + kb * 16 + quarter * 4 + i) & !(hidden >> kb & 1);
              least = min(least, there ? __float_as_uint(vs[kb][i]) : ~0u);
              vs[kb][i] = there ? vs[kb][i] : 0.f;
            }
        }
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = __float_as_uint(vs[kb][i]);
            top = max(top, x), most = max(most, __float_as_uint(ks[kb][i])), all_least = min(all_least, x);
          }
        if (__any(max(top, most) >= kNoScale)) {
          // (such values become zeros: the rows that see them get their NaN from the weight)
          top = 0;
#pragma unroll
          for (int kb = 0; kb < 4; ++kb)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool none = __float_as_uint(vs[kb][i]) >= kNoScale;
              nans |= none || __float_as_uint(ks[kb][i]) >= kNoScale ? 1u << (4 * kb + i) : 0u;
              vs[kb][i] = none ? 0.f : vs[kb][i];
              top = max(top, __float_as_uint(vs[kb][i]));
            }
        }
        e = uniform(tile_exponent(quarters_max(__uint_as_float(top))));
        if (whole) least = all_least;
        apart = e > kLeastExponent && __any(least < __float_as_uint(ldexpf(1.f, e - 1 - kSpreadV<true>)));
        const float down = ldexpf(1.f, -e);
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
          for (int i = 0; i < 4; ++i) kf[kb][i] = kBlocks == 1 ? ks[kb][i] * score[0] : ks[kb][i], vm[kb][i] = vs[kb][i] * down;
      }
      const bool poisoned = __any(nans != 0);

      // kPart key blocks of 16 at a time.  (Products are made for every row block, live or not.  With those of the second
      // behind a branch the compiler counted the wait between a product and the first read of its result along the longer
      // way alone: where the branch was taken, scores were read before they were there.)
#pragma unroll
      for (int k0 = 0; k0 < 4; k0 += kPart) {
        // scores
        f32x4 s[kPart][kBlocks];
#pragma unroll
        for (int kb = 0; kb < kPart; ++kb) {
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) s[kb][b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int st = 0; st < kSteps; ++st) {
            const uint4 w = k_raw[k0 + kb][st / 2];
            const uint32_t w0 = (st % 2 ? w.z : w.x) ^ kByteBias, w1 = (st % 2 ? w.w : w.y) ^ kByteBias;
            const f16x2 h[4] = {bytes_to_f16(__builtin_amdgcn_perm(0u, w0, 0x0c010c00u)),
                                bytes_to_f16(__builtin_amdgcn_perm(0u, w0, 0x0c030c02u)),
                                bytes_to_f16(__builtin_amdgcn_perm(0u, w1, 0x0c010c00u)),
                                bytes_to_f16(__builtin_amdgcn_perm(0u, w1, 0x0c030c02u))};
            const f16x8 kf16 = __builtin_shufflevector(__builtin_shufflevector(h[0], h[1], 0, 1, 2, 3),
                                                       __builtin_shufflevector(h[2], h[3], 0, 1, 2, 3), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
              for (int t = 0; t < kTerms; ++t)
                s[kb][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf16, q[b][t][st], s[kb][b], 0, 0, 0);
          }
        }
        if (k0 + kPart == 4 && next < v1) {
          // the next tile's keys are on their way from here on
          if ((turn + 1) % 16 == 0) load_ids(next);
          load_k(next, turn + 1);
        }
        // weights
        f16x8 w[kBlocks][kTerms][kPart / 2] = {};
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
          if (b == 0 || b < blocks) {
            uint32_t seen = 0xffffu;
#pragma unroll
            for (int kb = 0; kb < kPart; ++kb)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float f = kBlocks == 1 ? kf[k0 + kb][i] : kf[k0 + kb][i] * score[b];
                s[kb][b][i] = product(s[kb][b][i], f);
              }
            if (!whole) {
              // (a lane's keys are four of each sixteen)
              const uint64_t keys_seen = sight[b].seen(a, u, key, hidden) >> 4 * quarter;
              seen = 0;
#pragma unroll
              for (int kb = 0; kb < 4; ++kb) seen |= uint32_t(keys_seen >> 16 * kb & 15) << 4 * kb;
#pragma unroll
              for (int kb = 0; kb < kPart; ++kb)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  s[kb][b][i] = seen >> (4 * (k0 + kb) + i) & 1 ? s[kb][b][i] : -__builtin_inff();
            }
            float top = -__builtin_inff();
#pragma unroll
            for (int kb = 0; kb < kPart; ++kb)
#pragma unroll
              for (int i = 0; i < 4; ++i) top = fmaxf(top, s[kb][b][i]);
            const int least_own = max(kLeastExponent - e, -100);
            if (apart) {
              // each with its own exponent: those of small scales may have large weights, which float32 holds
              top = -__builtin_inff();
#pragma unroll
              for (int kb = 0; kb < kPart; ++kb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float m = vm[k0 + kb][i];
                  top = fmaxf(top, s[kb][b][i] + float(m > 0.f ? max(__builtin_amdgcn_frexp_expf(m), least_own) : least_own));
                }
            }
            top = quarters_max(top) + float(e) - kHeadroom<true>;
            const float m = fmaxf(M[b], top);
            float less = m - float(e);
            const float fade = __builtin_amdgcn_exp2f(M[b] - m);
            M[b] = m;
            if (__any(fabsf(less) > kFarScore && m != kNoScore)) {
#pragma unroll
              for (int kb = 0; kb < kPart; ++kb)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  s[kb][b][i] = far_score(s[kb][b][i], less, kMostWeight - fmaxf(__builtin_amdgcn_logf(vm[k0 + kb][i]), float(least_own)));
              less = 0.f;
            }
            float sum = 0.f;
#pragma unroll
            for (int kb = 0; kb < kPart; ++kb)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[kb][b][i] = __builtin_amdgcn_exp2f(s[kb][b][i] - less);
            if (poisoned) {
#pragma unroll
              for (int kb = 0; kb < kPart; ++kb)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (nans & seen & 1u << (4 * (k0 + kb) + i)) s[kb][b][i] = __builtin_nanf("");
            }
            uint32_t r[kTerms][2 * kPart];
#pragma unroll
            for (int kb = 0; kb < kPart; ++kb) {
              float p[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                sum += s[kb][b][i];
                p[i] = s[kb][b][i] * vm[k0 + kb][i];
              }
              r[0][2 * kb] = pack_f16(p[0], p[1]), r[0][2 * kb + 1] = pack_f16(p[2], p[3]);
              if constexpr (F32) {
                const f16x2 r0 = __builtin_bit_cast(f16x2, r[0][2 * kb]), r1 = __builtin_bit_cast(f16x2, r[0][2 * kb + 1]);
                r[kTerms - 1][2 * kb] = pack_f16(p[0] - float(r0.x), p[1] - float(r0.y));
                r[kTerms - 1][2 * kb + 1] = pack_f16(p[2] - float(r1.x), p[3] - float(r1.y));
              }
            }
            l[b] = fmaf(l[b], fade, sum * ldexpf(1.f, -e));
            if (__any(fade != 1.f)) {
#pragma unroll
              for (int c = 0; c < kCols; ++c) o[b][c] *= fade;
            }
#pragma unroll
            for (int t = 0; t < kTerms; ++t)
#pragma unroll
              for (int h = 0; h < kPart / 2; ++h)
                w[b][t][h] = frag(r[t][4 * h], r[t][4 * h + 1], r[t][4 * h + 2], r[t][4 * h + 3]);
          }
        // outputs
#pragma unroll
        for (int h = 0; h < kPart / 2; ++h)
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            constexpr uint32_t kPick[4] = {0x0c040c00u, 0x0c050c01u, 0x0c060c02u, 0x0c070c03u};
            f16x2 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // keys 0, 1 and 2, 3 of the first block of 16, then of the second
              const int n = 4 * (k0 + 2 * h + i / 2) + 2 * (i % 2);
              x[i] = bytes_to_f16(__builtin_amdgcn_perm(v_raw[n + 1][c / 4] ^ kByteBias, v_raw[n][c / 4] ^ kByteBias, kPick[c % 4]));
            }
            const f16x8 vf = __builtin_shufflevector(__builtin_shufflevector(x[0], x[1], 0, 1, 2, 3),
                                                     __builtin_shufflevector(x[2], x[3], 0, 1, 2, 3), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
              for (int t = 0; t < kTerms; ++t)
                o[b][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, w[b][t][h], o[b][c], 0, 0, 0);
          }
      }
      if (next < v1) load_v(next, turn + 1);
    }

    // the waves' softmaxes meet
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      l[b] = quarters_sum(l[b]);
      if (quarter == 0) lds_m[wave][b * 16 + col] = M[b], lds_l[wave][b * 16 + col] = l[b];
    }
    lds_barrier();
    const int row_in = threadIdx.x / 16, d0 = threadIdx.x % 16 * kCols;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
      if (b == 0 || b < blocks) {
        float m = lds_m[0][b * 16 + col];
#pragma unroll
        for (int x = 1; x < kFewWaves; ++x) m = fmaxf(m, lds_m[x][b * 16 + col]);
        const float fade = __builtin_amdgcn_exp2f(M[b] - m);
        if (b > 0) lds_barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < kCols; c += 4)
            *reinterpret_cast<float4 *>(&lds_o[wave][col][(4 * quarter + i) * kCols + c]) =
                make_float4(o[b][c][i] * fade, o[b][c + 1][i] * fade, o[b][c + 2][i] * fade, o[b][c + 3][i] * fade);
        lds_barrier();
        const int row = b * 16 + row_in;
        if (row < u.rows) {
          float mr = lds_m[0][row], sum = 0.f;
#pragma unroll
          for (int x = 1; x < kFewWaves; ++x) mr = fmaxf(mr, lds_m[x][row]);
#pragma unroll
          for (int x = 0; x < kFewWaves; ++x) sum += lds_l[x][row] * __builtin_amdgcn_exp2f(lds_m[x][row] - mr);
          float y[kCols];
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            float4 t = *reinterpret_cast<const float4 *>(&lds_o[0][row_in][d0 + c]);
#pragma unroll
            for (int x = 1; x < kFewWaves; ++x) {
              const float4 n = *reinterpret_cast<const float4 *>(&lds_o[x][row_in][d0 + c]);
              t.x += n.x, t.y += n.y, t.z += n.z, t.w += n.w;
            }
            y[c] = t.x * kByteScale, y[c + 1] = t.y * kByteScale, y[c + 2] = t.z * kByteScale, y[c + 3] = t.w * kByteScale;
          }
          if (u.nsplit == 1) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            E *to = row_at<E>(a, a.out, u, head, row) + d0;
#pragma unroll
            for (int c = 0; c < kCols; c += 4) {
              const float f[4] = {y[c] * inv, y[c + 1] * inv, y[c + 2] * inv, y[c + 3] * inv};
              store_four(to + c, f, D - d0 - c);
            }
          } else {
            const int64_t at = (int64_t(u.slot + piece) * kv + head) * a.s.few_rows + row;
            float *part = reinterpret_cast<float *>(a.ws + a.s.part[ATTN_FEW]) + at * DP + d0;
#pragma unroll
            for (int c = 0; c < kCols; c += 4) gstore(part + c, make_float4(y[c], y[c + 1], y[c + 2], y[c + 3]));
            if (d0 == 0) gstore(reinterpret_cast<float *>(a.ws + a.s.stat[ATTN_FEW]) + at * 2, make_float2(mr, sum));
          }
        }
      }
    lds_barrier();  // the next item writes what was read here
    if (item + int(gridDim.y) < n_items) im = load_item(a, ATTN_FEW, item + gridDim.y);
  }
}

template <int DP, int kBlocks, bool F32>
void launch_few(const AttnArgs &a, hipStream_t stream) {
  attention_few_kernel<DP, kBlocks, F32><<<item_grid(a, ATTN_FEW), kFewThreads, 0, stream>>>(a);
}

}  // namespace

hipError_t launch_attention_few(const AttnArgs &a, int dtype, hipStream_t stream) {
  const int dp = a.s.dp, b = a.s.few_blocks;
  if (dtype == LORA_BF16) {
    if (dp == 64) b == 1 ? launch_few<64, 1, false>(a, stream) : launch_few<64, 2, false>(a, stream);
    else if (dp == 128) b == 1 ? launch_few<128, 1, false>(a, stream) : launch_few<128, 2, false>(a, stream);
    else b == 1 ? launch_few<256, 1, false>(a, stream) : launch_few<256, 2, false>(a, stream);
  } else {
    if (dp == 64) b == 1 ? launch_few<64, 1, true>(a, stream) : launch_few<64, 2, true>(a, stream);
    else if (dp == 128) b == 1 ? launch_few<128, 1, true>(a, stream) : launch_few<128, 2, true>(a, stream);
    else launch_few<256, 1, true>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace lora
