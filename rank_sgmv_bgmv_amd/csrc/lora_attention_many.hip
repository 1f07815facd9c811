// Attention of many rows over the 8-bit cache (prompts, long drafts), and the
// joining of cut units.
//
// A workgroup takes 32 rows a wave of a sequence's (query, query head) pairs for
// one cache head, and goes over their key tiles of 64.  A tile is widened to
// float16 once for all waves and laid in LDS, K as it is and V transposed, two
// tiles in turn: while one is used the next is converted and the one after it is
// on its way from memory.
//
//     S^T = K Q^T      32 x 32 x 16 products of float16: keys are rows, queries columns
//     O^T += V^T P^T   the same; P^T comes out of S^T in the lanes that need it
//
// V^T's keys stand in LDS in the order in which a lane holds its weights, so
// that an operand is 16 bytes in a row; pieces of 16 bytes are exchanged within
// rows so that neighbouring lanes meet different banks.
//
// For bf16 the scales go into the float16 values, over a power of two common to
// a tile (eK, eV): one rounding of 2^-12 a value, as many as the weights have,
// and nothing is left to do per score but exp2.  For fp32 the 8-bit values are
// widened exactly, the scales meet scores and weights in float32, and queries
// and weights are two float16 numbers each.  Maximum and sum as in the kernel
// for few rows.

#include "lora_attention.hpp"

namespace lora {
namespace {

// NW waves; DP: the head padded; F32: queries and outputs in float32.
template <int DP, int NW, bool F32>
__global__ __launch_bounds__(64 * NW, NW / 4) void attention_many_kernel(AttnArgs a) {
  typedef std::conditional_t<F32, float, uint16_t> E;
  constexpr int kThreads = 64 * NW, kSteps = DP / 16, kBlocks = DP / 32, kTerms = F32 ? 2 : 1;
  constexpr int kChunks = DP / 8;               // 16-byte pieces of a K row
  constexpr int kMask = kChunks < 16 ? kChunks - 1 : 15;
  constexpr int kKUnits = 64 * DP / 16, kKPer = (kKUnits + kThreads - 1) / kThreads;
  constexpr int kVUnits = 16 * DP / 4, kVPer = (kVUnits + kThreads - 1) / kThreads;
  constexpr int kPages = 1024;                  // key blocks whose pages are looked up at once
  extern __shared__ __align__(16) char lds[];
  uint4 *lds_k = reinterpret_cast<uint4 *>(lds);                      // [2][64][kChunks]
  uint4 *lds_v = lds_k + 2 * 64 * kChunks;                            // [2][DP][8]
  float *lds_s = reinterpret_cast<float *>(lds_v + 2 * DP * 8);       // F32: [2][2][64] scales of K and V
  int *lds_pages = reinterpret_cast<int *>(lds_s + (F32 ? 256 : 0));  // [kPages]

  if (!plan_matches(a)) {
    if (!a.s.few_blocks && blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(a.plan + H_ERR, 1);  // (else counted there)
    return;
  }
  const int tid = threadIdx.x, lane = tid % 64, wave = uniform(tid / 64), col = lane % 32, half = lane / 32;
  const int kv = a.s.kv_heads, D = a.s.head_dim;
  const int64_t n_items = int64_t(uniform(gload<int>(a.plan + A_ITEMS + ATTN_MANY))) * kv;

  for (int64_t it = blockIdx.x; it < n_items; it += gridDim.x) {
    const int item = int(it / kv), head = int(it % kv);
    const int2 im = gload<int2>(reinterpret_cast<const char *>(a.plan) + a.s.item[ATTN_MANY] + size_t(item) * 8);
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
      const E *p = row < row_end ? row_at<const E>(a, a.q, u, head, row) : nullptr;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const int d = 16 * s + 8 * half;
        load_query<E, 8>(p + d, row < row_end ? D - d : 0, f[s]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float v = fabsf(f[s][i]);
          top = fmaxf(top, v < __uint_as_float(0x7f800000u) ? v : 0.f);
        }
      }
      top = wave_max_f(top);
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

    // staging: raw values of a tile and the scales they are widened with
    uint4 k_raw[kKPer];
    uint32_t v_raw[kVPer][4];
    float k_sc[kKPer], top_k = 0.f, top_v = 0.f;
    float4 v_sc[kVPer];
    int e_k = 0, e_v = 0, bad = 0;
    uint64_t nan = 0;

    auto fetch_pages = [&](int v) {  // of tiles v .. v + kPages / 4
      lds_barrier();
      for (int i = tid; i < kPages; i += kThreads) {
        const int t = v + i / 4;
        lds_pages[i] = t < v1 ? block_page(a, u, tile_key(u, t) + (i % 4) * 16) : -1;
      }
      lds_barrier();
    };
    auto load_tile = [&](int v) {
      const int key = tile_key(u, v), at = (v - v0) % (kPages / 4) * 4;
      const int in_page = (1 << a.page_bits) - 1;
      const int4 ids = *reinterpret_cast<const int4 *>(lds_pages + at);
      bad = uniform((ids.x < 0 ? 1 : 0) | (ids.y < 0 ? 2 : 0) | (ids.z < 0 ? 4 : 0) | (ids.w < 0 ? 8 : 0));
#pragma unroll
      for (int i = 0; i < kKPer; ++i) {
        const int n = i * kThreads + tid, r = n / (DP / 16), byte = n % (DP / 16) * 16;
        k_raw[i] = make_uint4(0u, 0u, 0u, 0u);
        k_sc[i] = 0.f;
        if (kKUnits % kThreads && n >= kKUnits) continue;
        const int page = lds_pages[at + r / 16];
        if (page >= 0) {
          const int64_t slot = (int64_t(head) << a.page_bits) + ((key + r) & in_page);
          if (byte < a.pitch) k_raw[i] = gload<uint4>(a.c.k + page * a.c.k_page + slot * a.pitch + byte);
          k_sc[i] = gload<float>(a.c.k_scale + page * a.c.k_scale_page + slot);
        }
      }
#pragma unroll
      for (int i = 0; i < kVPer; ++i) {
        const int n = i * kThreads + tid, byte = n % (DP / 4) * 4, r = n / (DP / 4) * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) v_raw[i][j] = 0u;
        v_sc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (kVUnits % kThreads && n >= kVUnits) continue;
        const int page = lds_pages[at + r / 16];
        if (page >= 0) {
          const int64_t slot = (int64_t(head) << a.page_bits) + ((key + r) & in_page);
          const int8_t *p = a.c.v + page * a.c.v_page + slot * a.pitch + byte;
          if (byte < a.pitch) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v_raw[i][j] = gload<uint32_t>(p + j * a.pitch);
          }
          v_sc[i] = gload<float4>(a.c.v_scale + page * a.c.v_scale_page + slot);
        }
      }
      // every wave finds the tile's largest scales by itself
      top_k = top_v = 0.f;
      const int page = lds_pages[at + lane / 16];
      if (page >= 0) {
        const int64_t slot = (int64_t(head) << a.page_bits) + ((key + lane) & in_page);
        top_k = gload<float>(a.c.k_scale + page * a.c.k_scale_page + slot);
        top_v = gload<float>(a.c.v_scale + page * a.c.v_scale_page + slot);
      }
    };
    auto put_tile = [&](int buf) {
      nan = __ballot(top_v != top_v);
      if constexpr (F32) {
        if (wave == 0) lds_s[(buf * 2) * 64 + lane] = top_k;
      }
      const float tk = wave_max_f(fmaxf(top_k, 0.f)), tv = wave_max_f(fmaxf(top_v, 0.f));
      e_k = uniform(tile_exponent(tk)), e_v = uniform(tile_exponent(tv));
      const float down_k = ldexpf(1.f, -e_k), down_v = ldexpf(1.f, -e_v);
      if constexpr (F32) {
        if (wave == 0) lds_s[(buf * 2 + 1) * 64 + lane] = top_v == top_v ? top_v * down_v : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kKPer; ++i) {
        const int n = i * kThreads + tid, r = n / (DP / 16), chunk = n % (DP / 16) * 2;
        if (kKUnits % kThreads && n >= kKUnits) continue;
        const uint32_t w[4] = {k_raw[i].x, k_raw[i].y, k_raw[i].z, k_raw[i].w};
        uint32_t h[8];
        if constexpr (F32) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            h[j] = __builtin_bit_cast(uint32_t, bytes_to_f16(__builtin_amdgcn_perm(0u, w[j / 2] ^ kByteBias, j % 2 ? 0x0c030c02u : 0x0c010c00u)));
        } else {
          const float f = k_sc[i] * down_k;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            h[j] = pack_f16(float(int8_t(w[j / 2] >> (j % 2 * 16))) * f, float(int8_t(w[j / 2] >> (j % 2 * 16 + 8))) * f);
        }
        uint4 *to = lds_k + (buf * 64 + r) * kChunks;
        to[chunk ^ (r & kMask)] = make_uint4(h[0], h[1], h[2], h[3]);
        to[(chunk + 1) ^ (r & kMask)] = make_uint4(h[4], h[5], h[6], h[7]);
      }
#pragma unroll
      for (int i = 0; i < kVPer; ++i) {
        const int n = i * kThreads + tid, c = n % (DP / 4), quad = n / (DP / 4);
        if (kVUnits % kThreads && n >= kVUnits) continue;
        float f[4] = {v_sc[i].x * down_v, v_sc[i].y * down_v, v_sc[i].z * down_v, v_sc[i].w * down_v};
        // NaN scales: the rows that see the key get their NaN from its weight
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = f[j] == f[j] ? f[j] : 0.f;
        // keys 4 quad .. of a 16-key block are places 8 (quad & 1) + 4 (quad >> 1) .. of its 16
        const int chunk = quad / 4 * 2 + (quad & 1), part = quad >> 1 & 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t lo, hi;
          if constexpr (F32) {
            const uint32_t pick = 0x0c040c00u + 0x10001u * j;
            lo = __builtin_bit_cast(uint32_t, bytes_to_f16(__builtin_amdgcn_perm(v_raw[i][1] ^ kByteBias, v_raw[i][0] ^ kByteBias, pick)));
            hi = __builtin_bit_cast(uint32_t, bytes_to_f16(__builtin_amdgcn_perm(v_raw[i][3] ^ kByteBias, v_raw[i][2] ^ kByteBias, pick)));
          } else {
            lo = pack_f16(float(int8_t(v_raw[i][0] >> (8 * j))) * f[0], float(int8_t(v_raw[i][1] >> (8 * j))) * f[1]);
            hi = pack_f16(float(int8_t(v_raw[i][2] >> (8 * j))) * f[2], float(int8_t(v_raw[i][3] >> (8 * j))) * f[3]);
          }
          const int d = 4 * c + j;
          uint2 *to = reinterpret_cast<uint2 *>(lds_v + (buf * DP + d) * 8 + (chunk ^ ((d ^ d >> 2) & 7)));
          to[part] = make_uint2(lo, hi);
        }
      }
    };

    auto use_tile = [&](int buf, int key, int ek, int ev, int hidden, uint64_t nans) {
      // rows that see nothing of the tile: before its first key, or beyond the window
      if (idle || (!a.tree && key > p_hi) || (p_lo - (key + kKeyTile - 1) >= a.window && key >= a.sinks)) return;
      const bool whole = hidden == 0 && nans == 0 && all_seen(a, u, key, p_lo, p_hi);
      f32x16 s[2];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][i] = 0.f;
        const int r = kb * 32 + col;
        const uint4 *from = lds_k + (buf * 64 + r) * kChunks;
#pragma unroll
        for (int st = 0; st < kSteps; ++st) {
          const f16x8 kf = __builtin_bit_cast(f16x8, from[(2 * st + half) ^ (r & kMask)]);
#pragma unroll
          for (int t = 0; t < kTerms; ++t) s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, q[t][st], s[kb], 0, 0, 0);
        }
      }
      if constexpr (F32) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float4 f = *reinterpret_cast<const float4 *>(lds_s + buf * 128 + kb * 32 + g * 8 + half * 4);
            s[kb][4 * g] *= f.x, s[kb][4 * g + 1] *= f.y, s[kb][4 * g + 2] *= f.z, s[kb][4 * g + 3] *= f.w;
          }
      }
      uint32_t seen = 0xffffffffu;
      if (!whole) {
        seen = 0;
#pragma nounroll
        for (int n = 0; n < 32; ++n) {
          const int at = n / 4 * 8 + half * 4 + n % 4;
          seen |= !(hidden >> (at / 16) & 1) && sight.sees(a, u, key + at) ? 1u << n : 0u;
        }
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[kb][i] = seen >> (kb * 16 + i) & 1 ? s[kb][i] : -__builtin_inff();
      }
      // (held away from zero, where a hidden key's score would be NaN; it is what scores near zero are multiplied with)
      const float factor = fminf(fmaxf(F32 ? score : ldexpf(score, ek), 1e-37f), 1e37f);
      float top = -__builtin_inff();
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kb][i]);
      top = half_max(top);
      const float m = fmaxf(M, top * factor + float(ev) - 14.f), less = m - float(ev);
      const float fade = __builtin_amdgcn_exp2f(M - m);
      M = m;
      float sum = 0.f;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[kb][i] = __builtin_amdgcn_exp2f(fmaf(s[kb][i], factor, -less));
      if (nans) {
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if ((nans >> (kb * 32 + i / 4 * 8 + half * 4 + i % 4) & 1) && (seen >> (kb * 16 + i) & 1)) s[kb][i] = __builtin_nanf("");
      }
      uint32_t r[kTerms][16];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] = s[kb][4 * g + i];
            sum += p[i];
          }
          if constexpr (F32) {
            const float4 f = *reinterpret_cast<const float4 *>(lds_s + buf * 128 + 64 + kb * 32 + g * 8 + half * 4);
            p[0] *= f.x, p[1] *= f.y, p[2] *= f.z, p[3] *= f.w;
          }
          uint32_t *to = r[0] + kb * 8 + 2 * g;
          to[0] = pack_f16(p[0], p[1]), to[1] = pack_f16(p[2], p[3]);
          if constexpr (F32) {
            const f16x2 r0 = __builtin_bit_cast(f16x2, to[0]), r1 = __builtin_bit_cast(f16x2, to[1]);
            r[kTerms - 1][kb * 8 + 2 * g] = pack_f16(p[0] - float(r0.x), p[1] - float(r0.y));
            r[kTerms - 1][kb * 8 + 2 * g + 1] = pack_f16(p[2] - float(r1.x), p[3] - float(r1.y));
          }
        }
      l = fmaf(l, fade, sum * ldexpf(1.f, -ev));
      if (__any(fade != 1.f)) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) o[b] *= fade;
      }
#pragma unroll
      for (int st = 0; st < 4; ++st)
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const int d = b * 32 + col;
          const f16x8 vf = __builtin_bit_cast(f16x8, lds_v[(buf * DP + d) * 8 + ((2 * st + half) ^ ((d ^ d >> 2) & 7))]);
#pragma unroll
          for (int t = 0; t < kTerms; ++t)
            o[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, frag(r[t][4 * st], r[t][4 * st + 1], r[t][4 * st + 2], r[t][4 * st + 3]), o[b], 0, 0, 0);
        }
    };

    if (v0 < v1) {
      fetch_pages(v0);
      load_tile(v0);
      // what the tile in use was put with (bad: of the tile that is being loaded)
      int hidden = bad;
      put_tile(0);
      if (v0 + 1 < v1) load_tile(v0 + 1);
      lds_barrier();
      for (int v = v0; v < v1; ++v) {
        const int buf = (v - v0) & 1, key = tile_key(u, v), ek = e_k, ev = e_v, hid = hidden;
        const uint64_t nans = nan;
        if (v + 1 < v1) {
          hidden = bad;
          put_tile(buf ^ 1);
          if (v + 2 < v1) {
            if ((v + 2 - v0) % (kPages / 4) == 0) fetch_pages(v + 2);
            load_tile(v + 2);
          }
        }
        use_tile(buf, key, ek, ev, hid, nans);
        lds_barrier();
      }
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
                   make_float4(o[b][4 * g] * up, o[b][4 * g + 1] * up, o[b][4 * g + 2] * up, o[b][4 * g + 3] * up));
        if (half == 0) gstore(reinterpret_cast<float *>(a.ws + a.s.stat[ATTN_MANY]) + at * 2, make_float2(M, l));
      }
    }
  }
}

template <int DP, int NW, bool F32>
hipError_t launch_many(const AttnArgs &a, hipStream_t stream) {
  const auto kernel = attention_many_kernel<DP, NW, F32>;
  constexpr size_t smem = size_t(2) * 64 * DP * 2 * 2 + (F32 ? 1024 : 0) + 4096;
  static const bool once = raise_lds_limit(reinterpret_cast<const void *>(kernel), smem);
  (void)once;
  const int64_t items = int64_t(a.s.items[ATTN_MANY]) * a.s.kv_heads;
  kernel<<<dim3(uint32_t(items < 65536 ? items : 65536)), 64 * NW, smem, stream>>>(a);
  return hipGetLastError();
}

constexpr int kJoinThreads = 256, kJoinRows = 16;

// out = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) l_i over the pieces of a cut unit, in their order; 16 rows of a cache
// head a workgroup.
template <int DP, typename E>
__global__ __launch_bounds__(kJoinThreads) void attention_join_kernel(AttnArgs a, int kind, int most_rows) {
  constexpr int kCols = DP / 16;
  if (!plan_matches(a)) return;
  const int kv = a.s.kv_heads, D = a.s.head_dim, tiles = (most_rows + kJoinRows - 1) / kJoinRows;
  const int64_t n = int64_t(uniform(gload<int>(a.plan + A_CUT + kind))) * kv * tiles;
  const int row_in = threadIdx.x / 16, d0 = threadIdx.x % 16 * kCols;
  for (int64_t it = blockIdx.x; it < n; it += gridDim.x) {
    const int tile = int(it % tiles), head = int(it / tiles % kv), cut = int(it / tiles / kv);
    const int m = uniform(gload<int>(reinterpret_cast<const char *>(a.plan) + a.s.cutlist[kind] + size_t(cut) * 4));
    const AttnUnit u = load_unit(a, kind, m);
    const int r = tile * kJoinRows + row_in;
    if (r >= u.rows) continue;
    const float *part = reinterpret_cast<const float *>(a.ws + a.s.part[kind]);
    const float *stat = reinterpret_cast<const float *>(a.ws + a.s.stat[kind]);
    float M = kNoScore, l = 0.f, y[kCols];
#pragma unroll
    for (int c = 0; c < kCols; ++c) y[c] = 0.f;
    for (int i = 0; i < u.nsplit; ++i) {
      const int64_t at = (int64_t(u.slot + i) * kv + head) * most_rows + r;
      const float2 ml = gload<float2>(stat + at * 2);
      const float top = fmaxf(M, ml.x), old = __builtin_amdgcn_exp2f(M - top), now = __builtin_amdgcn_exp2f(ml.x - top);
      M = top;
      l = l * old + ml.y * now;
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        const float4 v = gload<float4>(part + at * DP + d0 + c);
        y[c] = y[c] * old + v.x * now, y[c + 1] = y[c + 1] * old + v.y * now;
        y[c + 2] = y[c + 2] * old + v.z * now, y[c + 3] = y[c + 3] * old + v.w * now;
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
hipError_t launch_join(const AttnArgs &a, int kind, hipStream_t stream) {
  const int rows = kind == ATTN_FEW ? a.s.few_rows : a.s.many_rows;
  const int64_t n = int64_t(a.s.cut[kind]) * a.s.kv_heads * ((rows + kJoinRows - 1) / kJoinRows);
  const dim3 grid(uint32_t(n < 16384 ? n : 16384));
  if (a.s.dp == 64) attention_join_kernel<64, E><<<grid, kJoinThreads, 0, stream>>>(a, kind, rows);
  else if (a.s.dp == 128) attention_join_kernel<128, E><<<grid, kJoinThreads, 0, stream>>>(a, kind, rows);
  else attention_join_kernel<256, E><<<grid, kJoinThreads, 0, stream>>>(a, kind, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attention_many(const AttnArgs &a, int dtype, hipStream_t stream) {
  if (dtype == LORA_BF16) {
    if (a.s.dp == 64) return launch_many<64, 8, false>(a, stream);
    if (a.s.dp == 128) return launch_many<128, 8, false>(a, stream);
    return launch_many<256, 4, false>(a, stream);
  }
  if (a.s.dp == 64) return launch_many<64, 4, true>(a, stream);
  if (a.s.dp == 128) return launch_many<128, 4, true>(a, stream);
  return launch_many<256, 4, true>(a, stream);
}

hipError_t launch_attention(const AttnArgs &a, int dtype, hipStream_t stream) {
  hipError_t e = hipSuccess;
  if (a.s.few_blocks) e = launch_attention_few(a, dtype, stream);
  if (e == hipSuccess && a.s.many_rows) e = launch_attention_many(a, dtype, stream);
  for (int kind = 0; kind < ATTN_KINDS; ++kind)
    if (e == hipSuccess && a.s.cut[kind]) e = dtype == LORA_BF16 ? launch_join<uint16_t>(a, kind, stream) : launch_join<float>(a, kind, stream);
  return e;
}

}  // namespace lora
