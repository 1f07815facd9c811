// C-ABI entry points of include/lora_layer.h: host checks, the sizes of plans
// and workspaces, launches.  No host synchronization and no allocation.

#include <cmath>
#include <cstring>

#include "lora_checks.hpp"
#include "lora_layer.hpp"

using namespace lora;

namespace {

struct Bytes {
  const void *p;
  size_t n;
};
bool meets(const Bytes &a, const Bytes &b) { return a.p && b.p && overlap(a.p, a.n, b.p, b.n); }

// One array of a cache: n pages of `bytes`, `stride` apart.
struct Pages {
  const char *p;
  int64_t stride, bytes, n;
  size_t span() const { return size_t((n - 1) * stride + bytes); }
  Bytes all() const { return {p, span()}; }
};
// Pages of two arrays share no byte: their spans are apart, or they lie side by side at one stride.
bool pages_apart(const Pages &a, const Pages &b) {
  if (!overlap(a.p, a.span(), b.p, b.span())) return true;
  if (a.stride != b.stride || a.stride <= 0) return false;
  int64_t off = int64_t(b.p - a.p) % a.stride;
  if (off < 0) off += a.stride;
  return off >= a.bytes && off + b.bytes <= a.stride;
}

int log2_of(int v) {
  int b = 0;
  while ((1 << b) < v) ++b;
  return b;
}

// The sizes of a cache, without its memory.
lora_status check_cache_sizes(const lora_cache *c) {
  if (!c) return LORA_EINVAL;
  if (c->n_pages < 1 || c->n_heads < 1 || c->head_dim < 1) return LORA_ESHAPE;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return LORA_ESHAPE;
  if (c->head_dim > LORA_MAX_CACHE_HEAD_DIM || c->n_heads > LORA_MAX_CACHE_HEADS) return LORA_EUNSUPPORTED;
  return LORA_OK;
}

lora_status check_cache(const lora_cache *c, Pages (&pages)[4]) {
  if (lora_status st = check_cache_sizes(c)) return st;
  const int64_t slots = int64_t(c->n_heads) * c->page_size, bytes = slots * cache_pitch(c->head_dim);
  const struct { const void *p; int64_t stride, bytes; } arrays[4] = {
      {c->k, c->k_page, bytes}, {c->v, c->v_page, bytes},
      {c->k_scale, c->k_scale_page, slots}, {c->v_scale, c->v_scale_page, slots}};
  for (int i = 0; i < 4; ++i) {
    const int eb = i < 2 ? 1 : 4;
    if (!arrays[i].p || !aligned16(arrays[i].p)) return LORA_EINVAL;
    if (c->n_pages > 1 && arrays[i].stride < arrays[i].bytes) return LORA_ESHAPE;
    if (arrays[i].stride < 0 || !fits(c->n_pages, arrays[i].stride)) return LORA_ESHAPE;
    if (c->n_pages > 1 && arrays[i].stride * eb % 16) return LORA_EINVAL;
    pages[i] = {static_cast<const char *>(arrays[i].p), arrays[i].stride * eb, arrays[i].bytes * eb, c->n_pages};
  }
  return LORA_OK;
}

// Heads of n tokens, as bytes; `apart`: each value has to have a place of its own.
lora_status check_heads(const lora_heads *h, int64_t T, int64_t n_heads, int64_t d, int64_t eb, bool apart, Heads &to) {
  if (!h) return LORA_EINVAL;
  for (int64_t s : {h->token, h->head})
    if (s < 0 || !fits(int32_t(T), s) || !fits(int32_t(n_heads), s)) return LORA_ESHAPE;
  if (!h->data || !aligned_to(h->data, eb)) return LORA_EINVAL;
  to = {static_cast<const char *>(h->data), h->token * eb, h->head * eb, T, n_heads, d * eb};
  return apart && !to.apart() ? LORA_ESHAPE : LORA_OK;
}

lora_status cache_call(const lora_cache *cache, const int32_t *slots, int32_t n_tokens, const lora_heads *k,
                       const lora_heads *v, lora_dtype dtype, bool write, hipStream_t stream) {
  if (lora_status st = check_dtype(dtype)) return st;
  Pages pages[4];
  if (lora_status st = check_cache(cache, pages)) return st;
  if (n_tokens < 0) return LORA_ESHAPE;
  if (n_tokens == 0) return LORA_OK;
  if (!slots || !aligned_to(slots, 4)) return LORA_EINVAL;
  const int eb = elem_bytes(dtype);
  Heads hk, hv;
  if (lora_status st = check_heads(k, n_tokens, cache->n_heads, cache->head_dim, eb, !write, hk)) return st;
  if (lora_status st = check_heads(v, n_tokens, cache->n_heads, cache->head_dim, eb, !write, hv)) return st;
  const Bytes named{slots, size_t(n_tokens) * 4};
  for (int i = 0; i < 4; ++i) {
    for (const Heads *h : {&hk, &hv})
      if (meets(pages[i].all(), {h->p, h->span()})) return LORA_EINVAL;
    if (write && meets(pages[i].all(), named)) return LORA_EINVAL;
    for (int j = 0; j < i; ++j)
      if (write && !pages_apart(pages[i], pages[j])) return LORA_EINVAL;
  }
  if (!write && (!disjoint(hk, hv) || meets(named, {hk.p, hk.span()}) || meets(named, {hv.p, hv.span()})))
    return LORA_EINVAL;
  const CacheArgs a{*cache, cache_pitch(cache->head_dim), log2_of(cache->page_size), slots, *k, *v, n_tokens};
  return (write ? launch_cache_write(a, dtype, stream) : launch_cache_read(a, dtype, stream)) == hipSuccess ? LORA_OK
                                                                                                           : LORA_EHIP;
}

lora_status check_attention(const lora_attention *t, const lora_cache *c, const lora_attention_batch *b) {
  if (!t || !b) return LORA_EINVAL;
  if (lora_status st = check_dtype(t->dtype)) return st;
  if (lora_status st = check_cache_sizes(c)) return st;
  if (t->n_heads < 1 || t->n_heads % c->n_heads || t->window < 0 || t->sinks < 0) return LORA_ESHAPE;
  if (t->n_heads > LORA_MAX_CACHE_HEADS) return LORA_EUNSUPPORTED;
  if (!(t->scale > 0) || !std::isfinite(t->scale)) return LORA_ESHAPE;
  if (b->n_tokens < 0 || b->n_seqs < 0 || b->max_q < 1 || b->max_pages < 1 || b->ld_pages < b->max_pages ||
      !fits(b->n_seqs, b->ld_pages))
    return LORA_ESHAPE;
  if (int64_t(b->max_pages) * c->page_size > LORA_MAX_CONTEXT) return LORA_EUNSUPPORTED;
  if (b->tree && b->max_q > LORA_MAX_TREE) return LORA_EUNSUPPORTED;
  if (int64_t(b->n_tokens) * t->n_heads > (1 << 30) || b->n_seqs > (1 << 24)) return LORA_EUNSUPPORTED;
  return LORA_OK;
}

// Which kernels a batch of this shape can need, and how its plan and workspace lie.
AttnShape attention_shape(const lora_attention &t, const lora_cache &c, const lora_attention_batch &b) {
  AttnShape s{};
  s.T = b.n_tokens, s.S = b.n_seqs, s.kv_heads = c.n_heads, s.group = t.n_heads / c.n_heads, s.head_dim = c.head_dim;
  s.dp = c.head_dim <= 64 ? 64 : c.head_dim <= 128 ? 128 : 256;
  const bool f32 = t.dtype == LORA_F32;
  // The kernel for few rows has registers for two row blocks of 16 (one of fp32 heads beyond 128); with four it spilled
  // and took near three times the other kernel's time.  Where both serve, 32 rows of 8 cache heads over 8192 keys each, bf16
  // heads of 128: one sequence 26 us here and 38 there, four 68 and 60, 32 of them 230 and 220 (heads of 64: 22 and 27, 55
  // and 44, 171 and 145).  32 sequences with heads of 256: 698 and 1039; fp32 heads of 64: 181 and 326, of 128: 255 and
  // 455.
  const bool one = f32 ? s.dp == 256 : s.dp <= 128 && int64_t(s.S) * s.kv_heads > 32;
  const int blocks = one ? 1 : 2;
  const int64_t q = b.max_q < s.T ? b.max_q : s.T, most = q * s.group;
  // All sequences are short, or those of one token are; there are none of these where all sequences are as long as can be
  // (else the launch costs the 4.5 us of a kernel that finds nothing to do).
  const int64_t few = most <= 16 * blocks ? most : s.group <= 16 * blocks && s.T < s.S * q ? s.group : 0;
  s.few_blocks = few == 0 ? 0 : few <= 16 ? 1 : 2;
  s.few_rows = 16 * s.few_blocks;
  // Units of 128 rows, two workgroups a CU, where no sequence has more: 32 drafts of 24 tokens for 32 heads after up to
  // 16384 keys take 315 us, 447 in units of 256; a prompt of 16384 takes 1261 us in units of 256 and 1391 in those of 128.
  s.many_rows = most <= s.few_rows ? 0 : s.dp == 256 || f32 || most <= 128 ? 128 : 256;
  const int64_t wide = int64_t(s.T) * s.group;
  s.units[ATTN_FEW] = s.few_rows ? s.S : 0;
  s.units[ATTN_MANY] = s.many_rows ? int(s.S + wide / s.many_rows) : 0;
  // the key tiles that a unit can have at most
  int64_t tiles = (int64_t(b.max_pages) * c.page_size - 1) / kKeyTile + 1;
  if (t.window) {
    const int64_t seen = (int64_t(t.window) + b.max_q) / kKeyTile + 2 + (int64_t(t.sinks) + kKeyTile - 1) / kKeyTile;
    tiles = tiles < seen ? tiles : seen;
  }
  // Pieces of all heads that a launch aims at.  Few rows: four times as many as find room at once, which come out even
  // however long the sequences are (64 of up to 32768 keys 522 us, 541 with half as many, 543 with four times as many; the
  // builds of one workgroup a CU: fp32 heads of 128 652, 680 and 811, bf16 heads of 256 1017, 1013 and 1188).
  // Many rows: of 256 one a CU (beside 256 single tokens four prompts of 512 after up to 4096 keys 730 us, with two as
  // well), of 128 three (32 drafts of 24 after up to 16384 keys 315 us; 368 with two, 329 with four, 382 with one).
  const int total[ATTN_KINDS] = {2048, s.many_rows == 256 ? 256 : 768};
  size_t at = align256(sizeof(int) * H_WORDS), ws = 0;
  auto take = [](size_t &off, size_t bytes) { const size_t o = off; off = align256(off + bytes); return o; };
  s.toff = take(at, sizeof(int) * (size_t(s.S) + 1));
  for (int k = 0; k < ATTN_KINDS; ++k) {
    const int rows = k == ATTN_FEW ? s.few_rows : s.many_rows;
    s.target[k] = (total[k] - 1) / s.kv_heads + 1;
    // (four tiles are one a wave of few rows: a request of 4097 keys takes 15.0 us, 18.0 with two, 16.9 with eight; seven
    // fp32 drafts of many rows 25.1 us with two, 28.9 with four, 38.4 with one, a second round)
    s.least[k] = k == ATTN_FEW ? 4 : 2;
    // a unit is cut into no more than twice its share of the target, and not at all where it has few tiles
    s.cut[k] = s.units[k] && tiles > s.least[k] ? (s.units[k] < s.target[k] ? s.units[k] : s.target[k]) : 0;
    s.items[k] = s.units[k] + (s.cut[k] ? s.target[k] : 0);
    s.unit[k] = take(at, sizeof(AttnUnit) * size_t(s.units[k]));
    s.item[k] = take(at, 8 * size_t(s.items[k]));
    s.cutlist[k] = take(at, 4 * size_t(s.cut[k]));
    const size_t pieces = s.cut[k] ? size_t(2) * s.target[k] * s.kv_heads * rows : 0;
    s.part[k] = take(ws, pieces * s.dp * 4);
    s.stat[k] = take(ws, pieces * 2 * 4);
  }
  s.plan_bytes = at;
  s.ws_bytes = ws;
  return s;
}

void plan_key(const lora_attention &t, const lora_cache &c, const lora_attention_batch &b, int *key) {
  const int k[A_KEYS] = {kAttnMagic, b.n_tokens, b.n_seqs, t.n_heads, c.n_heads, c.head_dim, int(t.dtype),
                         t.window, t.sinks, b.max_q, b.max_pages * c.page_size, b.tree ? 1 : 0};
  std::memcpy(key, k, sizeof(k));
}

}  // namespace

extern "C" {

lora_status lora_norm_apply(const lora_norm *norm, const void *x, int64_t ldx, const void *residual, int64_t ldr,
                            void *total, int64_t ldt, void *y, int64_t ldy, int8_t *q, int64_t ldq, float *scale,
                            int32_t n_rows, lora_dtype dtype, hipStream_t stream) {
  if (lora_status st = check_dtype(dtype)) return st;
  if (!norm) return LORA_EINVAL;
  const int d = norm->d, eb = elem_bytes(dtype);
  if (d < 1) return LORA_ESHAPE;
  if (d > LORA_MAX_NORM_D) return LORA_EUNSUPPORTED;
  if (!norm->weight || !aligned_to(norm->weight, 4)) return LORA_EINVAL;
  if (!(norm->eps >= 0) || !std::isfinite(norm->eps)) return LORA_EINVAL;
  if (n_rows < 0) return LORA_ESHAPE;
  if (n_rows == 0) return LORA_OK;
  if (!x || (!y && !q) || (!q != !scale) || (total && !residual)) return LORA_EINVAL;
  struct Rows {
    const void *p;
    int64_t ld;
    int eb;
    bool written;
  };
  const Rows rows[5] = {{x, ldx, eb, false}, {residual, ldr, eb, false}, {total, ldt, eb, true}, {y, ldy, eb, true}, {q, ldq, 1, true}};
  Bytes at[7];
  for (int i = 0; i < 5; ++i) {
    at[i] = {rows[i].p, 0};
    if (!rows[i].p) continue;
    if (rows[i].ld < d || !fits(n_rows, rows[i].ld)) return LORA_ESHAPE;
    if (!aligned_to(rows[i].p, rows[i].eb)) return LORA_EINVAL;
    at[i].n = span_bytes(n_rows, rows[i].ld, d, rows[i].eb);
  }
  if (!aligned_to(scale, 4)) return LORA_EINVAL;
  at[5] = {scale, size_t(n_rows) * 4};
  at[6] = {norm->weight, size_t(d) * 4};
  for (int i = 2; i < 6; ++i)
    for (int j = 0; j < 7; ++j) {
      if (i == j || !meets(at[i], at[j])) continue;
      // in place: the total over x or the residual, y over x
      const bool same = j < 2 && rows[i < 5 ? i : 4].p == rows[j].p && (n_rows == 1 || rows[i < 5 ? i : 4].ld == rows[j].ld);
      if (!(same && (i == 2 || (i == 3 && j == 0)))) return LORA_EINVAL;
    }
  const NormArgs a{x, residual, norm->weight, total, y, q, scale, ldx, ldr, ldt, ldy, ldq, norm->eps, n_rows, d};
  return launch_norm(a, dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

int32_t lora_cache_pitch(int32_t head_dim) {
  return head_dim >= 1 && head_dim <= LORA_MAX_CACHE_HEAD_DIM ? cache_pitch(head_dim) : 0;
}

lora_status lora_cache_write(const lora_cache *cache, const int32_t *slots, int32_t n_tokens, const lora_heads *k,
                             const lora_heads *v, lora_dtype dtype, hipStream_t stream) {
  return cache_call(cache, slots, n_tokens, k, v, dtype, true, stream);
}

lora_status lora_cache_read(const lora_cache *cache, const int32_t *slots, int32_t n_tokens, const lora_heads *k,
                            const lora_heads *v, lora_dtype dtype, hipStream_t stream) {
  return cache_call(cache, slots, n_tokens, k, v, dtype, false, stream);
}

size_t lora_attention_plan_size(const lora_attention *attention, const lora_cache *cache,
                                const lora_attention_batch *batch) {
  if (check_attention(attention, cache, batch) != LORA_OK) return 0;
  return attention_shape(*attention, *cache, *batch).plan_bytes;
}

size_t lora_attention_workspace_size(const lora_attention *attention, const lora_cache *cache,
                                     const lora_attention_batch *batch) {
  if (check_attention(attention, cache, batch) != LORA_OK) return 0;
  return align256(attention_shape(*attention, *cache, *batch).ws_bytes + 1);
}

lora_status lora_attention_plan(const lora_attention *attention, const lora_cache *cache,
                                const lora_attention_batch *batch, void *plan, size_t plan_bytes, hipStream_t stream) {
  if (lora_status st = check_attention(attention, cache, batch)) return st;
  AttnPlanArgs a;
  std::memset(&a, 0, sizeof(a));
  a.s = attention_shape(*attention, *cache, *batch);
  if (!plan || plan_bytes < a.s.plan_bytes) return LORA_EWORKSPACE;
  if (!aligned16(plan)) return LORA_EINVAL;
  if (batch->n_seqs > 0) {
    if (!batch->q_off || !batch->lens || !aligned_to(batch->q_off, 4) || !aligned_to(batch->lens, 4)) return LORA_EINVAL;
    const size_t n = size_t(batch->n_seqs) * 4;
    if (overlap(plan, plan_bytes, batch->q_off, n + 4) || overlap(plan, plan_bytes, batch->lens, n)) return LORA_EINVAL;
  }
  a.q_off = batch->q_off;
  a.lens = batch->lens;
  a.plan = static_cast<int *>(plan);
  a.max_q = batch->max_q;
  a.capacity = batch->max_pages * cache->page_size;
  // (no key is further away than that)
  a.window = attention->window < LORA_MAX_CONTEXT ? attention->window : LORA_MAX_CONTEXT;
  a.sinks = attention->sinks;
  a.tree = batch->tree != nullptr;
  plan_key(*attention, *cache, *batch, a.key);
  return launch_attention_plan(a, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

lora_status lora_attention_apply(const lora_attention *attention, const lora_cache *cache,
                                 const lora_attention_batch *batch, const void *plan, size_t plan_bytes,
                                 const lora_heads *q, const lora_heads *out, void *ws, size_t ws_bytes,
                                 hipStream_t stream) {
  if (lora_status st = check_attention(attention, cache, batch)) return st;
  Pages pages[4];
  if (lora_status st = check_cache(cache, pages)) return st;
  const int64_t T = batch->n_tokens;
  if (T == 0 || batch->n_seqs == 0) return LORA_OK;
  AttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.s = attention_shape(*attention, *cache, *batch);
  if (!plan || plan_bytes < a.s.plan_bytes) return LORA_EWORKSPACE;
  if (!ws || ws_bytes < a.s.ws_bytes) return LORA_EWORKSPACE;
  if (!aligned16(plan) || !aligned16(ws)) return LORA_EINVAL;
  if (!batch->pages || !aligned_to(batch->pages, 4) || !aligned_to(batch->tree, 8)) return LORA_EINVAL;
  const int eb = elem_bytes(attention->dtype), D = cache->head_dim;
  Heads hq, ho;
  if (lora_status st = check_heads(q, T, attention->n_heads, D, eb, false, hq)) return st;
  if (lora_status st = check_heads(out, T, attention->n_heads, D, eb, true, ho)) return st;
  if (q->data == out->data) {
    if ((T > 1 && q->token != out->token) || (attention->n_heads > 1 && q->head != out->head)) return LORA_ESHAPE;
  } else if (!disjoint(hq, ho)) {
    return LORA_EINVAL;
  }
  const Bytes written[2] = {{ho.p, ho.span()}, {ws, ws_bytes}};
  const Bytes read[4] = {{batch->pages, (size_t(batch->n_seqs - 1) * batch->ld_pages + batch->max_pages) * 4},
                         {batch->tree, size_t(T) * 8},
                         {plan, plan_bytes},
                         {hq.p, hq.span()}};
  for (int w = 0; w < 2; ++w) {
    for (int i = 0; i < 4; ++i)
      if (meets(written[w], pages[i].all()) || ((i < 3 || w == 1) && meets(written[w], read[i]))) return LORA_EINVAL;
  }
  if (meets(written[0], written[1])) return LORA_EINVAL;
  a.c = *cache;
  a.pitch = cache_pitch(D);
  a.page_bits = log2_of(cache->page_size);
  a.q = *q;
  a.out = *out;
  a.pages = batch->pages;
  a.ld_pages = batch->ld_pages;
  a.tree = batch->tree;
  a.plan = static_cast<int *>(const_cast<void *>(plan));
  a.ws = static_cast<char *>(ws);
  a.window = attention->window ? attention->window : 0x7fffffff;
  a.sinks = attention->sinks;
  a.scale = attention->scale * 1.44269504088896340736f;
  plan_key(*attention, *cache, *batch, a.key);
  return launch_attention(a, attention->dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

}  // extern "C"
