// C-ABI entry points of include/lora_base.h: host checks, workspace layout and
// launches.  No host synchronization and no allocation.

#include <cmath>
#include <cstring>

#include "lora_base.hpp"

using namespace lora;

namespace {

bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

lora_status check_dtype(lora_dtype d) { return d == LORA_F32 || d == LORA_BF16 ? LORA_OK : LORA_EINVAL; }

// Whether byte offsets over n rows at a stride of ld elements stay within 62 bits.
bool fits(int32_t n, int64_t ld) { return __int128(n) * ld < (__int128(1) << 59); }

lora_status check_weight(const lora_base_weight *w) {
  if (!w) return LORA_EINVAL;
  if (w->d_in < 1 || w->d_out < 1) return LORA_ESHAPE;
  if (w->d_in > LORA_MAX_BASE_D_IN) return LORA_EUNSUPPORTED;
  if (w->ldw < w->d_in || !fits(w->d_out, w->ldw)) return LORA_ESHAPE;
  if (!w->W || !w->scale) return LORA_EINVAL;
  if (!aligned_to(w->scale, 4) || !aligned_to(w->bias, 4)) return LORA_EINVAL;
  return LORA_OK;
}

// Whether [p, p + n) meets anything that a product reads of its weight.
bool meets_weight(const lora_base_weight *w, const void *p, size_t n) {
  const size_t f = size_t(w->d_out) * 4;
  return overlap(p, n, w->W, span_bytes(w->d_out, w->ldw, w->d_in, 1)) || overlap(p, n, w->scale, f) ||
         (w->bias && overlap(p, n, w->bias, f));
}

lora_status check_y(const lora_base_weight *w, int32_t n_tokens, const void *y, int64_t ldy, lora_dtype dtype) {
  if (n_tokens < 0 || ldy < w->d_out || !fits(n_tokens, ldy)) return LORA_ESHAPE;
  if (n_tokens == 0) return LORA_OK;
  if (!y || !aligned_to(y, elem_bytes(dtype))) return LORA_EINVAL;
  if (meets_weight(w, y, span_bytes(n_tokens, ldy, w->d_out, elem_bytes(dtype)))) return LORA_EINVAL;
  return LORA_OK;
}

// The quantised rows of lora_base_apply in its workspace: rows of d_in bytes
// at a pitch of whole 16s, as the product's kernels for aligned rows need it
// where d_in and the weight's rows are whole 16s too, then a scale for each row.
struct BaseLayout {
  int64_t pitch;
  size_t scale, total;
};
BaseLayout base_layout(int d_in, int n_tokens) {
  BaseLayout L;
  L.pitch = (int64_t(d_in) + 15) / 16 * 16;
  L.scale = align256(size_t(L.pitch) * n_tokens);
  L.total = L.scale + align256(size_t(4) * n_tokens);
  return L;
}

// The bytes of one tensor of heads: [T][n_heads][head_dim] with two strides.
struct Heads {
  const char *p;
  int64_t token, head;  // strides in bytes
  int64_t T, n, d;      // tokens, heads, bytes of a head

  size_t span() const { return size_t((T - 1) * token + (n - 1) * head + d); }
  // bytes from the first to the last value of a token, and of a head
  int64_t token_span() const { return (n - 1) * head + d; }
  int64_t head_span() const { return (T - 1) * token + d; }
  // every value has a place of its own
  bool apart() const {
    const bool tokens_outer = (n == 1 || head >= d) && (T == 1 || token >= token_span());
    const bool heads_outer = (T == 1 || token >= d) && (n == 1 || head >= head_span());
    return tokens_outer || heads_outer;
  }
};

// Two tensors share no byte: their spans are apart, or they are column ranges
// of one buffer (same outer stride, and the inner extents lie side by side).
bool disjoint(const Heads &a, const Heads &b) {
  if (!overlap(a.p, a.span(), b.p, b.span())) return true;
  auto beside = [&](int64_t stride_a, int64_t stride_b, int64_t ext_a, int64_t ext_b) {
    if (stride_a != stride_b || stride_a <= 0 || ext_a > stride_a || ext_b > stride_a) return false;
    int64_t off = int64_t(b.p - a.p) % stride_a;
    if (off < 0) off += stride_a;
    return off >= ext_a && off + ext_b <= stride_a;
  };
  return beside(a.token, b.token, a.token_span(), b.token_span()) ||
         beside(a.head, b.head, a.head_span(), b.head_span());
}

}  // namespace

extern "C" {

lora_status lora_quantize_rows(const void *x, int64_t ldx, lora_dtype dtype, int32_t n_rows, int32_t d, int8_t *q,
                               int64_t ldq, float *scale, hipStream_t stream) {
  if (lora_status st = check_dtype(dtype)) return st;
  if (n_rows < 0 || d < 1 || ldx < d || ldq < d || !fits(n_rows, ldx) || !fits(n_rows, ldq)) return LORA_ESHAPE;
  if (n_rows == 0) return LORA_OK;
  const int eb = elem_bytes(dtype);
  if (!x || !q || !scale || !aligned_to(x, eb) || !aligned_to(scale, 4)) return LORA_EINVAL;
  const size_t xs = span_bytes(n_rows, ldx, d, eb), qs = span_bytes(n_rows, ldq, d, 1), ss = size_t(n_rows) * 4;
  if (overlap(x, xs, q, qs) || overlap(x, xs, scale, ss) || overlap(q, qs, scale, ss)) return LORA_EINVAL;
  const QuantArgs a{x, q, scale, ldx, ldq, n_rows, d};
  return launch_quantize(a, dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

lora_status lora_base_product(const lora_base_weight *weight, const int8_t *q, int64_t ldq, const float *q_scale,
                              int32_t n_tokens, void *y, int64_t ldy, lora_dtype dtype, hipStream_t stream) {
  if (lora_status st = check_dtype(dtype)) return st;
  if (lora_status st = check_weight(weight)) return st;
  if (lora_status st = check_y(weight, n_tokens, y, ldy, dtype)) return st;
  if (ldq < weight->d_in || !fits(n_tokens, ldq)) return LORA_ESHAPE;
  if (n_tokens == 0) return LORA_OK;
  if (!q || !q_scale || !aligned_to(q_scale, 4)) return LORA_EINVAL;
  const size_t ys = span_bytes(n_tokens, ldy, weight->d_out, elem_bytes(dtype));
  if (overlap(y, ys, q, span_bytes(n_tokens, ldq, weight->d_in, 1)) || overlap(y, ys, q_scale, size_t(n_tokens) * 4))
    return LORA_EINVAL;
  const ProductArgs a{q,   weight->W,   q_scale, weight->scale, weight->bias, y,
                      ldq, weight->ldw, ldy,     n_tokens,      weight->d_in, weight->d_out, 0};
  return launch_product(a, dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

// For the tests, in no header: the kernel that one launch of these sizes takes (16-byte aligned q and W), and in
// *first the rows that go in a launch of their own before the others.
int32_t lora_base_product_choice(int32_t n_tokens, int32_t d_in, int32_t d_out, int64_t ldq, int64_t ldw, int32_t *first) {
  ProductArgs a{};
  a.T = n_tokens;
  a.d_in = d_in;
  a.d_out = d_out;
  a.ldq = ldq;
  a.ldw = ldw;
  const ProductChoice c = choose_product(a);
  *first = c.first;
  return c.kernel;
}

size_t lora_base_workspace_size(const lora_base_weight *weight, int32_t n_tokens) {
  if (check_weight(weight) != LORA_OK || n_tokens < 1) return 0;
  return base_layout(weight->d_in, n_tokens).total;
}

lora_status lora_base_apply(const lora_base_weight *weight, const void *x, int64_t ldx, int32_t n_tokens, void *y,
                            int64_t ldy, lora_dtype dtype, void *ws, size_t ws_bytes, hipStream_t stream) {
  if (lora_status st = check_dtype(dtype)) return st;
  if (lora_status st = check_weight(weight)) return st;
  if (lora_status st = check_y(weight, n_tokens, y, ldy, dtype)) return st;
  if (ldx < weight->d_in || !fits(n_tokens, ldx)) return LORA_ESHAPE;
  if (n_tokens == 0) return LORA_OK;
  const int eb = elem_bytes(dtype);
  if (!x || !aligned_to(x, eb)) return LORA_EINVAL;
  const BaseLayout L = base_layout(weight->d_in, n_tokens);
  if (!ws || ws_bytes < L.total) return LORA_EWORKSPACE;
  if (!aligned16(ws)) return LORA_EINVAL;
  const size_t xs = span_bytes(n_tokens, ldx, weight->d_in, eb), ys = span_bytes(n_tokens, ldy, weight->d_out, eb);
  if (overlap(x, xs, y, ys) || overlap(ws, L.total, x, xs) || overlap(ws, L.total, y, ys) ||
      meets_weight(weight, ws, L.total))
    return LORA_EINVAL;
  int8_t *q = static_cast<int8_t *>(ws);
  float *scale = reinterpret_cast<float *>(static_cast<char *>(ws) + L.scale);
  const QuantArgs qa{x, q, scale, ldx, L.pitch, n_tokens, weight->d_in};
  if (launch_quantize(qa, dtype, stream) != hipSuccess) return LORA_EHIP;
  const ProductArgs a{q,       weight->W,   scale, weight->scale, weight->bias, y,
                      L.pitch, weight->ldw, ldy,   n_tokens,      weight->d_in, weight->d_out, 0};
  return launch_product(a, dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

lora_status lora_rotary_apply(const lora_rotary *rotary, const int32_t *positions, int32_t n_tokens, int32_t n_slices,
                              const lora_rotary_slice *slices, lora_dtype dtype, int32_t inverse, hipStream_t stream) {
  if (lora_status st = check_dtype(dtype)) return st;
  if (!rotary || !slices || !rotary->freq || !aligned_to(rotary->freq, 8)) return LORA_EINVAL;
  if ((rotary->interleaved & ~1) || (inverse & ~1)) return LORA_EINVAL;
  const int D = rotary->head_dim, rot = rotary->rot_dim;
  if (D < 1 || rot < 2 || rot > D || rot % 2) return LORA_ESHAPE;
  if (D > LORA_MAX_HEAD_DIM) return LORA_EUNSUPPORTED;
  if (n_tokens < 0 || n_slices < 1 || n_slices > LORA_MAX_SLICES) return LORA_ESHAPE;
  const int64_t eb = elem_bytes(dtype), T = n_tokens;
  Heads src[LORA_MAX_SLICES], dst[LORA_MAX_SLICES];
  RotaryArgs a;
  std::memset(&a, 0, sizeof(a));
  for (int i = 0; i < n_slices; ++i) {
    const lora_rotary_slice &s = slices[i];
    if (s.n_heads < 1 || s.n_heads > LORA_MAX_HEADS) return LORA_ESHAPE;
    for (int64_t v : {s.src_token, s.src_head, s.dst_token, s.dst_head})
      if (v < 0 || !fits(n_tokens, v) || !fits(s.n_heads, v)) return LORA_ESHAPE;
    a.s[i] = s;
    a.n_heads += s.n_heads;
    if (T == 0) continue;
    if (!s.src || !s.dst || !aligned_to(s.src, eb) || !aligned_to(s.dst, eb)) return LORA_EINVAL;
    src[i] = {static_cast<const char *>(s.src), s.src_token * eb, s.src_head * eb, T, s.n_heads, D * eb};
    dst[i] = {static_cast<const char *>(s.dst), s.dst_token * eb, s.dst_head * eb, T, s.n_heads, D * eb};
    if (!dst[i].apart()) return LORA_ESHAPE;
    if (s.src == s.dst) {
      if ((T > 1 && s.src_token != s.dst_token) || (s.n_heads > 1 && s.src_head != s.dst_head)) return LORA_ESHAPE;
    } else if (!disjoint(src[i], dst[i])) {
      return LORA_EINVAL;
    }
  }
  if (T == 0) return LORA_OK;
  if (!positions || !aligned_to(positions, 4)) return LORA_EINVAL;
  for (int i = 0; i < n_slices; ++i) {
    const Heads &o = dst[i];
    if (overlap(o.p, o.span(), positions, size_t(T) * 4) || overlap(o.p, o.span(), rotary->freq, size_t(rot) * 4))
      return LORA_EINVAL;
    for (int j = 0; j < n_slices; ++j)
      if (j != i && (!disjoint(o, src[j]) || (j > i && !disjoint(o, dst[j])))) return LORA_EINVAL;
  }
  a.freq = rotary->freq;
  a.positions = positions;
  a.T = n_tokens;
  a.head_dim = D;
  a.rot_dim = rot;
  a.interleaved = rotary->interleaved;
  a.mscale = rotary->mscale;
  a.sign = inverse ? -1.f : 1.f;
  a.n_slices = n_slices;
  return launch_rotary(a, dtype, stream) == hipSuccess ? LORA_OK : LORA_EHIP;
}

lora_status lora_rotary_frequencies(lora_rotary_scaling scaling, double base, int32_t rot_dim, double factor,
                                    double length, double low, double high, double *freq) {
  if (!freq || scaling < LORA_ROTARY_PLAIN || scaling > LORA_ROTARY_PARTS) return LORA_EINVAL;
  if (rot_dim < 2 || rot_dim % 2) return LORA_ESHAPE;
  if (!(base > 0) || !std::isfinite(base)) return LORA_ESHAPE;
  if (scaling != LORA_ROTARY_PLAIN && (!(factor > 0) || !std::isfinite(factor))) return LORA_ESHAPE;
  if (scaling == LORA_ROTARY_BASE) {
    if (rot_dim < 4) return LORA_ESHAPE;
    base *= std::pow(factor, double(rot_dim) / (rot_dim - 2));
    if (!(base > 0) || !std::isfinite(base)) return LORA_ESHAPE;
  }
  if (scaling == LORA_ROTARY_PARTS &&
      (!(length > 0) || !std::isfinite(length) || !(low >= 0) || !(high > low) || !std::isfinite(high)))
    return LORA_ESHAPE;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int j = 0; j < rot_dim / 2; ++j) {
    double f = std::pow(base, -2.0 * j / rot_dim);
    if (scaling == LORA_ROTARY_LINEAR) f /= factor;
    if (scaling == LORA_ROTARY_PARTS) {
      const double turns = length * f / kTwoPi;
      const double keep = turns >= high ? 1.0 : turns <= low ? 0.0 : (turns - low) / (high - low);
      f = keep * f + (1.0 - keep) * (f / factor);
    }
    freq[j] = f;
  }
  return LORA_OK;
}

}  // extern "C"
