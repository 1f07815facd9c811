// Host checks shared by the entry points of include/lora_base.h and lora_layer.h.
#pragma once

#include "lora_internal.hpp"

namespace lora {

inline bool aligned_to(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline lora_status check_dtype(lora_dtype d) { return d == LORA_F32 || d == LORA_BF16 ? LORA_OK : LORA_EINVAL; }

// Whether byte offsets over n rows at a stride of ld elements stay within 62 bits.
inline bool fits(int32_t n, int64_t ld) { return __int128(n) * ld < (__int128(1) << 59); }

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
inline bool disjoint(const Heads &a, const Heads &b) {
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

}  // namespace lora
