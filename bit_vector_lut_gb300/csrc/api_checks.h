// Argument checks that the entry points of the token mixers share.
#pragma once

#include "vq3_internal.h"

namespace vq3 {

inline bool on(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }
inline int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}
// A stride in elements of an axis of `extent`: whole 16-byte steps, rows of `row` elements apart.
// An axis of one element has no stride to speak of: `row` is used.
inline int check_stride(long long* s, long long extent, long long row, const char* who, const char* what) {
  if (extent <= 1) {
    *s = row;
    return VQ3_OK;
  }
  if (*s < row || *s >= (1LL << 38))
    return report_error(VQ3_EINVAL, "%s: %s stride %lld must be at least %lld (and below 2^38)", who, what, *s, row);
  if (*s % 8) return report_error(VQ3_EALIGN, "%s: %s stride %lld is not a multiple of 8 elements", who, what, *s);
  return VQ3_OK;
}
// Whether rows [tokens][heads][dim] with these strides overlap (checked by check_stride).
inline bool rows_overlap(int tokens, long long token, int heads, long long head, int dim) {
  return tokens > 1 && heads > 1 && token < (heads - 1) * head + dim && head < (tokens - 1) * token + dim;
}

}  // namespace vq3
