// Argument checks that the C ABI's files share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "salr.h"

namespace salr {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline int status(hipError_t e) { return e == hipSuccess ? SALR_OK : SALR_ERR_HIP; }

inline bool type_ok(int32_t t) { return t == SALR_TYPE_BF16 || t == SALR_TYPE_F32; }

// A buffer of a call, and whether two share no byte.
struct Span {
  const void* p;
  size_t bytes;
};
inline bool apart(const Span& x, const Span& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return !x.p || !y.p || !x.bytes || !y.bytes || a + x.bytes <= b || b + y.bytes <= a;
}
// What a call writes shares no byte with anything else of it.
template <size_t nw, size_t nr>
bool writes_apart(const Span (&written)[nw], const Span (&read)[nr]) {
  for (size_t i = 0; i < nw; ++i) {
    for (size_t j = i + 1; j < nw; ++j)
      if (!apart(written[i], written[j])) return false;
    for (const Span& r : read)
      if (!apart(written[i], r)) return false;
  }
  return true;
}

struct Range {
  uintptr_t a, b;
};

// Whether any two of the ranges written share a byte, or any range read
// shares one with a range written.  Sorts `written`.
inline bool overlaps(Range* written, size_t nw, const Range* read, size_t nr) {
  std::sort(written, written + nw, [](const Range& x, const Range& y) { return x.a < y.a; });
  for (size_t i = 1; i < nw; ++i)
    if (written[i].a < written[i - 1].b) return true;
  for (size_t i = 0; i < nr; ++i) {
    // the last written range that begins before this one ends
    const Range* w =
        std::lower_bound(written, written + nw, read[i].b, [](const Range& x, uintptr_t v) { return x.a < v; });
    if (w != written && (w - 1)->b > read[i].a) return true;
  }
  return false;
}

}  // namespace salr
