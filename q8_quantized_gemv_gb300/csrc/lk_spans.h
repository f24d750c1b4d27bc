// Host helpers of the calls that check what they are given against each other,
// and the launch of a kernel with dynamic shared memory.
#pragma once

#include <stddef.h>

#include "lk_host.h"

namespace lkh {

// n bytes at p, where there are any
struct Span {
  const void* p;
  size_t n;
};
inline bool overlap(const Span& x, const Span& y) {
  const uintptr_t a = (uintptr_t)x.p, b = (uintptr_t)y.p;
  return x.p && y.p && x.n && y.n && a < b + y.n && b < a + x.n;
}
// Whether one of the `nw` written spans, which come first, overlaps another of the n.
inline bool spans_clash(const Span* s, int nw, int n) {
  for (int i = 0; i < nw; ++i)
    for (int k = i + 1; k < n; ++k)
      if (overlap(s[i], s[k])) return true;
  return false;
}

}  // namespace lkh
