// Host-side argument checks shared by the C entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <functional>

#include "../../include/w4a16.h"

namespace w4a16 {
namespace checks {

constexpr int64_t kMaxM = int64_t(1) << 22;    // batch rows per call
// Packed codes of one matrix are addressed with 32-bit byte offsets.
constexpr int64_t kMaxPackedBytes = (int64_t(1) << 31) - (int64_t(1) << 20);

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

inline bool known_act(int act) { return act >= W4A16_ACT_NONE && act <= W4A16_ACT_GELU_TANH; }

struct Range {
  const void *p;
  size_t n;
};

inline bool overlap(const Range &a, const Range &b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const char *x = static_cast<const char *>(a.p), *y = static_cast<const char *>(b.p);
  return std::less<const char *>()(x, y + b.n) && std::less<const char *>()(y, x + a.n);
}

// An output that may also be exactly the input it replaces, element by element.
inline bool overlap_but_same(const Range &out, const Range &in) { return out.p != in.p && overlap(out, in); }

}  // namespace checks
}  // namespace w4a16
