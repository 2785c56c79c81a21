// Host helpers of the C ABI's argument checks: alignment and overlap.
#pragma once

#include <cstdint>

namespace qg {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// bytes [begin, end) that an array touches
struct Span {
  uintptr_t begin, end;
};
inline bool overlap(const Span& a, const Span& b) {
  return a.begin < a.end && b.begin < b.end && a.begin < b.end && b.begin < a.end;
}
inline Span span(const void* p, int64_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p);
  return {x, x + (bytes > 0 ? (uintptr_t)bytes : 0)};
}

}  // namespace qg
