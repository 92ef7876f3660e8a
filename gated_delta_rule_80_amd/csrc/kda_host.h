// Argument checks shared by the host runtime's entry points: address ranges of
// the caller's buffers, sizes without overflow, status of a launch.
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "kda.h"

namespace kda {

struct Span {
  uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when lo == hi
};

inline Span span(const void* p, size_t bytes) {
  Span s;
  if (p != nullptr && bytes > 0) {
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + bytes;
  }
  return s;
}
inline bool overlaps(Span a, Span b) { return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi; }
inline bool same_or_disjoint(Span a, Span b) { return (a.lo == b.lo && a.hi == b.hi) || !overlaps(a, b); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t esize(int io) { return io == KDA_FP32 ? 4 : 2; }

// a * b * c * d without overflow past 2^62; returns false on overflow.
inline bool mul_ok(size_t& out, std::initializer_list<size_t> xs) {
  size_t acc = 1;
  for (size_t x : xs) {
    if (x != 0 && acc > (size_t(1) << 62) / x) return false;
    acc *= x;
  }
  out = acc;
  return true;
}

inline kda_status hip_status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

}  // namespace kda
