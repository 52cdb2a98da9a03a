// Host helpers of the C-ABI entry points: alignment, element sizes, overlap.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/muon.h"

namespace muon {

constexpr size_t kAlign = 256;   // of the blocks inside a workspace

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t dtype_size(int dt) { return dt == MUON_BF16 ? 2 : 4; }
inline bool overlaps(const char* a, size_t na, const char* b, size_t nb) { return a < b + nb && b < a + na; }

// Bytes an operand spans.
struct Span {
  const char* p;
  size_t n;
};
inline Span span(const void* p, size_t bytes) { return {static_cast<const char*>(p), bytes}; }
// No output may overlap an input or another output (null operands overlap nothing).
inline bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span* a = outs.begin(); a != outs.end(); ++a) {
    if (a->p == nullptr) continue;
    for (const Span& b : ins)
      if (b.p != nullptr && overlaps(a->p, a->n, b.p, b.n)) return true;
    for (const Span* b = a + 1; b != outs.end(); ++b)
      if (b->p != nullptr && overlaps(a->p, a->n, b->p, b->n)) return true;
  }
  return false;
}

// Whether a strided operand's bytes can be counted: no memory holds 2^60.
inline bool extent_ok(std::initializer_list<long long> steps, std::initializer_list<long long> strides) {
  long long sum = 0, p;
  const long long* st = strides.begin();
  for (long long n : steps)
    if (__builtin_mul_overflow(n, *st++, &p) || __builtin_add_overflow(sum, p, &sum) || sum > 1LL << 58) return false;
  return true;
}
// A dimension of a launch has fewer than 2^32 work items; past that a grid is
// taken modulo 2^32, without an error.
inline bool launchable(long long blocks, int threads) { return blocks <= 0xffffffffLL / threads; }
inline bool rows_ok(long long rows, int n, long long ld) { return ld >= n && (rows == 0 || extent_ok({rows - 1}, {ld})); }
inline Span rows_span(const void* p, long long rows, int n, long long ld, size_t es) {
  return span(p, rows == 0 ? 0 : static_cast<size_t>((rows - 1) * ld + n) * es);
}

}  // namespace muon
