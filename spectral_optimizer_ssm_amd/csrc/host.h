// Host helpers of the C-ABI entry points: alignment, element sizes, overlap.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/muon.h"

namespace muon {

constexpr size_t kAlign = 256;   // of the blocks inside a workspace

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t dtype_size(int dt) { return dt == MUON_BF16 ? 2 : 4; }
inline bool overlaps(const char* a, size_t na, const char* b, size_t nb) { return a < b + nb && b < a + na; }

}  // namespace muon
