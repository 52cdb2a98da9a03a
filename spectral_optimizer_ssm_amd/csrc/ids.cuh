// Token numbers, 32 or 64 bits wide, in runs of a stride.
#pragma once
#include "launch.h"

namespace muon {

__device__ __forceinline__ long long id_at(const IdsOperand& a, uint32_t t) {
  const uint32_t q = __umulhi(t, a.magic) >> a.shift;
  const long long e = static_cast<long long>(q) * a.stride + static_cast<long long>(t - q * a.run) * a.step;
  return a.wide ? static_cast<const long long*>(a.p)[e] : static_cast<const int*>(a.p)[e];
}

}  // namespace muon
