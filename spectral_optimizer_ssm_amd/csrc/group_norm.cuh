// What the group norm's two directions share: how a group of channels lies on
// threads, the gate's function and sums over the threads of a group.
#pragma once
#include "launch.h"
#include "rows.cuh"

namespace muon {

// Threads that share a group of w channels and the pieces that each takes (0: more
// than a workgroup holds, or less than a piece): as few threads as hold it, down to
// eight, so that narrow groups share a wave.
struct GroupPlan {
  int threads, pieces;
};
inline GroupPlan group_plan(int w, int elems) {
  if (w < elems) return {0, 0};
  const long long p = (static_cast<long long>(w) + elems - 1) / elems;
  if (p <= 8) return {8, 1};
  if (p <= 16) return {16, 1};
  if (p <= 32) return {16, 2};
  if (p <= 4 * 64) return {64, static_cast<int>((p + 63) / 64)};
  if (p <= 4 * 256) return {256, p <= 2 * 256 ? 2 : 4};
  if (p <= 4 * 512) return {512, 4};
  return {0, 0};
}

constexpr int kGroupThreads = 256;
// Threads of a workgroup whose groups take TPR threads each.
template <int TPR>
constexpr int group_threads() { return TPR < kGroupThreads ? kGroupThreads : TPR; }

// Sum over the TPR threads that share a group; every one of them gets it.
constexpr int kDppMirror = 0x140;
template <int TPR>
__device__ __forceinline__ float group_total(float v, float* red) {
  if constexpr (TPR <= 16) {
    v += dpp_f<kDppXor1>(v);
    v += dpp_f<kDppXor2>(v);
    v += dpp_f<kDppHalfMirror>(v);
    if constexpr (TPR == 16) v += dpp_f<kDppMirror>(v);
    return v;
  } else if constexpr (TPR == kWave) {
    return wave_total(v);
  } else {
    return block_sum(v, red);
  }
}

// 1 / (1 + e^-z): with float32 rows e is the full-accuracy one.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  const float e = sizeof(T) == 2 ? __expf(-z) : expf(-z);
  return __builtin_amdgcn_rcpf(1.0f + e);
}
// d silu(z) / dz from s = sigmoid(z)
__device__ __forceinline__ float silu_slope(float z, float s) { return s * fmaf(z, 1.0f - s, 1.0f); }

}  // namespace muon
