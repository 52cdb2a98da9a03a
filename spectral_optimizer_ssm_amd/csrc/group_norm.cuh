// What the group norm's two directions share: how a group of channels lies on
// threads, the gate's function and sums over the threads of a group.
#pragma once
#include "launch.h"
#include "rows.cuh"

namespace muon {

// Threads that share a group of w channels and the pieces that each takes (no threads:
// more than a workgroup holds): as few threads as hold it, down to one, so that narrow
// groups share a wave; tiny: less than a piece, one thread and its elements one by one.
struct GroupPlan {
  int threads, pieces;
  bool tiny;
};
inline GroupPlan group_plan(int w, int elems) {
  if (w < elems) return {1, 1, true};
  const long long p = (static_cast<long long>(w) + elems - 1) / elems;
  // four threads with three pieces leave fewer idle than sixteen with one (24 groups of 75,
  // 13,981 rows of bfloat16: 40 and 72 us, 43 and 79; float32 pieces are too short for it)
  if (elems == 8 && p > 8 && p <= 12) return {4, 3, false};
  for (int t : {1, 2, 4, 8, 16})
    if (p <= t) return {t, 1, false};
  if (p <= 32) return {16, 2, false};
  if (p <= 4 * 64) return {64, static_cast<int>((p + 63) / 64), false};
  if (p <= 4 * 256) return {256, p <= 2 * 256 ? 2 : 4, false};
  if (p <= 4 * 512) return {512, 4, false};
  return {0, 0, false};
}

// A Piece, or a tiny group's elements.
template <typename T, int TPR, bool TINY>
struct GroupPiece : Piece<T, TPR> {
  __device__ __forceinline__ GroupPiece(int i, int t, int w) : Piece<T, TPR>(i, t, w) {}
};
template <typename T, int TPR>
struct GroupPiece<T, TPR, true> {
  static constexpr int V = Vec<T>::n, base = 0;
  int w;
  __device__ __forceinline__ GroupPiece(int, int, int w_) : w(w_) {}
  __device__ __forceinline__ bool counts(int e) const { return e < w; }
};
template <typename T, int TPR, bool TINY>
__device__ __forceinline__ u32x4_t group_raw(const T* row, int i, int t, int w) {
  if constexpr (!TINY) return load_raw<T, TPR>(row, i, t, w);
  u32x4_t o = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < Vec<T>::n; ++e)
    if (e < w) {
      if constexpr (sizeof(T) == 2) o[e / 2] |= static_cast<uint32_t>(row[e]) << (16 * (e % 2));
      else o[e] = __float_as_uint(row[e]);
    }
  return o;
}
template <typename T, int TPR, bool TINY>
__device__ __forceinline__ void group_param(const float* row, int i, int t, int w, float (&o)[Vec<T>::n]) {
  if constexpr (!TINY) {
    load_param<T, TPR>(row, i, t, w, o);
  } else {
#pragma unroll
    for (int e = 0; e < Vec<T>::n; ++e) o[e] = e < w ? row[e] : 0.0f;
  }
}
template <typename T, int TPR, bool TINY>
__device__ __forceinline__ void group_store(T* row, int i, int t, int w, const float (&v)[Vec<T>::n]) {
  if constexpr (!TINY) {
    store_piece<T, TPR>(row, i, t, w, v);
  } else {
#pragma unroll
    for (int e = 0; e < Vec<T>::n; ++e)
      if (e < w) {
        if constexpr (sizeof(T) == 2) row[e] = f32_to_bf16(v[e]);
        else row[e] = v[e];
      }
  }
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
    if constexpr (TPR >= 2) v += dpp_f<kDppXor1>(v);
    if constexpr (TPR >= 4) v += dpp_f<kDppXor2>(v);
    if constexpr (TPR >= 8) v += dpp_f<kDppHalfMirror>(v);
    if constexpr (TPR >= 16) v += dpp_f<kDppMirror>(v);
    return v;
  } else if constexpr (TPR == kWave) {
    return wave_total(v);
  } else {
    return block_sum(v, red);
  }
}

// 1 / (1 + e^-z).  With float32 rows what rounding -z log2(e) loses is put back, so that
// e^-z is off by a few 2^-24 wherever s is neither 0 nor 1; past +-128 it is.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  constexpr float kLog2e = 1.44269504088896341f, kLow = 1.92596299e-8f, kLn2 = 0.69314718055994531f;   // log2(e) = kLog2e + kLow
  float e;
  if constexpr (sizeof(T) == 2) {
    e = __builtin_amdgcn_exp2f(-kLog2e * z);
  } else {
    const float x = -__builtin_amdgcn_fmed3f(z, -128.0f, 128.0f), t = x * kLog2e;
    e = __builtin_amdgcn_exp2f(t) * fmaf(fmaf(x, kLow, fmaf(x, kLog2e, -t)), kLn2, 1.0f);
  }
  return __builtin_amdgcn_rcpf(1.0f + e);
}
// d silu(z) / dz from s = sigmoid(z)
__device__ __forceinline__ float silu_slope(float z, float s) { return s * fmaf(z, 1.0f - s, 1.0f); }

}  // namespace muon
