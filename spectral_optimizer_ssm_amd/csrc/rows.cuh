// Rows in pieces of 16 bytes: what the kernels that walk rows of any length and
// alignment share (layer_norm.hip, group_norm.hip, embedding.hip, token_logprobs.hip).
#pragma once
#include "common.cuh"

namespace muon {

template <typename T>
__device__ __forceinline__ float element(T v) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(v);
  else return v;
}

template <typename T>
struct Vec {
  static constexpr int n = 16 / static_cast<int>(sizeof(T));   // elements of a piece
};

// Piece i of a row of n elements that thread t takes, of the TPR that share it:
// 16 adjacent bytes from element `base`, of which those from `first` on count.
// The memory takes 16 bytes at any address, so rows need no alignment, and a
// piece that would pass the row's end is moved back to end with it: what it then
// shares with its neighbour both compute and store alike, and only one counts in
// sums (16,384 bfloat16 rows of 767: 13 us forward and 22 backward, as of 768).
template <typename T, int TPR>
struct Piece {
  static constexpr int V = Vec<T>::n;
  int base, first;
  __device__ __forceinline__ Piece(int i, int t, int n) {
    const int col = (i * TPR + t) * V;
    base = col < n - V ? col : n - V;
    first = col - base;
  }
  __device__ __forceinline__ bool any() const { return first < V; }
  __device__ __forceinline__ bool counts(int e) const { return e >= first; }
};

typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <typename T, int TPR>
__device__ __forceinline__ u32x4_t load_raw(const T* row, int i, int t, int n) {
  return *reinterpret_cast<const u32x4_any*>(row + Piece<T, TPR>(i, t, n).base);
}
template <typename T>
__device__ __forceinline__ void unpack(u32x4_t w, float (&o)[Vec<T>::n]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (sizeof(T) == 2) {
      o[2 * e] = lo_bf16(w[e]);
      o[2 * e + 1] = hi_bf16(w[e]);
    } else {
      o[e] = __uint_as_float(w[e]);
    }
  }
}
// The float parameters at a piece's columns.
template <typename T, int TPR>
__device__ __forceinline__ void load_param(const float* row, int i, int t, int n, float (&o)[Vec<T>::n]) {
  const float* p = row + Piece<T, TPR>(i, t, n).base;
#pragma unroll
  for (int e = 0; e < Vec<T>::n; e += 4) {
    const u32x4_t w = *reinterpret_cast<const u32x4_any*>(p + e);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[e + k] = __uint_as_float(w[k]);
  }
}

template <typename T, int TPR>
__device__ __forceinline__ void store_piece(T* row, int i, int t, int n, const float (&v)[Vec<T>::n]) {
  const Piece<T, TPR> p(i, t, n);
  if (!p.any()) return;
  u32x4_t w;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (sizeof(T) == 2) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
    else w[e] = __float_as_uint(v[e]);
  }
  *reinterpret_cast<u32x4_any*>(row + p.base) = w;
}

// A dimension of a launch has fewer than 2^32 work items, which 2^24 rows of a
// workgroup each exceed: past 2^20 workgroups the grid has a second dimension.
inline dim3 grid_of(long long blocks) {
  const long long x = blocks < (1 << 20) ? blocks : 1 << 20;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>((blocks + x - 1) / x));
}
__device__ __forceinline__ long long block_of_grid() { return static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x; }

}  // namespace muon
