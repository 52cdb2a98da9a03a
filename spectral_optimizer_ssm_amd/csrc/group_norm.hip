// Group norm of rows, channels last, with a gate z (silu(z) = z / (1 + e^-z)):
//   before:  u = x silu(z),  y = (u - mu) r w + b          (the Mamba-2 block's)
//   after:   u = x,          y = ((u - mu) r w + b) silu(z)
//   none:    u = x,          y = act((u - mu) r w + b),  act the identity or silu
// mu and r = 1 / sqrt(mean((u - mu)^2) + eps) of each group of w channels of a row,
// mu = 0 without centering.
//
// Bound by memory.  A group is read once into the registers of 1 to 64 threads, or of
// a workgroup (16,384 bfloat16 or 8,192 float32 channels; wider ones are read three
// times); the variance is taken from the registers around the mean.  16,384 bfloat16
// rows of 1,536 with a gate take 28 us (151 MB, 5.3 TB/s), in groups of 8 channels 31,
// of 75, whose rows lie at odd elements, 40.
#include "group_norm.cuh"

namespace muon {
namespace {

template <typename T, NormGate G, int TPR, int PIECES, bool TINY>
__global__ void __launch_bounds__(group_threads<TPR>()) group_norm_kernel(GroupNormLaunch A) {
  constexpr int V = Vec<T>::n, kUnits = group_threads<TPR>() / TPR;
  __shared__ float red[group_threads<TPR>() / kWave];
  const int sub = kUnits == 1 ? 0 : threadIdx.x / TPR, t = threadIdx.x % TPR;
  const long long unit = block_of_grid() * kUnits + sub;
  if (unit >= static_cast<long long>(A.rows) * A.groups) return;   // whole groups of threads
  const unsigned row = A.groups == 1 ? static_cast<unsigned>(unit) : static_cast<unsigned>(unit) / A.groups;
  const int c0 = (static_cast<int>(static_cast<unsigned>(unit) - row * A.groups)) * A.w;
  const T* x = static_cast<const T*>(A.x) + row * A.ldx + c0;
  const T* z = G == kGateNone ? nullptr : static_cast<const T*>(A.z) + row * A.ldz + c0;
  float v[PIECES][V], a[PIECES][V];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    unpack<T>(group_raw<T, TPR, TINY>(x, i, t, A.w), v[i]);
    if constexpr (G != kGateNone) unpack<T>(group_raw<T, TPR, TINY>(z, i, t, A.w), a[i]);
  }
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const GroupPiece<T, TPR, TINY> p(i, t, A.w);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (G != kGateNone) a[i][e] *= sigmoid<T>(a[i][e]);
      if constexpr (G == kGateBefore) v[i][e] *= a[i][e];
      s += p.counts(e) ? v[i][e] : 0.0f;
    }
  }
  const float inv_w = 1.0f / static_cast<float>(A.w);
  const float mu = A.center ? group_total<TPR>(s, red) * inv_w : 0.0f;
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const GroupPiece<T, TPR, TINY> p(i, t, A.w);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      v[i][e] -= mu;
      const float d = p.counts(e) ? v[i][e] : 0.0f;
      q = fmaf(d, d, q);
    }
  }
  const float r = 1.0f / sqrtf(group_total<TPR>(q, red) * inv_w + A.eps);
  T* y = static_cast<T*>(A.y) + row * A.ldy + c0;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    float p[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] *= r;
    if (A.weight != nullptr) {
      group_param<T, TPR, TINY>(A.weight + c0, i, t, A.w, p);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] *= p[e];
    }
    if (A.bias != nullptr) {
      group_param<T, TPR, TINY>(A.bias + c0, i, t, A.w, p);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] += p[e];
    }
    if constexpr (G == kGateAfter) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] *= a[i][e];
    }
    if (G == kGateNone && A.act == kActSilu) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] *= sigmoid<T>(v[i][e]);
    }
    group_store<T, TPR, TINY>(y, i, t, A.w, v[i]);
  }
  if (t == 0) {
    if (A.mean != nullptr) A.mean[unit] = mu;
    if (A.rstd != nullptr) A.rstd[unit] = r;
  }
}

// Groups of any width: a workgroup a group, three readings.
template <typename T, NormGate G>
__global__ void __launch_bounds__(kGroupThreads) group_norm_any_kernel(GroupNormLaunch A) {
  constexpr int TPR = kGroupThreads;
  __shared__ float red[kGroupThreads / kWave];
  const int t = threadIdx.x;
  const long long unit = block_of_grid();
  if (unit >= static_cast<long long>(A.rows) * A.groups) return;
  const unsigned row = static_cast<unsigned>(unit) / A.groups;
  const int c0 = (static_cast<int>(static_cast<unsigned>(unit) - row * A.groups)) * A.w;
  const T* x = static_cast<const T*>(A.x) + row * A.ldx + c0;
  const T* z = G == kGateNone ? nullptr : static_cast<const T*>(A.z) + row * A.ldz + c0;
  const float inv_w = 1.0f / static_cast<float>(A.w);
  const auto silu_z = [&](int c) {
    const float g = element(z[c]);
    return g * sigmoid<T>(g);
  };
  const auto at = [&](int c) {
    if constexpr (G == kGateBefore) return element(x[c]) * silu_z(c);
    else return element(x[c]);
  };
  float mu = 0.0f;
  if (A.center) {
    float s = 0.0f;
    for (int c = t; c < A.w; c += TPR) s += at(c);
    mu = group_total<TPR>(s, red) * inv_w;
  }
  float q = 0.0f;
  for (int c = t; c < A.w; c += TPR) {
    const float d = at(c) - mu;
    q = fmaf(d, d, q);
  }
  const float r = 1.0f / sqrtf(group_total<TPR>(q, red) * inv_w + A.eps);
  T* y = static_cast<T*>(A.y) + row * A.ldy + c0;
  for (int c = t; c < A.w; c += TPR) {
    float o = (at(c) - mu) * r;
    if (A.weight != nullptr) o *= A.weight[c0 + c];
    if (A.bias != nullptr) o += A.bias[c0 + c];
    if constexpr (G == kGateAfter) o *= silu_z(c);
    if (G == kGateNone && A.act == kActSilu) o *= sigmoid<T>(o);
    if constexpr (sizeof(T) == 2) y[c] = f32_to_bf16(o);
    else y[c] = o;
  }
  if (t == 0) {
    if (A.mean != nullptr) A.mean[unit] = mu;
    if (A.rstd != nullptr) A.rstd[unit] = r;
  }
}

template <typename T, NormGate G, int TPR, int PIECES, bool TINY = false>
hipError_t run(const GroupNormLaunch& A, hipStream_t st) {
  constexpr int kUnits = group_threads<TPR>() / TPR;
  const long long units = static_cast<long long>(A.rows) * A.groups;
  hipLaunchKernelGGL((group_norm_kernel<T, G, TPR, PIECES, TINY>), grid_of((units + kUnits - 1) / kUnits), dim3(group_threads<TPR>()), 0, st, A);
  return hipGetLastError();
}

template <typename T, NormGate G>
hipError_t run_any(const GroupNormLaunch& A, hipStream_t st) {
  const GroupPlan p = group_plan(A.w, Vec<T>::n);
  switch (p.threads) {
    case 1: return p.tiny ? run<T, G, 1, 1, true>(A, st) : run<T, G, 1, 1>(A, st);
    case 2: return run<T, G, 2, 1>(A, st);
    case 4:
      if constexpr (sizeof(T) == 2)
        if (p.pieces == 3) return run<T, G, 4, 3>(A, st);
      return run<T, G, 4, 1>(A, st);
    case 8: return run<T, G, 8, 1>(A, st);
    case 16: return p.pieces == 1 ? run<T, G, 16, 1>(A, st) : run<T, G, 16, 2>(A, st);
    case 64:
      return p.pieces == 1 ? run<T, G, 64, 1>(A, st) : p.pieces == 2 ? run<T, G, 64, 2>(A, st) : p.pieces == 3 ? run<T, G, 64, 3>(A, st) : run<T, G, 64, 4>(A, st);
    case 256: return p.pieces == 2 ? run<T, G, 256, 2>(A, st) : run<T, G, 256, 4>(A, st);
    case 512: return run<T, G, 512, 4>(A, st);
  }
  hipLaunchKernelGGL((group_norm_any_kernel<T, G>), grid_of(static_cast<long long>(A.rows) * A.groups), dim3(kGroupThreads), 0, st, A);
  return hipGetLastError();
}

template <typename T>
hipError_t run_gate(const GroupNormLaunch& A, NormGate gate, hipStream_t st) {
  return gate == kGateBefore ? run_any<T, kGateBefore>(A, st) : gate == kGateAfter ? run_any<T, kGateAfter>(A, st) : run_any<T, kGateNone>(A, st);
}

}  // namespace

hipError_t launch_group_norm(const GroupNormLaunch& A, NormGate gate, bool bf16, hipStream_t st) {
  return bf16 ? run_gate<bf16_t>(A, gate, st) : run_gate<float>(A, gate, st);
}

}  // namespace muon
