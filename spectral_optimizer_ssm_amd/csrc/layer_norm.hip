// Layer norm over rows of n elements and its gradients:
//   y = (x - mu) r w + bias,  mu = mean(x),  r = 1 / sqrt(mean((x - mu)^2) + eps)
//   with xh = (x - mu) r and t = dy w:
//   dx = r (t - mean(t) - xh mean(t xh)),  dw = sum_rows dy xh,  dbias = sum_rows dy.
// Without centering mu = 0 and mean(t) leaves dx (a root-mean-square norm).
//
// Bound by HBM: a row is read once into registers (a wave a row, a workgroup a
// row beyond kWaveMax 16-byte pieces a lane), the variance is taken from the
// registers around the mean (two passes, so a large mean costs no digits), and
// every statistic and sum is float32.  Rows longer than a workgroup's
// registers are read again from cache.  The backward pass keeps one column sum
// per element of its registers over all the rows that it walks; workgroups'
// sums go to the workspace and a second kernel adds them in fixed order.
#include "launch.h"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;       // most 16-byte pieces a thread holds of a row

template <typename T>
struct Vec;
template <>
struct Vec<bf16_t> {
  static constexpr int n = 8;
};
template <>
struct Vec<float> {
  static constexpr int n = 4;
};

// Elements [col, col + n) of a row as floats (0 past `width`).
template <typename T>
__device__ __forceinline__ void load_piece(const T* row, int col, int width, bool vec, float (&o)[Vec<T>::n]) {
#pragma unroll
  for (int i = 0; i < Vec<T>::n; ++i) o[i] = 0.0f;
  if (col >= width) return;
  if (vec) {
    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(row + col);
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = lo_bf16(w[i]);
        o[2 * i + 1] = hi_bf16(w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __uint_as_float(w[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::n; ++i)
      if (col + i < width) {
        if constexpr (sizeof(T) == 2) o[i] = bf16_to_f32(row[col + i]);
        else o[i] = row[col + i];
      }
  }
}

template <typename T>
__device__ __forceinline__ void store_piece(T* row, int col, int width, bool vec, const float (&v)[Vec<T>::n]) {
  if (col >= width) return;
  if (vec) {
    u32x4_t w;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    }
    *reinterpret_cast<u32x4_t*>(row + col) = w;
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::n; ++i)
      if (col + i < width) {
        if constexpr (sizeof(T) == 2) row[col + i] = f32_to_bf16(v[i]);
        else row[col + i] = v[i];
      }
  }
}

// Sum over the TPR threads that share a row; every thread gets it.
template <int TPR>
__device__ __forceinline__ float row_total(float v, float* red) {
  if constexpr (TPR == kWave) return wave_total(v);
  else return block_sum(v, red);
}

// PIECES 16-byte pieces of a row a thread, TPR threads a row.
template <typename T, int TPR, int PIECES>
__global__ void __launch_bounds__(kThreads) norm_kernel(NormLaunch A) {
  constexpr int V = Vec<T>::n;
  __shared__ float red[kThreads / kWave];
  const int sub = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * (kThreads / TPR) + sub;
  if (row >= A.rows) return;   // whole waves or whole workgroups
  const T* x = static_cast<const T*>(A.x) + row * A.ldx;
  float v[PIECES][V];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    load_piece<T>(x, (i * TPR + t) * V, A.n, A.vec, v[i]);
#pragma unroll
    for (int e = 0; e < V; ++e) s += v[i][e];
  }
  const float inv_n = 1.0f / static_cast<float>(A.n);
  const float mu = A.center ? row_total<TPR>(s, red) * inv_n : 0.0f;
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = (i * TPR + t) * V + e < A.n ? v[i][e] - mu : 0.0f;
      v[i][e] = d;
      q = fmaf(d, d, q);
    }
  const float r = 1.0f / sqrtf(row_total<TPR>(q, red) * inv_n + A.eps);
  T* y = static_cast<T*>(A.y) + row * A.ldy;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int col = (i * TPR + t) * V;
    float wv[V], bv[V];
    if (A.w != nullptr) {
#pragma unroll
      for (int u = 0; u < V / 4; ++u) load_piece<float>(A.w, col + 4 * u, A.n, A.pvec, *reinterpret_cast<float(*)[4]>(wv + 4 * u));
    }
    if (A.bias != nullptr) {
#pragma unroll
      for (int u = 0; u < V / 4; ++u) load_piece<float>(A.bias, col + 4 * u, A.n, A.pvec, *reinterpret_cast<float(*)[4]>(bv + 4 * u));
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float o = v[i][e] * r;
      if (A.w != nullptr) o *= wv[e];
      if (A.bias != nullptr) o += bv[e];
      v[i][e] = o;
    }
    store_piece<T>(y, col, A.n, A.vec, v[i]);
  }
  if (t == 0) {
    if (A.mean != nullptr) A.mean[row] = mu;
    if (A.rstd != nullptr) A.rstd[row] = r;
  }
}

// Rows of any length: a workgroup a row, three readings.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_long_kernel(NormLaunch A) {
  constexpr int V = Vec<T>::n;
  __shared__ float red[kThreads / kWave];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(A.x) + row * A.ldx;
  const float inv_n = 1.0f / static_cast<float>(A.n);
  float mu = 0.0f, v[V];
  if (A.center) {
    float s = 0.0f;
    for (int col = threadIdx.x * V; col < A.n; col += kThreads * V) {
      load_piece<T>(x, col, A.n, A.vec, v);
#pragma unroll
      for (int e = 0; e < V; ++e) s += v[e];
    }
    mu = block_sum(s, red) * inv_n;
  }
  float q = 0.0f;
  for (int col = threadIdx.x * V; col < A.n; col += kThreads * V) {
    load_piece<T>(x, col, A.n, A.vec, v);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = col + e < A.n ? v[e] - mu : 0.0f;
      q = fmaf(d, d, q);
    }
  }
  const float r = 1.0f / sqrtf(block_sum(q, red) * inv_n + A.eps);
  T* y = static_cast<T*>(A.y) + row * A.ldy;
  for (int col = threadIdx.x * V; col < A.n; col += kThreads * V) {
    load_piece<T>(x, col, A.n, A.vec, v);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float o = (v[e] - mu) * r;
      if (col + e < A.n) {
        if (A.w != nullptr) o *= A.w[col + e];
        if (A.bias != nullptr) o += A.bias[col + e];
      }
      v[e] = o;
    }
    store_piece<T>(y, col, A.n, A.vec, v);
  }
  if (threadIdx.x == 0) {
    if (A.mean != nullptr) A.mean[row] = mu;
    if (A.rstd != nullptr) A.rstd[row] = r;
  }
}

// Workgroup b walks rows b kThreads / TPR + 0.., a grid apart, and leaves its
// column sums in part[b][2][n] (or, alone in the grid, in dw and dbias).
template <typename T, int TPR, int PIECES>
__global__ void __launch_bounds__(kThreads) norm_grad_kernel(NormGradLaunch A) {
  constexpr int V = Vec<T>::n;
  constexpr int kRows = kThreads / TPR;
  __shared__ float red[kThreads / kWave];
  __shared__ float cols[TPR == kWave ? kWave * V * PIECES : 1];
  const int sub = threadIdx.x / TPR, t = threadIdx.x % TPR;
  const float inv_n = 1.0f / static_cast<float>(A.n);
  float wv[PIECES][V], dw[PIECES][V], db[PIECES][V];
#pragma unroll
  for (int i = 0; i < PIECES; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int col = (i * TPR + t) * V + e;
      wv[i][e] = col < A.n ? (A.w != nullptr ? A.w[col] : 1.0f) : 0.0f;
      dw[i][e] = db[i][e] = 0.0f;
    }
  for (long long row = static_cast<long long>(blockIdx.x) * kRows + sub; row < A.rows;
       row += static_cast<long long>(gridDim.x) * kRows) {
    const T* x = static_cast<const T*>(A.x) + row * A.ldx;
    const T* dy = static_cast<const T*>(A.dy) + row * A.lddy;
    const float mu = A.mean != nullptr ? A.mean[row] : 0.0f, r = A.rstd[row];
    float xh[PIECES][V], g[PIECES][V];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      load_piece<T>(x, (i * TPR + t) * V, A.n, A.vec, xh[i]);
      load_piece<T>(dy, (i * TPR + t) * V, A.n, A.vec, g[i]);
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        xh[i][e] = (xh[i][e] - mu) * r;   // past the row: times g = 0
        dw[i][e] = fmaf(g[i][e], xh[i][e], dw[i][e]);
        db[i][e] += g[i][e];
        g[i][e] *= wv[i][e];
        s1 += g[i][e];
        s2 = fmaf(g[i][e], xh[i][e], s2);
      }
    s1 = A.mean != nullptr ? row_total<TPR>(s1, red) * inv_n : 0.0f;
    s2 = row_total<TPR>(s2, red) * inv_n;
    T* dx = static_cast<T*>(A.dx) + row * A.lddx;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) g[i][e] = r * (g[i][e] - s1 - xh[i][e] * s2);
      store_piece<T>(dx, (i * TPR + t) * V, A.n, A.vec, g[i]);
    }
  }
  float* out[2];
  out[0] = gridDim.x == 1 ? A.dw : A.part + 2LL * blockIdx.x * A.n;
  out[1] = gridDim.x == 1 ? A.dbias : A.part + (2LL * blockIdx.x + 1) * A.n;
  if (gridDim.x > 1) {   // sums that nobody asked for are not written
    if (A.dw == nullptr) out[0] = nullptr;
    if (A.dbias == nullptr) out[1] = nullptr;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float (&acc)[PIECES][V] = k == 0 ? dw : db;
    if (out[k] == nullptr) continue;
    if constexpr (TPR == kWave) {
      // the waves' sums, in order
      for (int u = 0; u < kRows; ++u) {
        __syncthreads();
        if (sub == u) {
#pragma unroll
          for (int i = 0; i < PIECES; ++i)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              float* c = cols + (i * V + e) * kWave + t;
              *c = u == 0 ? acc[i][e] : *c + acc[i][e];
            }
        }
      }
      __syncthreads();
      for (int col = threadIdx.x; col < A.n; col += kThreads) {
        const int piece = col / V, e = col % V;
        out[k][col] = cols[((piece / kWave) * V + e) * kWave + piece % kWave];
      }
    } else {
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int col = (i * TPR + t) * V + e;
          if (col < A.n) out[k][col] = acc[i][e];
        }
    }
  }
}

// Rows of any length: a workgroup a row at a time, column sums in the
// workspace (each element always by the same thread).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_grad_long_kernel(NormGradLaunch A) {
  constexpr int V = Vec<T>::n;
  __shared__ float red[kThreads / kWave];
  const float inv_n = 1.0f / static_cast<float>(A.n);
  float* pw = A.part + 2LL * blockIdx.x * A.n;
  float* pb = pw + A.n;
  bool first = true;
  for (long long row = blockIdx.x; row < A.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(A.x) + row * A.ldx;
    const T* dy = static_cast<const T*>(A.dy) + row * A.lddy;
    const float mu = A.mean != nullptr ? A.mean[row] : 0.0f, r = A.rstd[row];
    float xv[V], g[V], s1 = 0.0f, s2 = 0.0f;
    for (int col = threadIdx.x * V; col < A.n; col += kThreads * V) {
      load_piece<T>(x, col, A.n, A.vec, xv);
      load_piece<T>(dy, col, A.n, A.vec, g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (col + e >= A.n) continue;
        const float xh = (xv[e] - mu) * r, t = A.w != nullptr ? g[e] * A.w[col + e] : g[e];
        s1 += t;
        s2 = fmaf(t, xh, s2);
        pw[col + e] = first ? g[e] * xh : fmaf(g[e], xh, pw[col + e]);
        pb[col + e] = first ? g[e] : pb[col + e] + g[e];
      }
    }
    first = false;
    s1 = A.mean != nullptr ? block_sum(s1, red) * inv_n : 0.0f;
    s2 = block_sum(s2, red) * inv_n;
    T* dx = static_cast<T*>(A.dx) + row * A.lddx;
    for (int col = threadIdx.x * V; col < A.n; col += kThreads * V) {
      load_piece<T>(x, col, A.n, A.vec, xv);
      load_piece<T>(dy, col, A.n, A.vec, g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float t = A.w != nullptr && col + e < A.n ? g[e] * A.w[col + e] : g[e];
        g[e] = r * (t - s1 - (xv[e] - mu) * r * s2);
      }
      store_piece<T>(dx, col, A.n, A.vec, g);
    }
  }
  if (first)   // no rows: empty sums
    for (int col = threadIdx.x; col < 2 * A.n; col += kThreads) pw[col] = 0.0f;
}

// dw and dbias from the workgroups' sums: 64 columns a workgroup, its four
// waves each a quarter of the parts, added in order.
__global__ void __launch_bounds__(kThreads) norm_parts_kernel(const float* part, int parts, int n, float* dw, float* dbias) {
  __shared__ float s[kThreads];
  float* out = blockIdx.y == 0 ? dw : dbias;
  if (out == nullptr) return;
  const int col = static_cast<int>(blockIdx.x) * kWave + (threadIdx.x & 63), w = threadIdx.x >> 6;
  float acc = 0.0f;
  if (col < n)
    for (int p = w; p < parts; p += 4) acc += part[(2LL * p + blockIdx.y) * n + col];
  s[threadIdx.x] = acc;
  __syncthreads();
  if (w == 0 && col < n) out[col] = (s[threadIdx.x] + s[64 + threadIdx.x]) + (s[128 + threadIdx.x] + s[192 + threadIdx.x]);
}

// Pieces a lane needs when a wave (or a workgroup) takes the row.
int pieces(int n, int elems, int threads) { return (n + elems * threads - 1) / (elems * threads); }

template <typename T, int TPR>
hipError_t norm_pieces(const NormLaunch& A, int p, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>((A.rows + kThreads / TPR - 1) / (kThreads / TPR))), block(kThreads);
  if (p == 1) hipLaunchKernelGGL((norm_kernel<T, TPR, 1>), grid, block, 0, st, A);
  else if (p == 2) hipLaunchKernelGGL((norm_kernel<T, TPR, 2>), grid, block, 0, st, A);
  else hipLaunchKernelGGL((norm_kernel<T, TPR, 4>), grid, block, 0, st, A);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_any(const NormLaunch& A, hipStream_t st) {
  const int p = pieces(A.n, Vec<T>::n, kWave), pw = pieces(A.n, Vec<T>::n, kThreads);
  if (p <= kPieces) return norm_pieces<T, kWave>(A, p, st);
  if (pw <= kPieces) return norm_pieces<T, kThreads>(A, pw, st);
  hipLaunchKernelGGL((norm_long_kernel<T>), dim3(static_cast<unsigned>(A.rows)), dim3(kThreads), 0, st, A);
  return hipGetLastError();
}

template <typename T, int TPR>
hipError_t grad_pieces(const NormGradLaunch& A, int p, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(A.parts)), block(kThreads);
  if (p == 1) hipLaunchKernelGGL((norm_grad_kernel<T, TPR, 1>), grid, block, 0, st, A);
  else if (p == 2) hipLaunchKernelGGL((norm_grad_kernel<T, TPR, 2>), grid, block, 0, st, A);
  else hipLaunchKernelGGL((norm_grad_kernel<T, TPR, 4>), grid, block, 0, st, A);
  return hipGetLastError();
}

template <typename T>
hipError_t grad_any(const NormGradLaunch& A, hipStream_t st) {
  const int p = pieces(A.n, Vec<T>::n, kWave), pw = pieces(A.n, Vec<T>::n, kThreads);
  hipError_t e;
  bool direct = A.parts == 1;
  if (p <= kPieces) {
    e = grad_pieces<T, kWave>(A, p, st);
  } else if (pw <= kPieces) {
    e = grad_pieces<T, kThreads>(A, pw, st);
  } else {
    direct = false;
    hipLaunchKernelGGL((norm_grad_long_kernel<T>), dim3(static_cast<unsigned>(A.parts)), dim3(kThreads), 0, st, A);
    e = hipGetLastError();
  }
  if (e != hipSuccess || direct || (A.dw == nullptr && A.dbias == nullptr)) return e;
  hipLaunchKernelGGL(norm_parts_kernel, dim3((A.n + kWave - 1) / kWave, 2), dim3(kThreads), 0, st, A.part, A.parts, A.n, A.dw,
                     A.dbias);
  return hipGetLastError();
}

}  // namespace

// Workgroups of the backward pass: enough to fill the chip, at least eight
// rows a wave where there are that many.
int norm_grad_parts(long long rows, int n, bool bf16) {
  const bool wave_rows = pieces(n, bf16 ? Vec<bf16_t>::n : Vec<float>::n, kWave) <= kPieces;
  const long long per = wave_rows ? 4 * 8 : 8;
  const long long want = (rows + per - 1) / per;
  return static_cast<int>(want < 1 ? 1 : want > 512 ? 512 : want);
}

hipError_t launch_norm(const NormLaunch& A, bool bf16, hipStream_t st) {
  return bf16 ? norm_any<bf16_t>(A, st) : norm_any<float>(A, st);
}
hipError_t launch_norm_grad(const NormGradLaunch& A, bool bf16, hipStream_t st) {
  return bf16 ? grad_any<bf16_t>(A, st) : grad_any<float>(A, st);
}

}  // namespace muon
