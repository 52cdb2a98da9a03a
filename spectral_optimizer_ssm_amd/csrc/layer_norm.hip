// Layer norm over rows of n elements and its gradients:
//   y = (x - mu) r w + bias,  mu = mean(x),  r = 1 / sqrt(mean((x - mu)^2) + eps)
//   with xh = (x - mu) r and t = dy w:
//   dx = r (t - mean(t) - xh mean(t xh)),  dw = sum_rows dy xh,  dbias = sum_rows dy.
// Without centering mu = 0 and mean(t) leaves dx (a root-mean-square norm).
//
// Bound by memory: a row is read once into registers (by a wave, or by a workgroup
// of 256 or 512 threads beyond kPieces pieces a lane), the variance is taken
// from the registers around the mean (two passes, so a large mean costs no
// digits), and every statistic and sum is float32.  Rows longer than a
// workgroup's registers are read again from cache.  The backward pass keeps one
// column sum per element of its registers over all the rows that it walks, with
// the next row's loads in flight; the workgroups' sums go to the workspace and a
// second kernel adds them in fixed order.  16,384 bfloat16 rows of 768 take
// 12 us forward (50 MB, 4.2 TB/s) and 21 us backward (75 MB, 18 us of it the
// walk at 4.2 TB/s).
#include "launch.h"
#include "rows.cuh"

namespace muon {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;       // most pieces a thread holds of a row

// Sum over the TPR threads that share a row; every thread gets it.
template <int TPR>
__device__ __forceinline__ float row_total(float v, float* red) {
  if constexpr (TPR == kWave) return wave_total(v);
  else return block_sum(v, red);
}

// Threads of a workgroup whose rows take TPR threads each.
template <int TPR>
constexpr int threads_of() { return TPR < kThreads ? kThreads : TPR; }

// PIECES pieces of a row a thread, TPR threads a row.
template <typename T, int TPR, int PIECES>
__global__ void __launch_bounds__(threads_of<TPR>()) norm_kernel(NormLaunch A) {
  constexpr int V = Vec<T>::n, kRows = threads_of<TPR>() / TPR;
  __shared__ float red[threads_of<TPR>() / kWave];
  const int sub = kRows == 1 ? 0 : threadIdx.x / TPR, t = threadIdx.x % TPR;
  const long long row = block_of_grid() * kRows + sub;
  if (row >= A.rows) return;   // whole waves or whole workgroups
  const T* x = static_cast<const T*>(A.x) + row * A.ldx;
  float v[PIECES][V];
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) unpack<T>(load_raw<T, TPR>(x, i, t, A.n), v[i]);
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const Piece<T, TPR> p(i, t, A.n);
#pragma unroll
    for (int e = 0; e < V; ++e) s += p.counts(e) ? v[i][e] : 0.0f;
  }
  const float inv_n = 1.0f / static_cast<float>(A.n);
  const float mu = A.center ? row_total<TPR>(s, red) * inv_n : 0.0f;
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const Piece<T, TPR> p(i, t, A.n);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      v[i][e] -= mu;
      const float d = p.counts(e) ? v[i][e] : 0.0f;
      q = fmaf(d, d, q);
    }
  }
  const float r = 1.0f / sqrtf(row_total<TPR>(q, red) * inv_n + A.eps);
  T* y = static_cast<T*>(A.y) + row * A.ldy;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    float p[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[i][e] *= r;
    if (A.w != nullptr) {
      load_param<T, TPR>(A.w, i, t, A.n, p);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] *= p[e];
    }
    if (A.bias != nullptr) {
      load_param<T, TPR>(A.bias, i, t, A.n, p);
#pragma unroll
      for (int e = 0; e < V; ++e) v[i][e] += p[e];
    }
    store_piece<T, TPR>(y, i, t, A.n, v[i]);
  }
  if (t == 0) {
    if (A.mean != nullptr) A.mean[row] = mu;
    if (A.rstd != nullptr) A.rstd[row] = r;
  }
}

// Rows of any length: a workgroup a row, three readings.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_long_kernel(NormLaunch A) {
  __shared__ float red[kThreads / kWave];
  const long long row = block_of_grid();
  if (row >= A.rows) return;
  const T* x = static_cast<const T*>(A.x) + row * A.ldx;
  const float inv_n = 1.0f / static_cast<float>(A.n);
  const auto at = [&](int c) {
    if constexpr (sizeof(T) == 2) return bf16_to_f32(x[c]);
    else return x[c];
  };
  float mu = 0.0f;
  if (A.center) {
    float s = 0.0f;
    for (int c = threadIdx.x; c < A.n; c += kThreads) s += at(c);
    mu = block_sum(s, red) * inv_n;
  }
  float q = 0.0f;
  for (int c = threadIdx.x; c < A.n; c += kThreads) {
    const float d = at(c) - mu;
    q = fmaf(d, d, q);
  }
  const float r = 1.0f / sqrtf(block_sum(q, red) * inv_n + A.eps);
  T* y = static_cast<T*>(A.y) + row * A.ldy;
  for (int c = threadIdx.x; c < A.n; c += kThreads) {
    float o = (at(c) - mu) * r;
    if (A.w != nullptr) o *= A.w[c];
    if (A.bias != nullptr) o += A.bias[c];
    if constexpr (sizeof(T) == 2) y[c] = f32_to_bf16(o);
    else y[c] = o;
  }
  if (threadIdx.x == 0) {
    if (A.mean != nullptr) A.mean[row] = mu;
    if (A.rstd != nullptr) A.rstd[row] = r;
  }
}

// Workgroup b walks rows b kRows + 0.., a grid apart, and leaves its column
// sums in part[b][2][n] (or, alone in the grid, in dw and dbias).
template <typename T, int TPR, int PIECES>
__global__ void __launch_bounds__(threads_of<TPR>()) norm_grad_kernel(NormGradLaunch A) {
  constexpr int V = Vec<T>::n, kAll = threads_of<TPR>(), kRows = kAll / TPR;
  __shared__ float red[kAll / kWave];
  __shared__ float cols[TPR == kWave ? kWave * V * PIECES : 1];
  const int sub = kRows == 1 ? 0 : threadIdx.x / TPR, t = threadIdx.x % TPR;
  const float inv_n = 1.0f / static_cast<float>(A.n);
  float wv[PIECES][V], dw[PIECES][V], db[PIECES][V];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    if (A.w != nullptr) load_param<T, TPR>(A.w, i, t, A.n, wv[i]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (A.w == nullptr) wv[i][e] = 1.0f;
      dw[i][e] = db[i][e] = 0.0f;
    }
  }
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  const bool center = A.mean != nullptr;
  u32x4_t xn[PIECES], gn[PIECES];   // the next row's, as they are loaded
  float mun = 0.0f, rn = 0.0f;
  const auto load_row = [&](long long row) {
    const T* x = static_cast<const T*>(A.x) + row * A.ldx;
    const T* dy = static_cast<const T*>(A.dy) + row * A.lddy;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      xn[i] = load_raw<T, TPR>(x, i, t, A.n);
      gn[i] = load_raw<T, TPR>(dy, i, t, A.n);
    }
    mun = center ? A.mean[row] : 0.0f;
    rn = A.rstd[row];
  };
  long long row = static_cast<long long>(blockIdx.x) * kRows + sub;
  if (row < A.rows) load_row(row);
  for (; row < A.rows; row += step) {
    float xh[PIECES][V], g[PIECES][V];
    const float mu = mun, r = rn;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      asm volatile("" : "+v"(xn[i]), "+v"(gn[i]));   // unpacked here, not where they were loaded, in twice the registers
      unpack<T>(xn[i], xh[i]);
      unpack<T>(gn[i], g[i]);
    }
    load_row(row + step < A.rows ? row + step : row);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const Piece<T, TPR> p(i, t, A.n);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        xh[i][e] = (xh[i][e] - mu) * r;
        dw[i][e] = fmaf(g[i][e], xh[i][e], dw[i][e]);
        db[i][e] += g[i][e];
        g[i][e] *= wv[i][e];
        const float c = p.counts(e) ? g[i][e] : 0.0f;
        s1 += c;
        s2 = fmaf(c, xh[i][e], s2);
      }
    }
    asm volatile("" : "+v"(s1), "+v"(s2));   // both summed up before the branch: their terms take no registers across it
    s1 = center ? row_total<TPR>(s1, red) * inv_n : 0.0f;
    s2 = row_total<TPR>(s2, red) * inv_n;
    T* dx = static_cast<T*>(A.dx) + row * A.lddx;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) g[i][e] = r * (g[i][e] - s1 - xh[i][e] * s2);
      store_piece<T, TPR>(dx, i, t, A.n, g[i]);
    }
  }
  float* out[2] = {A.dw, A.dbias};
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float (&acc)[PIECES][V] = k == 0 ? dw : db;
    if (out[k] == nullptr) continue;   // a sum that nobody asked for
    float* to = gridDim.x == 1 ? out[k] : A.part + (2LL * blockIdx.x + k) * A.n;
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
      for (int j = threadIdx.x; j < kWave * V * PIECES; j += kAll) {
        const int slot = j / kWave;
        const Piece<T, TPR> p(slot / V, j % kWave, A.n);
        if (p.counts(slot % V)) to[p.base + slot % V] = cols[j];
      }
    } else {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const Piece<T, TPR> p(i, t, A.n);
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (p.counts(e)) to[p.base + e] = acc[i][e];
      }
    }
  }
}

// Rows of any length: a workgroup a row at a time, column sums in the
// workspace (each element always by the same thread).
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_grad_long_kernel(NormGradLaunch A) {
  __shared__ float red[kThreads / kWave];
  const float inv_n = 1.0f / static_cast<float>(A.n);
  float* pw = A.part + 2LL * blockIdx.x * A.n;
  float* pb = pw + A.n;
  bool first = true;
  for (long long row = blockIdx.x; row < A.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(A.x) + row * A.ldx;
    const T* dy = static_cast<const T*>(A.dy) + row * A.lddy;
    const float mu = A.mean != nullptr ? A.mean[row] : 0.0f, r = A.rstd[row];
    const auto val = [](T v) {
      if constexpr (sizeof(T) == 2) return bf16_to_f32(v);
      else return v;
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < A.n; c += kThreads) {
      const float xh = (val(x[c]) - mu) * r, g = val(dy[c]), t = A.w != nullptr ? g * A.w[c] : g;
      s1 += t;
      s2 = fmaf(t, xh, s2);
      pw[c] = first ? g * xh : fmaf(g, xh, pw[c]);
      pb[c] = first ? g : pb[c] + g;
    }
    first = false;
    s1 = A.mean != nullptr ? block_sum(s1, red) * inv_n : 0.0f;
    s2 = block_sum(s2, red) * inv_n;
    T* dx = static_cast<T*>(A.dx) + row * A.lddx;
    for (int c = threadIdx.x; c < A.n; c += kThreads) {
      const float xh = (val(x[c]) - mu) * r, g = val(dy[c]), t = A.w != nullptr ? g * A.w[c] : g;
      const float o = r * (t - s1 - xh * s2);
      if constexpr (sizeof(T) == 2) dx[c] = f32_to_bf16(o);
      else dx[c] = o;
    }
  }
  if (first)   // no rows: empty sums
    for (int c = threadIdx.x; c < 2 * A.n; c += kThreads) pw[c] = 0.0f;
}

// dw and dbias from the workgroups' sums: 64 columns a workgroup, its sixteen
// waves each every sixteenth part, their sums added in order.
constexpr int kPartWaves = 16;
__global__ void __launch_bounds__(kPartWaves * kWave) norm_parts_kernel(const float* part, int parts, int n, float* dw, float* dbias) {
  __shared__ float s[kPartWaves * kWave];
  float* out = blockIdx.y == 0 ? dw : dbias;
  if (out == nullptr) return;
  const int lane = threadIdx.x & (kWave - 1), col = static_cast<int>(blockIdx.x) * kWave + lane, w = threadIdx.x / kWave;
  float acc = 0.0f;
  if (col < n) {
    const float* p = part + static_cast<long long>(blockIdx.y) * n + col;
#pragma unroll 8
    for (int i = w; i < parts; i += kPartWaves) acc += p[2LL * i * n];
  }
  s[threadIdx.x] = acc;
  __syncthreads();
  if (w == 0 && col < n) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kPartWaves; ++i) t += s[i * kWave + lane];
    out[col] = t;
  }
}

// Threads that share a row of n elements (0: more than a workgroup holds, or less
// than a piece) and the pieces of it that each takes: as few threads as hold it.
// A wave needs no barrier: 8,192 bfloat16 rows of 2,048 take 15 us forward and 25 backward by
// waves, 29 and 80 by workgroups.  Reading a row again costs more than a larger
// workgroup: 1,024 rows of 16,384 take 15 and 52 us by 512 threads that hold it,
// 65 and 323 read in passes.
struct RowPlan {
  int threads, pieces;
};
RowPlan row_plan(int n, int elems) {
  if (n < elems) return {0, 0};
  for (int t : {kWave, kThreads, 2 * kThreads}) {
    const int p = (n + elems * t - 1) / (elems * t);
    if (p <= kPieces) return {t, p <= 1 ? 1 : p <= 2 ? 2 : 4};
  }
  return {0, 0};
}

template <typename T, int TPR, int PIECES>
hipError_t norm(const NormLaunch& A, hipStream_t st) {
  constexpr int kRows = threads_of<TPR>() / TPR;
  const dim3 grid = grid_of((A.rows + kRows - 1) / kRows), block(threads_of<TPR>());
  hipLaunchKernelGGL((norm_kernel<T, TPR, PIECES>), grid, block, 0, st, A);
  return hipGetLastError();
}

template <typename T>
hipError_t norm_any(const NormLaunch& A, hipStream_t st) {
  const RowPlan p = row_plan(A.n, Vec<T>::n);
  if (p.threads == kWave) return p.pieces == 1 ? norm<T, kWave, 1>(A, st) : p.pieces == 2 ? norm<T, kWave, 2>(A, st) : norm<T, kWave, 4>(A, st);
  if (p.threads == kThreads) return p.pieces == 2 ? norm<T, kThreads, 2>(A, st) : norm<T, kThreads, 4>(A, st);
  if (p.threads != 0) return norm<T, 2 * kThreads, 4>(A, st);
  hipLaunchKernelGGL((norm_long_kernel<T>), grid_of(A.rows), dim3(kThreads), 0, st, A);
  return hipGetLastError();
}

template <typename T, int TPR, int PIECES>
hipError_t grad(const NormGradLaunch& A, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(A.parts)), block(threads_of<TPR>());
  hipLaunchKernelGGL((norm_grad_kernel<T, TPR, PIECES>), grid, block, 0, st, A);
  return hipGetLastError();
}

template <typename T>
hipError_t grad_any(const NormGradLaunch& A, hipStream_t st) {
  const RowPlan p = row_plan(A.n, Vec<T>::n);
  hipError_t e;
  if (p.threads == kWave) {
    e = p.pieces == 1 ? grad<T, kWave, 1>(A, st) : p.pieces == 2 ? grad<T, kWave, 2>(A, st) : grad<T, kWave, 4>(A, st);
  } else if (p.threads == kThreads) {
    e = p.pieces == 2 ? grad<T, kThreads, 2>(A, st) : grad<T, kThreads, 4>(A, st);
  } else if (p.threads != 0) {
    e = grad<T, 2 * kThreads, 4>(A, st);
  } else {
    hipLaunchKernelGGL((norm_grad_long_kernel<T>), dim3(static_cast<unsigned>(A.parts)), dim3(kThreads), 0, st, A);
    e = hipGetLastError();
  }
  if (e != hipSuccess || (A.parts == 1 && p.threads != 0) || (A.dw == nullptr && A.dbias == nullptr)) return e;
  return launch_norm_parts(A.part, A.parts, A.n, A.dw, A.dbias, st);
}

}  // namespace

hipError_t launch_norm_parts(const float* part, int parts, int n, float* dw, float* db, hipStream_t st) {
  hipLaunchKernelGGL(norm_parts_kernel, dim3((n + kWave - 1) / kWave, 2), dim3(kPartWaves * kWave), 0, st, part, parts, n, dw, db);
  return hipGetLastError();
}

// Workgroups of the backward pass: enough to fill the chip, where there are that
// many rows eight to a wave, or four to a workgroup that takes a row together,
// since each leaves 2 n sums to be added: 1,024 bfloat16 rows of 16,384 take
// 52 us four to a workgroup, 80 two and 77 sixteen.  At most 512 (65,536 rows of
// 768: 70 us, 100 with 256, 76 with 1,024), or 256 of 512 threads, of which a
// compute unit holds one (1,031 float32 rows of 4,099: 21 us, 28 with 258).
int norm_grad_parts(long long rows, int n, bool bf16) {
  const RowPlan p = row_plan(n, bf16 ? Vec<bf16_t>::n : Vec<float>::n);
  const long long per = p.threads == kWave ? 8LL * kThreads / kWave : 4, most = p.threads == 2 * kThreads ? 256 : 512;
  const long long want = (rows + per - 1) / per;
  return static_cast<int>(want < 1 ? 1 : want > most ? most : want);
}

hipError_t launch_norm(const NormLaunch& A, bool bf16, hipStream_t st) {
  return bf16 ? norm_any<bf16_t>(A, st) : norm_any<float>(A, st);
}
hipError_t launch_norm_grad(const NormGradLaunch& A, bool bf16, hipStream_t st) {
  return bf16 ? grad_any<bf16_t>(A, st) : grad_any<float>(A, st);
}

}  // namespace muon
