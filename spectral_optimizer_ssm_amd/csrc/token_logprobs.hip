// Log probabilities of tokens from rows of logits x, and their gradients:
//   t_j = scale (x_j - m),  m = max x,  L = log sum_j e^{t_j}
//   log p_id = t_id - L,   H = L - sum_j e^{t_j} t_j / sum_j e^{t_j}
// and the k largest logits, ties by the lowest index.  With p_j = e^{t_j - L}:
//   dx_j = scale (dlogp ([j = id] - p_j) - dH p_j (log p_j + H)).
//
// Bound by memory: the logits are read once.  Every thread keeps a running maximum,
// the sum of exponentials around it and their first moment, rescaled when the
// maximum grows; every wave keeps its k best in a sorted list, one a lane.
#include "ids.cuh"
#include "rows.cuh"

#include <float.h>
#include <limits.h>

namespace muon {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr float kNever = -256.0f;   // 2^-256 is 0 in float32: a finite exponent in its place

// Loads of a thread in flight: 64 bytes.
template <typename T>
struct Tile {
  static constexpr int V = Vec<T>::n, U = 4, n = V * U, width = kThreads * n;
};

// Floats in order as whole numbers (no NaN; -0 and 0 are one).
__device__ __forceinline__ int key_of(float v) {
  const int b = __float_as_int(v + 0.0f);
  return b ^ ((b >> 31) & INT_MAX);
}
__device__ __forceinline__ float value_of(int key) { return __int_as_float(key ^ ((key >> 31) & INT_MAX)); }
constexpr int kInfKey = 0x7F800000, kMinusInfKey = -kInfKey - 1;

// A wave's k best, sorted, one a lane: key INT_MIN where there are fewer.
struct Best {
  int key = INT_MIN, idx = -1;
  int bar = kMinusInfKey;   // only keys above it enter (uniform): nothing that has no probability
  float barf = -INFINITY;

  __device__ __forceinline__ void raise(int to) {
    if (to > bar) {
      bar = to;
      barf = value_of(to);
    }
  }
  // The k-th largest of the lanes' values is no larger than the k-th of all: what lies below never enters.
  __device__ __forceinline__ void start(float lane_max, int k) {
    const int mine = key_of(lane_max), lane = threadIdx.x & (kWave - 1);
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < kWave; ++i) {
      const int other = __builtin_amdgcn_readlane(mine, i);
      rank += other > mine || (other == mine && i < lane);
    }
    const int at = __ffsll(__ballot(rank == k - 1)) - 1;
    const int kth = __builtin_amdgcn_readlane(mine, at);
    if (kth > kMinusInfKey) raise(kth - 1 - (kth == 0));   // below 0 comes the smallest number below it, not -0
  }
  // (key, idx) uniform, key above the bar; equal keys come in the order of their index
  __device__ __forceinline__ void insert(int k, int nkey, int nidx) {
    const int lane = threadIdx.x & (kWave - 1);
    const int pos = __popcll(__ballot(key >= nkey));
    const int up = __shfl_up(key, 1, kWave), upi = __shfl_up(idx, 1, kWave);
    key = lane < pos ? key : lane == pos ? nkey : up;
    idx = lane < pos ? idx : lane == pos ? nidx : upi;
    raise(__builtin_amdgcn_readlane(key, k - 1));
  }
};

struct Sums {
  float m = -FLT_MAX, s = 0.0f, h = 0.0f;   // base 2 exponents

  template <bool ENTROPY>
  __device__ __forceinline__ void rescale(float to, float c) {
    const float d = fmaxf((m - to) * c, kNever), f = exp2f(d);
    if constexpr (ENTROPY) h = f * fmaf(d, s, h);
    s *= f;
    m = to;
  }
  template <bool ENTROPY>
  __device__ __forceinline__ void wave_merge(float c) {
    float to = m;
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) to = fmaxf(to, __shfl_xor(to, off, kWave));
    rescale<ENTROPY>(to, c);
    s = wave_total(s);
    if constexpr (ENTROPY) h = wave_total(h);
  }
};

// What a row leaves, from its sums: called by one thread.
struct RowOut {
  float m, logsum;
  bool none;   // nothing in the row has a probability
};
template <typename T>
__device__ __forceinline__ RowOut finish(const LogpLaunch& A, long long row, const Sums& w) {
  RowOut o;
  o.none = w.s == 0.0f;
  o.m = o.none ? -INFINITY : w.s == w.s ? w.m : w.s;   // a NaN or +inf in the row: NaN
  o.logsum = logf(w.s);
  if (A.stats != nullptr) {
    A.stats[2 * row] = o.m;
    A.stats[2 * row + 1] = o.logsum;
  }
  if (A.entropy != nullptr) A.entropy[row] = o.none ? 0.0f : o.logsum - kLn2 * w.h / w.s;
  if (A.logp != nullptr) {
    const long long id = id_at(A.ids, static_cast<uint32_t>(row));
    float v = 0.0f;
    if (id >= 0 && id < A.vocab) {
      const T x = static_cast<const T*>(A.x)[row * A.ldx + id];
      float f;
      if constexpr (sizeof(T) == 2) f = bf16_to_f32(x);
      else f = x;
      v = o.none ? -INFINITY : (f - o.m) * A.scale - o.logsum;
    }
    A.logp[row] = v;
  }
  return o;
}

// Threads place the best of `lists` lists of k in LDS (sorted each) by counting what is better.
template <typename F>
__device__ __forceinline__ void place(const int* keys, const int* idx, int n, int k, const F& put) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int key = keys[i], at = idx[i];
    if (key == INT_MIN) continue;
    int rank = 0;
    for (int j = 0; j < n; ++j) rank += keys[j] > key || (keys[j] == key && idx[j] < at);
    if (rank < k) put(rank, key, at);
  }
}
__device__ __forceinline__ void put_top(const LogpLaunch& A, long long row, const RowOut& o, int rank, int key, int at) {
  const bool lost = o.logsum != o.logsum;   // a NaN or +inf in the row
  A.top_ids[row * A.top + rank] = lost ? -1 : at;
  A.top_logp[row * A.top + rank] = (value_of(key) - o.m) * A.scale - o.logsum;
}
__device__ __forceinline__ void clear_top(const LogpLaunch& A, long long row, const RowOut& o) {
  for (int i = threadIdx.x; i < A.top; i += kThreads) {
    A.top_ids[row * A.top + i] = -1;
    A.top_logp[row * A.top + i] = o.logsum != o.logsum ? o.logsum : -INFINITY;
  }
}

template <typename T, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(kThreads) logp_kernel(LogpLaunch A) {
  using L = Tile<T>;
  __shared__ float wsum[3][kWaves];
  __shared__ RowOut rout;
  __shared__ int keys[TOP ? kWaves * kLogpMaxTop : 1], idx[TOP ? kWaves * kLogpMaxTop : 1];
  const long long blk = block_of_grid();
  const long long row = A.splits == 1 ? blk : blk / A.splits;
  if (row >= A.rows) return;
  const int split = static_cast<int>(blk - row * A.splits);
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const T* x = static_cast<const T*>(A.x) + row * A.ldx;
  // this workgroup's columns, in whole pieces
  const long long per = (static_cast<long long>(A.vocab) + A.splits - 1) / A.splits;
  const long long len = (per + L::V - 1) / L::V * L::V;
  const int c0 = static_cast<int>(split * len < A.vocab ? split * len : A.vocab);
  const int c1 = static_cast<int>(c0 + len < A.vocab ? c0 + len : A.vocab);
  const float c = A.scale * kLog2e;
  Sums sum;
  Best best;
  for (int b = c0; b < c1; b += L::width) {
    float v[L::U][L::V];
    const int first = b + static_cast<int>(threadIdx.x) * L::V;
#pragma unroll
    for (int u = 0; u < L::U; ++u) {
      const int col = first + u * kThreads * L::V;
      if (col + L::V <= c1) {
        unpack<T>(*reinterpret_cast<const u32x4_any*>(x + col), v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < L::V; ++e) {
          v[u][e] = -INFINITY;
          if (col + e < c1) {
            if constexpr (sizeof(T) == 2) v[u][e] = bf16_to_f32(x[col + e]);
            else v[u][e] = x[col + e];
          }
        }
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int u = 0; u < L::U; ++u)
#pragma unroll
      for (int e = 0; e < L::V; ++e) top = fmaxf(top, v[u][e]);
    sum.rescale<ENTROPY>(fmaxf(sum.m, top), c);
#pragma unroll
    for (int u = 0; u < L::U; ++u)
#pragma unroll
      for (int e = 0; e < L::V; ++e) {
        const float t = (v[u][e] - sum.m) * c, ex = __builtin_amdgcn_exp2f(t);
        sum.s += ex;
        if constexpr (ENTROPY) sum.h = fmaf(ex, fmaxf(t, kNever), sum.h);
      }
    if constexpr (TOP) {
      if (b == c0) best.start(top, A.top);
      if (__ballot(top > best.barf) == 0) continue;
#pragma unroll
      for (int u = 0; u < L::U; ++u) {
        float most = -INFINITY;
#pragma unroll
        for (int e = 0; e < L::V; ++e) most = fmaxf(most, v[u][e]);
        unsigned long long in;
        while ((in = __ballot(most > best.barf)) != 0) {
          const int l = __ffsll(in) - 1;
#pragma unroll
          for (int e = 0; e < L::V; ++e) {
            const int key = key_of(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(v[u][e]), l)));
            if (key > best.bar && key <= kInfKey)
              best.insert(A.top, key, b + (u * kThreads + w * kWave + l) * L::V + e);
          }
          if (lane == l) most = -INFINITY;
        }
      }
    }
  }
  sum.wave_merge<ENTROPY>(c);
  if (lane == 0) {
    wsum[0][w] = sum.m;
    wsum[1][w] = sum.s;
    wsum[2][w] = sum.h;
  }
  if constexpr (TOP) {
    if (lane < A.top) {
      keys[w * A.top + lane] = best.key;
      idx[w * A.top + lane] = best.idx;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    Sums all;
    for (int i = 0; i < kWaves; ++i) all.m = fmaxf(all.m, wsum[0][i]);
    for (int i = 0; i < kWaves; ++i) {
      Sums o{wsum[0][i], wsum[1][i], wsum[2][i]};
      o.rescale<ENTROPY>(all.m, c);
      all.s += o.s;
      all.h += o.h;
    }
    if (A.splits == 1) {
      rout = finish<T>(A, row, all);
    } else {
      float* p = A.part + 3 * blk;
      p[0] = all.m;
      p[1] = all.s;
      p[2] = all.h;
    }
  }
  if constexpr (TOP) {
    if (A.splits == 1) {
      __syncthreads();
      clear_top(A, row, rout);
      __syncthreads();
      place(keys, idx, kWaves * A.top, A.top, [&](int rank, int key, int at) { put_top(A, row, rout, rank, key, at); });
    } else {
      for (int i = threadIdx.x; i < A.top; i += kThreads) A.keys[blk * A.top + i] = INT_MIN;
      __syncthreads();
      place(keys, idx, kWaves * A.top, A.top, [&](int rank, int key, int at) {
        A.keys[blk * A.top + rank] = key;
        A.idx[blk * A.top + rank] = at;
      });
    }
  }
}

constexpr int kMaxSplits = 32;

// The rows whose columns several workgroups shared.
template <typename T>
__global__ void __launch_bounds__(kThreads) logp_join_kernel(LogpLaunch A) {
  __shared__ int keys[kMaxSplits * kLogpMaxTop], idx[kMaxSplits * kLogpMaxTop];
  __shared__ RowOut rout;
  const long long row = block_of_grid();
  if (row >= A.rows) return;
  const int n = A.splits * A.top;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    keys[i] = A.keys[row * n + i];
    idx[i] = keys[i] == INT_MIN ? -1 : A.idx[row * n + i];
  }
  const float c = A.scale * kLog2e;
  if (threadIdx.x < kWave) {
    Sums s;
    if (threadIdx.x < A.splits) {
      const float* p = A.part + 3 * (row * A.splits + threadIdx.x);
      s.m = p[0];
      s.s = p[1];
      s.h = p[2];
    }
    s.wave_merge<true>(c);
    if (threadIdx.x == 0) rout = finish<T>(A, row, s);
  }
  __syncthreads();
  if (A.top == 0) return;
  clear_top(A, row, rout);
  __syncthreads();
  place(keys, idx, n, A.top, [&](int rank, int key, int at) { put_top(A, row, rout, rank, key, at); });
}

// A workgroup a tile of a row's columns.
template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(kThreads) logp_grad_kernel(LogpGradLaunch A, unsigned tiles) {
  using L = Tile<T>;
  const long long blk = block_of_grid();
  const long long row = blk / tiles;
  if (row >= A.rows) return;
  const int first = static_cast<int>(blk - row * tiles) * L::width + static_cast<int>(threadIdx.x) * L::V;
  const T* x = static_cast<const T*>(A.x) + row * A.ldx;
  T* dx = static_cast<T*>(A.dx) + row * A.lddx;
  const float m = A.stats[2 * row], logsum = A.stats[2 * row + 1];
  long long id = A.ids.p != nullptr ? id_at(A.ids, static_cast<uint32_t>(row)) : -1;
  if (id >= A.vocab) id = -1;
  const float dl = id >= 0 && A.dlogp != nullptr ? A.dlogp[row * A.sdlogp] : 0.0f;
  float dh = 0.0f, H = 0.0f;
  if constexpr (ENTROPY) {
    dh = A.dentropy[row * A.sdentropy];
    H = A.entropy[row];
  }
  // dx = p (a + b log2 p), and scale dl more at the token
  const float c = A.scale * kLog2e, l2 = logsum * kLog2e;
  const float a = -A.scale * (dl + dh * H), b = -A.scale * dh * kLn2;
  // nothing to pass on, or nothing that has a probability
  const bool zero = (dl == 0.0f && dh == 0.0f) || logsum == -INFINITY;
#pragma unroll
  for (int u = 0; u < L::U; ++u) {
    const int col = first + u * kThreads * L::V;
    if (col >= A.vocab) return;
    const bool whole = col + L::V <= A.vocab;
    float v[L::V];
    if (zero) {
#pragma unroll
      for (int e = 0; e < L::V; ++e) v[e] = 0.0f;
    } else {
      if (whole) {
        unpack<T>(*reinterpret_cast<const u32x4_any*>(x + col), v);
      } else {
#pragma unroll
        for (int e = 0; e < L::V; ++e) {
          v[e] = -INFINITY;
          if (col + e < A.vocab) {
            if constexpr (sizeof(T) == 2) v[e] = bf16_to_f32(x[col + e]);
            else v[e] = x[col + e];
          }
        }
      }
#pragma unroll
      for (int e = 0; e < L::V; ++e) {
        const float t = fmaf(v[e] - m, c, -l2), p = __builtin_amdgcn_exp2f(t);
        v[e] = p * (ENTROPY ? fmaf(fmaxf(t, kNever), b, a) : a);
        if (col + e == id) v[e] += A.scale * dl;
      }
    }
    if (whole) {
      u32x4_t w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
        else w[e] = __float_as_uint(v[e]);
      }
      *reinterpret_cast<u32x4_any*>(dx + col) = w;
    } else {
#pragma unroll
      for (int e = 0; e < L::V; ++e)
        if (col + e < A.vocab) {
          if constexpr (sizeof(T) == 2) dx[col + e] = f32_to_bf16(v[e]);
          else dx[col + e] = v[e];
        }
    }
  }
}

template <typename T>
hipError_t logp(const LogpLaunch& A, hipStream_t st) {
  const dim3 grid = grid_of(A.rows * A.splits), block(kThreads);
  if (A.entropy != nullptr) {
    if (A.top > 0) hipLaunchKernelGGL((logp_kernel<T, true, true>), grid, block, 0, st, A);
    else hipLaunchKernelGGL((logp_kernel<T, true, false>), grid, block, 0, st, A);
  } else {
    if (A.top > 0) hipLaunchKernelGGL((logp_kernel<T, false, true>), grid, block, 0, st, A);
    else hipLaunchKernelGGL((logp_kernel<T, false, false>), grid, block, 0, st, A);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || A.splits == 1) return e;
  hipLaunchKernelGGL((logp_join_kernel<T>), grid_of(A.rows), block, 0, st, A);
  return hipGetLastError();
}
template <typename T>
hipError_t logp_grad(const LogpGradLaunch& A, hipStream_t st) {
  const unsigned tiles = (static_cast<unsigned>(A.vocab) + Tile<T>::width - 1) / Tile<T>::width;
  const dim3 grid = grid_of(A.rows * tiles), block(kThreads);
  if (A.dentropy != nullptr) hipLaunchKernelGGL((logp_grad_kernel<T, true>), grid, block, 0, st, A, tiles);
  else hipLaunchKernelGGL((logp_grad_kernel<T, false>), grid, block, 0, st, A, tiles);
  return hipGetLastError();
}

}  // namespace

// Few rows share the chip: workgroups a row, each with half a tile or more.
int logp_splits(long long rows, int vocab, bool bf16) {
  const long long half = (bf16 ? Tile<bf16_t>::width : Tile<float>::width) / 2;
  const long long want = rows >= 512 ? 1 : 1024 / (rows < 1 ? 1 : rows), most = vocab / half;
  const long long s = want < most ? want : most;
  return static_cast<int>(s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s);
}

hipError_t launch_logp(const LogpLaunch& A, bool bf16, hipStream_t st) { return bf16 ? logp<bf16_t>(A, st) : logp<float>(A, st); }
hipError_t launch_logp_grad(const LogpGradLaunch& A, bool bf16, hipStream_t st) {
  return bf16 ? logp_grad<bf16_t>(A, st) : logp_grad<float>(A, st);
}

}  // namespace muon
