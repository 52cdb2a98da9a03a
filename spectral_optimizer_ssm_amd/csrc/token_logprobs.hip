// Log probabilities of tokens from rows of logits x, and their gradients:
//   t_j = scale (x_j - m),  m = max x,  L = log sum_j e^{t_j}
//   log p_id = t_id - L,   H = L - sum_j e^{t_j} t_j / sum_j e^{t_j}
// and the k largest logits, ties by the lowest index.  With p_j = e^{t_j - L}:
//   dx_j = scale (dlogp ([j = id] - p_j) - dH p_j (log p_j + H)).
//
// Bound by memory, with vector instructions close behind: the logits are read once.
// Every thread keeps a running maximum, the sum of exponentials around it and their
// first moment, rescaled when the maximum grows.  The k largest of the first tile's
// maxima is a bar that few of a row's logits pass; those are collected in LDS and the k
// best picked by counting.  16,384 bfloat16 rows of 50,280 take 288 us with the entropy
// (1.65 GB, 5.7 TB/s), their gradient 550 (3.3 GB, 6.0 TB/s); 1,021 float32 rows of
// 50,277 with the 20 likeliest 48 us, 40 without (205 MB); four rows, shared by twelve
// workgroups each, 8 + 4 us.
#include "ids.cuh"
#include "rows.cuh"

#include <float.h>

#include <algorithm>
#include <type_traits>

namespace muon {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.69314718055994531f;
constexpr float kNever = -256.0f;   // 2^-256 is 0 in float32: a finite exponent in its place

// U pieces of 16 bytes a thread.
template <typename T, int PIECES>
struct Tile {
  static constexpr int V = Vec<T>::n, U = PIECES, width = kThreads * V * U;
};
// (Forward, 64 bytes in flight a thread: 1,021 float32 rows with 20 likeliest 48 us, 56 with
// two pieces; gradient of 16,384 bfloat16 rows 550 us with two, 606 with four, 692 with one.)
constexpr int kPieces = 4, kGradPieces = 2;

// This thread's pieces of a row's columns [from, from + width), -inf from `end` on.  A
// tile that ends before it is loaded without a branch, so that its loads go out together.
template <typename T, int U>
__device__ __forceinline__ void load_tile(const T* x, int first, int from, int end, float (&v)[U][Vec<T>::n]) {
  using L = Tile<T, U>;
  if (end - from >= L::width) {
    u32x4_t w[L::U];
#pragma unroll
    for (int u = 0; u < L::U; ++u) w[u] = *reinterpret_cast<const u32x4_any*>(x + first + u * kThreads * L::V);
#pragma unroll
    for (int u = 0; u < L::U; ++u) unpack<T>(w[u], v[u]);
  } else {
#pragma unroll
    for (int u = 0; u < L::U; ++u) {
      const int col = first + u * kThreads * L::V;
      if (col + L::V <= end) {
        unpack<T>(*reinterpret_cast<const u32x4_any*>(x + col), v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < L::V; ++e) {
          v[u][e] = -INFINITY;
          if (col + e < end) v[u][e] = element(x[col + e]);
        }
      }
    }
  }
}

// A logit and its index as one number: larger is better, ties go to the lowest index
// (-0 and 0 are one; not for NaN).
typedef unsigned long long Rank;
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) { return __uint_as_float(key ^ (~static_cast<uint32_t>(static_cast<int>(key) >> 31) | 0x80000000u)); }
__device__ __forceinline__ Rank rank_of(float v, int idx) { return static_cast<Rank>(key_of(v)) << 32 | ~static_cast<uint32_t>(idx); }
__device__ __forceinline__ float value_of(Rank r) { return value_of(static_cast<uint32_t>(r >> 32)); }
__device__ __forceinline__ int index_of(Rank r) { return static_cast<int>(~static_cast<uint32_t>(r)); }
constexpr uint32_t kMinusInfKey = 0x007FFFFFu;
constexpr Rank kNobody = static_cast<Rank>(kMinusInfKey) << 32 | 0xFFFFFFFFu;   // only logits above -inf are better

// The best of a row so far: what passes the bar is put in `buf` in any order; when that
// fills up, the k best of it stay and the last of them is the new bar.
constexpr int kRoom = 1024;
struct Best {
  Rank buf[kRoom + 2], best[kLogpMaxTop];
  Rank bar;
  int count;

  // best[0..min(n, k)) of buf[0..n), by counting what is better; all threads call it.
  __device__ __forceinline__ void select(int n, int k) {
    if (threadIdx.x < 2) buf[n + threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const Rank mine = buf[i];
      int at = 0;
#pragma unroll 8
      for (int j = 0; j < n; j += 2) at += (buf[j] > mine) + (buf[j + 1] > mine);
      if (at < k) best[at] = mine;
    }
    __syncthreads();
  }
  __device__ __forceinline__ void keep(int n, int k) {
    select(n, k);
    if (threadIdx.x < k && threadIdx.x < n) buf[threadIdx.x] = best[threadIdx.x];
    if (threadIdx.x == 0) {
      count = n < k ? n : k;
      if (n >= k) bar = best[k - 1];
    }
    __syncthreads();
  }
  // The k-th largest of 64 values, each the largest of four threads', is no larger than
  // the k-th of all.
  __device__ __forceinline__ void start(float thread_max, int k) {
    float* all = reinterpret_cast<float*>(buf);
    all[threadIdx.x] = thread_max;
    if (threadIdx.x == 0) count = 0;
    __syncthreads();
    if (threadIdx.x < kWave) {
      float most = all[threadIdx.x];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) most = fmaxf(most, all[w * kWave + threadIdx.x]);
      const uint32_t mine = key_of(most);
      int at = 0;
#pragma unroll 8
      for (int j = 0; j < kWave; ++j) {
        const uint32_t other = __builtin_amdgcn_readlane(mine, j) + (j < static_cast<int>(threadIdx.x));   // ties: the lower lane first
        at += other > mine;
      }
      if (at == k - 1) bar = most > -INFINITY ? (static_cast<Rank>(mine) << 32) - 1 : kNobody;
    }
    __syncthreads();
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
      const float f = element(static_cast<const T*>(A.x)[row * A.ldx + id]);
      v = o.none ? -INFINITY : (f - o.m) * A.scale - o.logsum;
    }
    A.logp[row] = v;
  }
  return o;
}

// The places of a row's list from its n best.
__device__ __forceinline__ void put_top(const LogpLaunch& A, long long row, const RowOut& o, const Rank* best, int n) {
  const bool lost = o.logsum != o.logsum;   // a NaN or +inf in the row
  for (int i = threadIdx.x; i < A.top; i += kThreads) {
    A.top_ids[row * A.top + i] = i < n && !lost ? index_of(best[i]) : -1;
    A.top_logp[row * A.top + i] = lost ? o.logsum : i < n ? (value_of(best[i]) - o.m) * A.scale - o.logsum : -INFINITY;
  }
}

template <typename T, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(kThreads, 8) logp_kernel(LogpLaunch A) {
  using L = Tile<T, kPieces>;
  __shared__ float wsum[3][kWaves];
  __shared__ RowOut rout;
  __shared__ typename std::conditional<TOP, Best, int>::type best;
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
  for (int b = c0; b < c1; b += L::width) {
    float v[L::U][L::V];
    const int first = b + static_cast<int>(threadIdx.x) * L::V;
    load_tile(x, first, b, c1, v);
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
      // this thread's elements that may enter, by their place in the tile; read again, for they are few
      uint32_t pending = 0;
      const float barf = value_of(best.bar);
      if (top >= barf) {
#pragma unroll
        for (int u = 0; u < L::U; ++u)
#pragma unroll
          for (int e = 0; e < L::V; ++e) pending |= v[u][e] >= barf ? 1u << (u * L::V + e) : 0u;
      }
      for (;;) {
        const Rank bar = best.bar;
        for (uint32_t left = pending; left != 0; left &= left - 1) {
          const int i = __ffs(left) - 1, col = first + i / L::V * kThreads * L::V + i % L::V;
          float f = -INFINITY;
          if (col < c1) f = element(x[col]);
          const Rank mine = rank_of(f, col);
          int at = kRoom;
          if (mine > bar) at = atomicAdd(&best.count, 1);
          if (mine > bar && at < kRoom) best.buf[at] = mine;
          if (mine <= bar || at < kRoom) pending &= ~(left & -left);
        }
        __syncthreads();
        const int n = best.count;
        __syncthreads();   // all have read it before any adds to it
        if (n > A.top + kWave) best.keep(n < kRoom ? n : kRoom, A.top);
        if (n <= kRoom) break;   // else: what found no room comes again
      }
    }
  }
  sum.wave_merge<ENTROPY>(c);
  if (lane == 0) {
    wsum[0][w] = sum.m;
    wsum[1][w] = sum.s;
    wsum[2][w] = sum.h;
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
    const int found = c0 < c1 ? best.count : 0, n = found < A.top ? found : A.top;
    best.select(found, A.top);
    if (A.splits == 1) {
      put_top(A, row, rout, best.best, n);
    } else {
      for (int i = threadIdx.x; i < A.top; i += kThreads) A.ranks[blk * A.top + i] = i < n ? best.best[i] : 0;
    }
  }
}

constexpr int kMaxSplits = 32;

// The rows whose columns several workgroups shared.
template <typename T>
__global__ void __launch_bounds__(kThreads) logp_join_kernel(LogpLaunch A) {
  __shared__ Rank all[kMaxSplits * kLogpMaxTop + 2], best[kLogpMaxTop];
  __shared__ Rank low;
  __shared__ int count;
  __shared__ RowOut rout;
  const long long row = block_of_grid();
  if (row >= A.rows) return;
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
    // the splits hold as many as `top` that are no worse than the worst of their (top / splits)-ths
    if (A.top > 0) {
      const int nth = (A.top + A.splits - 1) / A.splits;
      Rank r = threadIdx.x < A.splits ? A.ranks[(row * A.splits + threadIdx.x) * A.top + nth - 1] : ~static_cast<Rank>(0);
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) {
        const Rank o = __shfl_xor(r, off, kWave);
        r = o < r ? o : r;
      }
      if (threadIdx.x == 0) low = r;
    }
    if (threadIdx.x == 0) {
      count = 0;
      rout = finish<T>(A, row, s);
    }
  }
  __syncthreads();
  if (A.top == 0) return;
  for (int i = threadIdx.x; i < A.splits * A.top; i += kThreads) {
    const Rank r = A.ranks[row * A.splits * A.top + i];
    if (r != 0 && r >= low) all[atomicAdd(&count, 1)] = r;
  }
  __syncthreads();
  const int n = count;
  if (threadIdx.x < 2) all[n + threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Rank mine = all[i];
    int at = 0;
#pragma unroll 8
    for (int j = 0; j < n; j += 2) at += (all[j] > mine) + (all[j + 1] > mine);
    if (at < A.top) best[at] = mine;
  }
  __syncthreads();
  put_top(A, row, rout, best, n < A.top ? n : A.top);
}

// A workgroup a tile of a row's columns.
template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(kThreads) logp_grad_kernel(LogpGradLaunch A, unsigned tiles) {
  using L = Tile<T, kGradPieces>;
  const long long blk = block_of_grid();
  const long long row = blk / tiles;
  if (row >= A.rows) return;
  const int from = static_cast<int>(blk - row * tiles) * L::width, first = from + static_cast<int>(threadIdx.x) * L::V;
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
  float v[L::U][L::V];
  if (zero) {
#pragma unroll
    for (int u = 0; u < L::U; ++u)
#pragma unroll
      for (int e = 0; e < L::V; ++e) v[u][e] = 0.0f;
  } else {
    load_tile(x, first, from, A.vocab, v);
    const int at = static_cast<int>(id) - first;   // of the token among this thread's elements
#pragma unroll
    for (int u = 0; u < L::U; ++u)
#pragma unroll
      for (int e = 0; e < L::V; ++e) {
        const float t = fmaf(v[u][e] - m, c, -l2), p = __builtin_amdgcn_exp2f(t);
        v[u][e] = p * (ENTROPY ? fmaf(fmaxf(t, kNever), b, a) : a);
        if (at == u * kThreads * L::V + e) v[u][e] += A.scale * dl;
      }
  }
#pragma unroll
  for (int u = 0; u < L::U; ++u) {
    const int col = first + u * kThreads * L::V;
    if (col + L::V <= A.vocab) {
      u32x4_t w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 2) w[e] = pack_bf16x2(v[u][2 * e], v[u][2 * e + 1]);
        else w[e] = __float_as_uint(v[u][e]);
      }
      *reinterpret_cast<u32x4_any*>(dx + col) = w;
    } else {
#pragma unroll
      for (int e = 0; e < L::V; ++e)
        if (col + e < A.vocab) {
          if constexpr (sizeof(T) == 2) dx[col + e] = f32_to_bf16(v[u][e]);
          else dx[col + e] = v[u][e];
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
  const unsigned tiles = (static_cast<unsigned>(A.vocab) + Tile<T, kGradPieces>::width - 1) / Tile<T, kGradPieces>::width;
  const dim3 grid = grid_of(A.rows * tiles), block(kThreads);
  if (A.dentropy != nullptr) hipLaunchKernelGGL((logp_grad_kernel<T, true>), grid, block, 0, st, A, tiles);
  else hipLaunchKernelGGL((logp_grad_kernel<T, false>), grid, block, 0, st, A, tiles);
  return hipGetLastError();
}

}  // namespace

// Few rows share the chip: workgroups a row, each with half a tile or more, and a second
// launch that joins them.  A row of 32 KB or less is one workgroup's (8,000 float32
// logits, up to 511 rows: 15 us a call, 18 shared), and so is one of 128 KB or less where
// there are 128 (200 rows of 50,280: bfloat16 15 and 18 us, but float32, of 200 KB, 28
// and 23 with the likeliest), and any where there are 512 (512 rows of 50,280 float32
// logits 21 us, 24 shared).
int logp_splits(long long rows, int vocab, bool bf16) {
  const long long bytes = static_cast<long long>(vocab) * (bf16 ? 2 : 4);
  if (rows < 1 || rows >= 512 || bytes <= 32 << 10 || (rows >= 128 && bytes <= 128 << 10)) return 1;
  const long long half = (bf16 ? Tile<bf16_t, kPieces>::width : Tile<float, kPieces>::width) / 2;
  return static_cast<int>(std::min({1024 / rows, vocab / half, static_cast<long long>(kMaxSplits)}));
}

hipError_t launch_logp(const LogpLaunch& A, bool bf16, hipStream_t st) { return bf16 ? logp<bf16_t>(A, st) : logp<float>(A, st); }
hipError_t launch_logp_grad(const LogpGradLaunch& A, bool bf16, hipStream_t st) {
  return bf16 ? logp_grad<bf16_t>(A, st) : logp_grad<float>(A, st);
}

}  // namespace muon
