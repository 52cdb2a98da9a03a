// Token embedding and its gradient:
//   y_t = scale table[id_t],   dtable[v] = scale sum_{t: id_t = v} dy_t,
// with zeros for ids outside the table, which take no gradient.
//
// The gradient's sums run over tokens sorted by id, in the tokens' order, so they
// need no atomics and repeat bit for bit.  Three launches:
//   1. a workgroup for each range of ids walks all ids twice, counts and places
//      those in its range; others write the table's zeros meanwhile;
//   2. a thread for 16 bytes of a row's columns and a chunk of the sorted tokens
//      adds up each id's rows; an id that spans two borders of chunks leaves a
//      part sum in each, all others are written at once;
//   3. the parts of those ids are added, in order.
#include "launch.h"
#include "ids.cuh"
#include "rows.cuh"

namespace muon {
namespace {

// V elements of T (16 bytes or less) at any element as floats, and back.
template <typename T, int V>
__device__ __forceinline__ void load_n(const T* p, float (&o)[V]) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) o[0] = bf16_to_f32(*p);
    else o[0] = *p;
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(V * sizeof(T) / 4), aligned(sizeof(T))));
    const words w = *reinterpret_cast<const words*>(p);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (sizeof(T) == 2) o[e] = e % 2 == 0 ? lo_bf16(w[e / 2]) : hi_bf16(w[e / 2]);
      else o[e] = __uint_as_float(w[e]);
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_n(T* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    if constexpr (sizeof(T) == 2) *p = f32_to_bf16(v[0]);
    else *p = v[0];
  } else if constexpr (sizeof(T) == 4 && V == 8) {
    store_n<T, 4>(p, {v[0], v[1], v[2], v[3]});
    store_n<T, 4>(p + 4, {v[4], v[5], v[6], v[7]});
  } else {
    typedef uint32_t words __attribute__((ext_vector_type(V * sizeof(T) / 4), aligned(sizeof(T))));
    words w;
#pragma unroll
    for (int e = 0; e < static_cast<int>(V * sizeof(T) / 4); ++e) {
      if constexpr (sizeof(T) == 2) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
      else w[e] = __float_as_uint(v[e]);
    }
    *reinterpret_cast<words*>(p) = w;
  }
}

// ---------------------------------------------------------------------------
// forward: a workgroup takes `per` tokens, a thread pieces of V columns; the last
// piece of a row is moved back to end with it
// ---------------------------------------------------------------------------
constexpr int kThreads = 256;

template <typename TT, typename T, int V>
__global__ void __launch_bounds__(kThreads) embed_kernel(EmbedLaunch A, uint32_t per, uint32_t pieces) {
  const long long first = block_of_grid() * per;
  if (first >= A.tokens) return;
  const uint32_t here = A.tokens - first < per ? static_cast<uint32_t>(A.tokens - first) : per;
  for (uint32_t i = threadIdx.x; i < here * pieces; i += kThreads) {
    const uint32_t t = i / pieces, col = (i - t * pieces) * V;
    const int c = static_cast<int>(col) < A.n - V ? static_cast<int>(col) : A.n - V;
    const long long token = first + t, id = id_at(A.ids, static_cast<uint32_t>(token));
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0.0f;
    if (id >= 0 && id < A.vocab) {
      load_n<TT, V>(static_cast<const TT*>(A.table) + id * A.ldt + c, v);
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] *= A.scale;
    }
    store_n<T, V>(static_cast<T*>(A.y) + token * A.ldy + c, v);
  }
}

template <typename TT, typename T, int V>
hipError_t embed(const EmbedLaunch& A, hipStream_t st) {
  const uint32_t pieces = (static_cast<uint32_t>(A.n) + V - 1) / V;
  const uint32_t most = pieces < 4 * kThreads ? 4 * kThreads / pieces : 1;
  uint32_t per = A.tokens / 1024;   // four workgroups a compute unit before any takes a second token
  per = per < 1 ? 1 : per > most ? most : per;
  const long long blocks = (static_cast<long long>(A.tokens) + per - 1) / per;
  hipLaunchKernelGGL((embed_kernel<TT, T, V>), grid_of(blocks), dim3(kThreads), 0, st, A, per, pieces);
  return hipGetLastError();
}
template <typename TT, typename T>
hipError_t embed_any(const EmbedLaunch& A, hipStream_t st) {
  return A.n >= 4 ? embed<TT, T, 4>(A, st) : embed<TT, T, 1>(A, st);
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
constexpr int kRange = 256;          // most ids of a workgroup
constexpr int kFillPerThread = 8;    // 16-byte stores

int range_of(int vocab) {
  const int r = (vocab + 255) / 256;   // a workgroup for each compute unit before ranges reach kRange
  return r < 1 ? 1 : r > kRange ? kRange : r;
}

// Blocks below `sorters`: ids [b range, (b + 1) range).  The others: zeros.
template <typename TT>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(EmbedGradLaunch A, int range, int sorters, int bits, long long bytes) {
  __shared__ int hist[kSortWaves][kRange];
  __shared__ int waves[kSortWaves];
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const long long blk = block_of_grid();
  if (blk >= sorters) {
    char* p = static_cast<char*>(A.dtable);
    const u32x4_t zero = {0, 0, 0, 0};
    long long at = ((blk - sorters) * kFillPerThread * kSortThreads + threadIdx.x) * 16;
#pragma unroll
    for (int i = 0; i < kFillPerThread; ++i, at += kSortThreads * 16) {
      if (at + 16 <= bytes) {
        *reinterpret_cast<u32x4_any*>(p + at) = zero;
      } else {
        for (long long b = at; b < bytes && b < at + 16; b += sizeof(TT)) *reinterpret_cast<TT*>(p + b) = TT(0);
      }
    }
    return;
  }
  const int lo = static_cast<int>(blk) * range, hi = A.vocab - lo < range ? A.vocab : lo + range;
  for (int i = threadIdx.x; i < kSortWaves * kRange; i += kSortThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  // this wave's tokens
  const uint32_t span = ((A.tokens + kSortWaves - 1) / kSortWaves + kWave - 1) / kWave * kWave;
  const uint32_t t0 = w * span < A.tokens ? w * span : A.tokens, t1 = A.tokens - t0 < span ? A.tokens : t0 + span;
  constexpr int U = 4;
  int below = 0;
  for (uint32_t t = t0; t < t1; t += U * kWave) {
    long long id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t at = t + u * kWave + lane;
      id[u] = at < t1 ? id_at(A.ids, at) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      below += id[u] >= 0 && id[u] < lo;
      if (id[u] >= lo && id[u] < hi) atomicAdd(&hist[w][id[u] - lo], 1);
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) below += __shfl_xor(below, off, kWave);
  if (lane == 0) waves[w] = below;
  __syncthreads();
  int base = 0;   // of the range in the sorted order
  for (int i = 0; i < kSortWaves; ++i) base += waves[i];
  __syncthreads();
  // places: by id, then by wave
  int total = 0;
  if (threadIdx.x < kRange) {
    for (int i = 0; i < kSortWaves; ++i) total += hist[i][threadIdx.x];
  }
  int incl = total;   // prefix over the ids: the first four waves hold them
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const int v = __shfl_up(incl, off, kWave);
    if (lane >= off) incl += v;
  }
  if (lane == kWave - 1) waves[w] = incl;
  __syncthreads();
  if (threadIdx.x < kRange) {
    int at = base + incl - total;
    for (int i = 0; i < w; ++i) at += waves[i];
    if (blk == sorters - 1 && threadIdx.x == kRange - 1) *A.count = at + total;
    for (int i = 0; i < kSortWaves; ++i) {
      const int n = hist[i][threadIdx.x];
      hist[i][threadIdx.x] = at;
      at += n;
    }
  }
  __syncthreads();
  for (uint32_t t = t0; t < t1; t += U * kWave) {
    long long id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t at = t + u * kWave + lane;
      id[u] = at < t1 ? id_at(A.ids, at) : -1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = id[u] >= lo && id[u] < hi;
      unsigned long long same = __ballot(in);   // lanes with this lane's id
      if (same == 0) continue;
      const int d = in ? static_cast<int>(id[u] - lo) : 0;
      for (int b = 0; b < bits; ++b) {
        const unsigned long long set = __ballot((d >> b) & 1);
        same &= (d >> b) & 1 ? set : ~set;
      }
      const int lead = __ffsll(same) - 1;
      const int before = __popcll(same & ((1ull << lane) - 1));
      int at = 0;
      if (in && lane == lead) at = atomicAdd(&hist[w][d], static_cast<int>(__popcll(same)));
      at = __shfl(at, lead < 0 ? 0 : lead, kWave) + before;
      if (in) {
        A.order[at] = static_cast<int>(t + u * kWave + lane);
        A.row[at] = static_cast<int>(id[u]);
      }
    }
  }
}

// A row's piece from its sum.
template <typename TT, int V>
__device__ __forceinline__ void put(const EmbedGradLaunch& A, int id, int c, float (&acc)[V]) {
  TT* to = static_cast<TT*>(A.dtable) + static_cast<long long>(id) * A.n + c;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] *= A.scale;
  if constexpr (sizeof(TT) == 4) {
    if (A.accumulate) {
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += to[e];
    }
  }
  store_n<TT, V>(to, acc);
}

// Borders are the multiples of `chunk` below the count.  An id whose run spans two
// borders or more is long: each chunk that it touches leaves its part.  A run that
// spans one belongs to the chunk where it starts.
struct Runs {
  const int* row;
  int count, chunk;
  __device__ __forceinline__ bool spans(int b, int id) const {   // border b inside the run of id
    return b > 0 && b < count && row[b - 1] == id && row[b] == id;
  }
  // a run that spans border b
  __device__ __forceinline__ bool long_at(int b) const {
    const int id = row[b];
    return spans(b - chunk, id) || spans(b + chunk, id);
  }
};

// The pieces of a row do not overlap here (the last one is short): part sums and
// gradients may be added to what is there.
template <typename T, typename TT, int V>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(EmbedGradLaunch A, int chunk, uint32_t pieces) {
  const long long i = block_of_grid() * kThreads + threadIdx.x;
  const int c = static_cast<int>(i / pieces), col = static_cast<int>(i - static_cast<long long>(c) * pieces) * V;
  const int count = *A.count;
  const int p0 = c * chunk;
  if (p0 >= count || static_cast<long long>(c) * chunk >= count) return;
  const Runs R{A.row, count, chunk};
  const T* dy = static_cast<const T*>(A.dy) + col;
  const int p1 = count - p0 < chunk ? count : p0 + chunk;
  int p = p0, id = A.row[p0];
  bool open = p0 > 0 && A.row[p0 - 1] == id;   // the run began before
  float* part = A.part + 2LL * c * A.n + col;
  if (open && !R.long_at(p0)) {   // the chunk before adds it up
    while (p < p1 && A.row[p] == id) ++p;
    open = false;
    if (p == p1) return;   // (a run over the whole chunk spans both its borders)
    id = A.row[p];
  }
  for (;;) {
    float acc[V], v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    while (p < p1 && A.row[p] == id) {
      load_n<T, V>(dy + static_cast<long long>(A.order[p]) * A.lddy, v);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += v[e];
      ++p;
    }
    const bool on = p == p1 && p1 < count && A.row[p1] == id;   // the run goes on
    if (open || (on && R.long_at(p1))) {
      store_n<float, V>(open ? part : part + A.n, acc);
    } else {
      if (on) {
        for (; p < count && A.row[p] == id; ++p) {
          load_n<T, V>(dy + static_cast<long long>(A.order[p]) * A.lddy, v);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] += v[e];
        }
      }
      put<TT, V>(A, id, col, acc);
    }
    if (p >= p1) return;
    id = A.row[p];
    open = false;
  }
}

// The long runs' parts: a workgroup looks for those that start in its chunks.
constexpr int kJoinThreads = 1024, kJoinWaves = kJoinThreads / kWave, kJoinChunks = 16;

template <typename TT>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(EmbedGradLaunch A, int chunk) {
  __shared__ float sums[kJoinWaves][kWave];
  const int count = *A.count;
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const Runs R{A.row, count, chunk};
  const int col = static_cast<int>(blockIdx.y) * kWave + lane;
  const long long c0 = static_cast<long long>(blockIdx.x) * kJoinChunks;
  for (int k = 0; k < kJoinChunks; ++k) {
    const long long b = (c0 + k + 1) * chunk;   // the border behind the chunk
    if (b >= count) return;
    const int p1 = static_cast<int>(b), id = A.row[p1];
    if (A.row[p1 - 1] != id || !R.long_at(p1) || R.spans(p1 - chunk, id)) continue;
    // the last border inside the run
    int lo = 1, hi = (count - 1 - p1) / chunk + 1;   // p1 + lo' chunk holds id for lo' < lo
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (A.row[p1 + mid * chunk] == id) lo = mid + 1;
      else hi = mid;
    }
    const long long c = c0 + k;
    float acc = 0.0f;
    if (col < A.n) {
      if (w == 0) acc = A.part[(2 * c + 1) * A.n + col];
      for (int j = w; j < lo; j += kJoinWaves) acc += A.part[2 * (c + 1 + j) * A.n + col];
    }
    __syncthreads();
    sums[w][lane] = acc;
    __syncthreads();
    if (w == 0 && col < A.n) {
      float v[1] = {0.0f};
      for (int j = 0; j < kJoinWaves; ++j) v[0] += sums[j][lane];
      put<TT, 1>(A, id, col, v);
    }
  }
}

template <typename T, typename TT, int V>
hipError_t sums(const EmbedGradLaunch& A, int chunk, hipStream_t st) {
  const long long chunks = (static_cast<long long>(A.tokens) + chunk - 1) / chunk;
  const uint32_t pieces = (static_cast<uint32_t>(A.n) + V - 1) / V;
  hipLaunchKernelGGL((embed_sum_kernel<T, TT, V>), grid_of((chunks * pieces + kThreads - 1) / kThreads), dim3(kThreads), 0, st, A, chunk, pieces);
  return hipGetLastError();
}

template <typename T, typename TT>
hipError_t embed_grad(const EmbedGradLaunch& A, hipStream_t st) {
  const int range = range_of(A.vocab), sorters = (A.vocab + range - 1) / range;
  int bits = 0;
  while ((1 << bits) < range) ++bits;
  const long long bytes = A.accumulate ? 0 : static_cast<long long>(A.vocab) * A.n * static_cast<long long>(sizeof(TT));
  const long long fill = (bytes + 16LL * kFillPerThread * kSortThreads - 1) / (16LL * kFillPerThread * kSortThreads);
  hipLaunchKernelGGL((embed_sort_kernel<TT>), grid_of(sorters + fill), dim3(kSortThreads), 0, st, A, range, sorters, bits, bytes);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || A.tokens == 0) return e;
  const int chunk = embed_grad_chunk(A.tokens);
  constexpr int V = Vec<T>::n;
  e = A.n % V == 0 ? sums<T, TT, V>(A, chunk, st) : sums<T, TT, 1>(A, chunk, st);
  if (e != hipSuccess) return e;
  const unsigned chunks = (A.tokens + chunk - 1) / chunk;
  hipLaunchKernelGGL((embed_join_kernel<TT>), dim3((chunks + kJoinChunks - 1) / kJoinChunks, (A.n + kWave - 1) / kWave), dim3(kJoinThreads), 0, st, A, chunk);
  return hipGetLastError();
}

}  // namespace

int embed_grad_chunk(uint32_t tokens) { return tokens > 16 * 4096 ? 32 : 16; }

hipError_t launch_embed(const EmbedLaunch& A, bool table_bf16, bool bf16, hipStream_t st) {
  if (table_bf16) return bf16 ? embed_any<bf16_t, bf16_t>(A, st) : embed_any<bf16_t, float>(A, st);
  return bf16 ? embed_any<float, bf16_t>(A, st) : embed_any<float, float>(A, st);
}
hipError_t launch_embed_grad(const EmbedGradLaunch& A, bool bf16, bool table_bf16, hipStream_t st) {
  if (bf16) return table_bf16 ? embed_grad<bf16_t, bf16_t>(A, st) : embed_grad<bf16_t, float>(A, st);
  return table_bf16 ? embed_grad<float, bf16_t>(A, st) : embed_grad<float, float>(A, st);
}

}  // namespace muon
