// Token embedding and its gradient:
//   y_t = scale table[id_t],   dtable[v] = scale sum_{t: id_t = v} dy_t,
// with zeros for ids outside the table, which take no gradient.
//
// The gradient's sums run over tokens sorted by id, in the tokens' order, so they
// need no atomics and repeat bit for bit (the sort's counters in LDS are the only
// ones, and their sums are whole numbers).  Three launches:
//   1. a workgroup for each range of ids walks all ids and places those in its range;
//      the other workgroups write the table's zeros meanwhile, which take longer;
//   2. a wave for a piece of the rows' columns and a chunk of the sorted tokens adds up
//      each id's rows; an id that spans two borders of chunks leaves a part sum in
//      each, all others are written at once;
//   3. the parts of those ids are added, in order.
// However often one id occurs, no wave adds more than two chunks.  Measured (bfloat16
// gradients, a float32 table of 50,280 rows, ids by Zipf's law): 16,384 tokens of 768
// take 21 + 13 + 6 us, bound by the zeros' 154 MB (7.2 TB/s) and the gathered rows;
// 131,071 tokens of 515 take 5 (a map of the ids' ranges) + 32 + 59 + 13 us: counting and
// placing the range of the most frequent id by one workgroup, and 240 MB of rows at odd
// addresses, sums and parts.  The forward pass of 16,384 tokens takes 10.5 us, 44 MB at
// 4.2 TB/s.
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
  return A.n >= 8 ? embed<TT, T, 8>(A, st) : A.n >= 4 ? embed<TT, T, 4>(A, st) : embed<TT, T, 1>(A, st);
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;
constexpr int kRangeBits = 9, kRange = 1 << kRangeBits;   // most ids of a workgroup
constexpr int kKept = 1792;          // tokens that a wave keeps between its two walks (112 KB of LDS)
constexpr int kFillPerThread = 8;    // 16-byte stores

// Ids of a workgroup: all walk all ids, so not more than half the compute units do, and
// the others write zeros meanwhile (16,384 tokens, table 50,280 x 768: 21 us, of which the
// zeros alone take 21; 27 with 256 workgroups).
int range_of(int vocab) {
  const int r = (vocab + 127) / 128;
  return r < 1 ? 1 : r > kRange ? kRange : r;
}

// Tokens of a wave of a workgroup that walks all: an odd number of `unit`s, so that the
// waves' places are on different channels of the L2.
__host__ __device__ __forceinline__ uint32_t wave_span(uint32_t tokens, uint32_t unit) {
  return (((tokens + kSortWaves - 1) / kSortWaves + unit - 1) / unit | 1) * unit;
}

// Many tokens: their ranges are looked up first, 16 bits a token, with counts by blocks
// of tokens, so that a workgroup looks at eight tokens a lane at once and need not count
// those below its range (131,071 tokens of 515: 5 + 32 us instead of 52; 50,000 of 768:
// 68 us in all instead of 77, but 33,000 of 128: 35 instead of 33).  A wave's list holds a
// token as its place among the wave's, above the kRangeBits of its id: no wave walks more
// than what those bits hold.
constexpr uint32_t kMapUnit = 512;            // tokens that a wave looks at at once
constexpr uint32_t kMapBlock = 2048;          // tokens of a block
constexpr int kMapRanges = 1024;              // most ranges
constexpr uint16_t kNoRange = 0xFFFF;

bool mapped(uint32_t tokens, int vocab) {
  const int range = range_of(vocab);
  return tokens > 40u << 10 && wave_span(tokens, kMapUnit) <= 1u << (32 - kRangeBits) && (vocab + range - 1) / range <= kMapRanges;
}

__global__ void __launch_bounds__(kSortThreads) embed_map_kernel(IdsOperand ids, uint32_t tokens, int vocab, int ranges, IdsOperand by_range,
                                                                 uint32_t padded, uint16_t* map, int* table) {
  __shared__ int hist[kMapRanges];
  for (int i = threadIdx.x; i < ranges; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  const uint32_t t0 = blockIdx.x * kMapBlock;
#pragma unroll
  for (uint32_t k = 0; k < kMapBlock / kSortThreads; ++k) {
    const uint32_t t = t0 + k * kSortThreads + threadIdx.x;
    const long long id = t < tokens ? id_at(ids, t) : -1;
    uint32_t r = kNoRange;
    if (id >= 0 && id < vocab) {
      r = static_cast<uint32_t>(id);   // over the ids of a range (magic 0: one)
      if (by_range.magic != 0) r = __umulhi(r, by_range.magic) >> by_range.shift;
      atomicAdd(&hist[r], 1);
    }
    if (t < padded) map[t] = static_cast<uint16_t>(r);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ranges; i += kSortThreads) table[static_cast<long long>(blockIdx.x) * ranges + i] = hist[i];
}

// What lanes of a wave wrote to LDS before is there for its other lanes.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Inclusive sums over the lanes.
__device__ __forceinline__ int lanes_prefix(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, kDppShr1, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, kDppShr2, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, kDppShr4, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, kDppShr8, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, kDppBcast15, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, kDppBcast31, 0xc, 0xf, false);
  return v;
}

// Calls f(token, id) for groups of 64 tokens in order, a token a lane (past `end` with
// id -1); `load` gives a token's id as it lies there.  Sixteen groups' loads are in flight.
__device__ __forceinline__ int narrow(int id) { return id; }
__device__ __forceinline__ int narrow(u32x2_t id) { return id[1] == 0 ? static_cast<int>(id[0]) : -1; }   // -1 past 32 bits
template <typename L, typename F>
__device__ __forceinline__ void walk(uint32_t from, uint32_t end, const L& load, const F& f) {
  constexpr uint32_t U = 16;
  const uint32_t lane = threadIdx.x & (kWave - 1);
  uint32_t t = from;
  for (; end - t >= U * kWave; t += U * kWave) {
    decltype(load(0)) id[U];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) id[u] = load(t + u * kWave + lane);
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) f(t + u * kWave + lane, narrow(id[u]));
  }
  for (; t < end; t += kWave) {
    const uint32_t at = t + lane;
    const int id = narrow(load(at < end ? at : end - 1));
    f(at, at < end ? id : -1);
  }
}
template <typename F>
__device__ __forceinline__ void walk_ids(const IdsOperand& ids, uint32_t from, uint32_t end, const F& f) {
  if (ids.magic != 0 || ids.step != 1) walk(from, end, [&](uint32_t t) { return __builtin_bit_cast(u32x2_t, id_at(ids, t)); }, f);
  else if (ids.wide) walk(from, end, [&](uint32_t t) { return static_cast<const u32x2_t*>(ids.p)[t]; }, f);
  else walk(from, end, [&](uint32_t t) { return static_cast<const int*>(ids.p)[t]; }, f);
}
// Lanes with a < b.
__device__ __forceinline__ unsigned long long lanes_below(uint32_t a, uint32_t b) { return __builtin_amdgcn_uicmp(a, b, 36); }

// Calls one(number, lanes, leader) for two of the lanes' numbers among those with `in`,
// which are most often nearly all, and returns the lanes of the others.
template <typename F>
__device__ __forceinline__ unsigned long long peel(bool in, int d, const F& one) {
  unsigned long long left = __ballot(in);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (left == 0) return 0;
    const int lead = __ffsll(left) - 1, of = __builtin_amdgcn_readlane(d, lead);
    const unsigned long long those = __ballot(in && d == of);
    one(of, those, lead);
    left &= ~those;
  }
  return left;
}
// The lanes that hold this lane's number (of kRangeBits bits): after two by peel, the
// others are told apart bit by bit.
__device__ __forceinline__ unsigned long long same_lanes(bool in, int d) {
  unsigned long long same = 0;
  const unsigned long long left = peel(in, d, [&](int of, unsigned long long those, int) { same = d == of ? those : same; });
  if (left == 0) return same;
  unsigned long long rest = left;
#pragma unroll
  for (int b = 0; b < kRangeBits; ++b) {
    const unsigned long long set = __ballot((d >> b) & 1);
    rest &= (d >> b) & 1 ? set : ~set;
  }
  return (left >> (threadIdx.x & (kWave - 1))) & 1 ? rest : same;
}

// Blocks below `sorters`: ids [b range, (b + 1) range).  The others: zeros.
template <typename TT, bool MAP>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(EmbedGradLaunch A, int range, int sorters, long long bytes) {
  __shared__ int hist[kSortWaves][kRange];
  __shared__ uint32_t kept[kSortWaves][kKept];   // (token from the wave's first) kRange + id from the range's first
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
  const int lo = static_cast<int>(blk) * range, here = A.vocab - lo < range ? A.vocab - lo : range;
  for (int i = threadIdx.x; i < kSortWaves * kRange; i += kSortThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  const uint32_t span = wave_span(A.tokens, MAP ? kMapUnit : kWave);
  const uint32_t t0 = w * span < A.tokens ? w * span : A.tokens, t1 = A.tokens - t0 < span ? A.tokens : t0 + span;
  uint32_t below = 0, found = 0;   // uniform
  // Calls f(token, in the range, id from its first) for groups of 64 of the list.
  const auto listed = [&](const auto& f) {
    wave_fence();
    for (uint32_t i = 0; i < found; i += kWave) {
      const bool in = i + lane < found;
      const uint32_t v = in ? kept[w][i + lane] : 0;
      f(t0 + (v >> kRangeBits), in, static_cast<int>(v & (kRange - 1)));
    }
  };
  // Fills the list by the map, eight tokens a lane, and calls full() when it is.
  const auto walk_map = [&](const auto& full) {
    const auto look_up = [&] {   // the listed tokens' ids
      constexpr uint32_t G = 4;
      wave_fence();
      for (uint32_t i = 0; i < found; i += G * kWave) {
        uint32_t off[G];
        int id[G];
#pragma unroll
        for (uint32_t g = 0; g < G; ++g) {
          const uint32_t k = i + g * kWave + lane;
          off[g] = kept[w][k < found ? k : i];
          id[g] = static_cast<int>(id_at(A.ids, t0 + off[g]));
        }
        wave_fence();
#pragma unroll
        for (uint32_t g = 0; g < G; ++g)
          if (i + g * kWave + lane < found) kept[w][i + g * kWave + lane] = off[g] << kRangeBits | static_cast<uint32_t>(id[g] - lo);
      }
    };
    const uint32_t mine = static_cast<uint32_t>(blk) * 0x10001u;
    const u32x4_t* map = reinterpret_cast<const u32x4_t*>(A.map + w * span);
    constexpr uint32_t U = 4;
    found = 0;
    for (uint32_t t = 0; t < t1 - t0; t += U * kMapUnit) {
      u32x4_t m[U];
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) m[u] = map[((t + u * kMapUnit < span ? t + u * kMapUnit : 0) / 8) + lane];
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) {
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t x = m[u][i] ^ mine;
          hits |= ((x & 0xFFFFu) == 0 ? 1u << (2 * i) : 0u) | (x < 0x10000u ? 2u << (2 * i) : 0u);
        }
        if (t + u * kMapUnit >= span) hits = 0;   // (uniform)
        const int n = __popc(hits), upto = lanes_prefix(n);
        uint32_t at = found + static_cast<uint32_t>(upto - n);
        for (; hits != 0; hits &= hits - 1, ++at) kept[w][at] = t + u * kMapUnit + 8 * lane + static_cast<uint32_t>(__ffs(hits) - 1);
        found += static_cast<uint32_t>(__builtin_amdgcn_readlane(upto, kWave - 1));
        if (found > kKept - kMapUnit) {
          look_up();
          full();
          found = 0;
          wave_fence();
        }
      }
    }
    look_up();
  };
  // The same of the ids themselves; the list ends where it is full.
  const uint32_t room = span <= 1u << (32 - kRangeBits) ? kKept : 0;
  const auto again = [&](const auto& f) {
    if (found <= room) {
      listed(f);
    } else {
      walk_ids(A.ids, t0, t1, [&](uint32_t t, int id) {
        const uint32_t d = static_cast<uint32_t>(id) - lo;
        const bool in = d < static_cast<uint32_t>(here);
        f(t, in, in ? static_cast<int>(d) : 0);
      });
    }
  };
  const auto count = [&](uint32_t, bool in, int d) {
    const unsigned long long left = peel(in, d, [&](int of, unsigned long long those, int lead) {
      if (lane == lead) atomicAdd(&hist[w][of], static_cast<int>(__popcll(those)));
    });
    if ((left >> lane) & 1) atomicAdd(&hist[w][d], 1);
  };
  bool whole = true;   // the list holds all of the wave's tokens
  if constexpr (MAP) {
    walk_map([&] {
      listed(count);
      whole = false;
    });
    listed(count);
    const int blocks = static_cast<int>((A.tokens + kMapBlock - 1) / kMapBlock);
    int sum = 0;
    for (int b = w; b < blocks; b += kSortWaves)
      for (int s = lane; s < static_cast<int>(blk); s += kWave) sum += A.table[static_cast<long long>(b) * sorters + s];
    below = static_cast<uint32_t>(__builtin_amdgcn_readlane(lanes_prefix(sum), kWave - 1));
  } else {
    walk_ids(A.ids, t0, t1, [&](uint32_t t, int id) {
      const uint32_t d = static_cast<uint32_t>(id) - lo;
      below += static_cast<uint32_t>(__popcll(lanes_below(static_cast<uint32_t>(id), static_cast<uint32_t>(lo))));
      const unsigned long long set = lanes_below(d, static_cast<uint32_t>(here));
      if (set == 0) return;
      const uint32_t at = found + static_cast<uint32_t>(__popcll(set & ((1ull << lane) - 1)));
      if (((set >> lane) & 1) && at < room) kept[w][at] = (t - t0) << kRangeBits | d;
      found += static_cast<uint32_t>(__popcll(set));
    });
    again(count);
  }
  if (lane == 0) waves[w] = static_cast<int>(below);
  __syncthreads();
  int base = 0;   // of the range in the sorted order
  for (int i = 0; i < kSortWaves; ++i) base += waves[i];
  __syncthreads();
  // places: by id, then by wave
  int total = 0;
  if (threadIdx.x < kRange) {
    for (int i = 0; i < kSortWaves; ++i) total += hist[i][threadIdx.x];
  }
  int incl = total;   // prefix over the ids: the first waves hold them
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
  // the tokens to their places: those of one id in the lanes' order
  const auto drop = [&](uint32_t t, bool in, int d) {
    const unsigned long long same = same_lanes(in, d);
    const int lead = in ? __ffsll(same) - 1 : 0;
    int at = 0;
    if (in && lane == lead) at = atomicAdd(&hist[w][d], static_cast<int>(__popcll(same)));
    at = __shfl(at, lead, kWave) + static_cast<int>(__popcll(same & ((1ull << lane) - 1)));
    if (in) A.sorted[at] = make_int2(static_cast<int>(t), lo + d);
  };
  if constexpr (MAP) {
    if (!whole) walk_map([&] { listed(drop); });
    listed(drop);
  } else {
    again(drop);
  }
}

// V columns of a row from their sum, of which those from `first` on are this thread's
// alone (those before are its neighbour's too, which stores the same).
template <typename TT, int V>
__device__ __forceinline__ void put(const EmbedGradLaunch& A, int id, int c, int first, float (&acc)[V]) {
  TT* to = static_cast<TT*>(A.dtable) + static_cast<long long>(id) * A.n + c;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] *= A.scale;
  if constexpr (sizeof(TT) == 4) {
    if (A.accumulate) {
      if (first > 0) {
#pragma unroll
        for (int e = 1; e < V; ++e)
          if (e >= first) to[e] += acc[e];
        return;
      }
      constexpr int W = V < 4 ? V : 4;
      float was[V / W][W];
#pragma unroll
      for (int k = 0; k < V / W; ++k) load_n<float, W>(to + k * W, was[k]);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += was[e / W][e % W];
    }
  }
  store_n<TT, V>(to, acc);
}

// Borders are the multiples of `chunk` below the count.  An id whose run spans two
// borders or more is long: each chunk that it touches leaves its part.  A run that
// spans one belongs to the chunk where it starts.
//
// A wave for 64 pieces of V columns (of a row's last ones, moved back to end with it) of
// a chunk of the sorted tokens: places and ids are uniform.  Eight tokens' rows are in
// flight, and the next eight's places.
template <typename T, typename TT, int V>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(EmbedGradLaunch A, const int2* __restrict__ sorted, const int* __restrict__ counted,
                                                             int chunk, uint32_t slices) {
  const long long i = block_of_grid() * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const long long c = i / slices;
  if (c * chunk >= A.tokens) return;
  const int col = (static_cast<int>(i - c * slices) * kWave + static_cast<int>(threadIdx.x & (kWave - 1))) * V;
  const int base = col < A.n - V ? col : A.n - V, first = col - base;
  constexpr int U = 8;
  // all that the chunk's state needs, in one go (places past the count hold anything)
  const int p0 = static_cast<int>(c) * chunk, last = static_cast<int>(A.tokens) - 1;
  const auto at = [&](int p) { return sorted[p < 0 ? 0 : p < last ? p : last]; };
  int2 s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) s[u] = at(p0 + u);
  const int before = at(p0 - 1).y, far = at(p0 - chunk - 1).y, next = at(p0 + chunk).y, next2 = at(p0 + 2 * chunk).y;
  const int count = *counted;
  if (p0 >= count) return;
  const int p1 = count - p0 < chunk ? count : p0 + chunk;
  const T* dy = static_cast<const T*>(A.dy) + base;
  float* part = A.part + 2 * c * A.n;
  int id = s[0].y;
  const int some = s[0].x;   // read in place of tokens past the count, whose rows there need not be
  // whose is the run at the start: this chunk's, the chunk's before (skip) or every chunk's that it touches (open)
  bool open = p0 > 0 && before == id, skip = false;
  if (open && !(p0 > chunk && far == id) && !(p0 + chunk < count && next == id)) {
    open = false;
    skip = true;
  }
  const bool far_on = p0 + 2 * chunk < count;
  float acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.0f;
  const auto leave = [&](bool goes_on) {   // the run ends, or goes on behind the chunk
    if (skip || first >= V) return;
    if (open || goes_on) store_n<float, V>((open ? part : part + A.n) + base, acc);
    else put<TT, V>(A, id, base, first, acc);
  };
  for (int q = p0;; q += U) {
    float v[U][V];
    int ids[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      ids[u] = s[u].y;
      load_n<T, V>(dy + static_cast<long long>(q + u < count ? s[u].x : some) * A.lddy, v[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) s[u] = at(q + U + u);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = q + u;
      const bool new_run = p >= count || ids[u] != id;
      if (new_run) leave(false);
      if (p >= p1) {
        if (new_run || skip) return;
        if (p == p1 && (open || (far_on && next2 == id))) {   // (the run spans this border)
          leave(true);
          return;
        }
      }
      if (new_run) {
        id = ids[u];
        open = skip = false;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.0f;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += v[u][e];
    }
  }
}

// The long runs' parts: the lanes look for those that start in the workgroup's chunks,
// then its waves share each one's parts (131,071 tokens of 515: 13 us, 15 with 1,024
// threads for sixteen chunks).
constexpr int kJoinThreads = 512, kJoinWaves = kJoinThreads / kWave, kJoinChunks = 4;

template <typename TT, int V>
__global__ void __launch_bounds__(kJoinThreads) embed_join_kernel(EmbedGradLaunch A, int chunk) {
  __shared__ float sums[kJoinWaves][V][kWave];
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int col = (static_cast<int>(blockIdx.z) * kWave + lane) * V;
  const int base = col < A.n - V ? col : A.n - V, first = col - base;
  const long long c0 = block_of_grid() * kJoinChunks;
  if (c0 * chunk >= A.tokens) return;
  const int last = static_cast<int>(A.tokens) - 1;
  const auto id_of = [&](long long p) { return A.sorted[p < 0 ? 0 : p < last ? p : last].y; };
  // the border behind the lane's chunk: spanned, and the one behind it, but not the one before
  const long long b0 = (c0 + (lane < kJoinChunks ? lane : 0) + 1) * chunk;
  const int mine = id_of(b0), before = id_of(b0 - 1), next = id_of(b0 + chunk), far = id_of(b0 - chunk - 1);
  const int count = *A.count;
  const bool starts = lane < kJoinChunks && b0 + chunk < count && before == mine && next == mine && !(b0 > chunk && far == mine);
  for (unsigned long long set = __ballot(starts); set != 0; set &= set - 1) {
    const int k = __ffsll(set) - 1, id = __builtin_amdgcn_readlane(mine, k);
    const long long c = c0 + k, p1 = (c + 1) * chunk;
    // borders inside the run: `parts` are, and one of the `more` after them is the first that is not
    int parts = 0, more = (count - 1 - static_cast<int>(p1)) / chunk + 2;
    while (more > 1) {
      const int step = (more + kWave - 2) / kWave;   // the lanes cover more - 1 of them
      const long long b = p1 + static_cast<long long>(parts + step * lane + step - 1) * chunk;
      const int n = static_cast<int>(__popcll(__ballot(b < count && id_of(b) == id)));
      parts += n * step;
      more = step;
    }
    float acc[V], v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.0f;
    const float* part = A.part + 2 * (c + 1) * A.n + base;
    if (w == 0) load_n<float, V>(part - A.n, acc);
#pragma unroll 16
    for (int j = w; j < parts; j += kJoinWaves) {
      load_n<float, V>(part + 2LL * j * A.n, v);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += v[e];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) sums[w][e][lane] = acc[e];
    __syncthreads();
    if (w == 0 && col < A.n) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        acc[e] = 0.0f;
        for (int j = 0; j < kJoinWaves; ++j) acc[e] += sums[j][e][lane];
      }
      put<TT, V>(A, id, base, first, acc);
    }
  }
}

// Few tokens: one launch.  A workgroup owns `range` rows of the table, looks for their
// ids among all and writes the rows, a wave each, zeros or sums over the tokens in order
// (128 tokens of 768, table of 50,280 rows: 22 us, 29 sorted; of 1,000 rows: 10 and 16,
// the host's time.  If all have one id, which a wave then adds: 36 and 30, with 256
// tokens 59 and 30).
constexpr int kFew = 128;

template <typename T, typename TT, int V>
__global__ void __launch_bounds__(kThreads) embed_few_kernel(EmbedGradLaunch A, int range) {
  __shared__ int ids[kFew];
  __shared__ int tokens[kThreads / kWave][kFew];
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const long long row0 = block_of_grid() * range;
  if (row0 >= A.vocab) return;
  {
    const long long id = threadIdx.x < A.tokens ? id_at(A.ids, threadIdx.x) : -1;
    if (threadIdx.x < kFew) ids[threadIdx.x] = id >= 0 && id < A.vocab ? static_cast<int>(id) : -1;
  }
  __syncthreads();
  const int rows = A.vocab - row0 < range ? static_cast<int>(A.vocab - row0) : range;
  for (int r = w; r < rows; r += kThreads / kWave) {
    const int id = static_cast<int>(row0) + r;
    int found = 0;
#pragma unroll
    for (int k = 0; k < kFew / kWave; ++k) {
      const bool hit = ids[k * kWave + lane] == id;
      const unsigned long long set = __ballot(hit);
      if (hit) tokens[w][found + static_cast<int>(__popcll(set & ((1ull << lane) - 1)))] = k * kWave + lane;
      found += static_cast<int>(__popcll(set));
    }
    if (found == 0) {
      if (A.accumulate) continue;
      constexpr int W = V * sizeof(TT) > 16 ? 16 / static_cast<int>(sizeof(TT)) : V;   // 16 bytes or less; a row holds V elements
      const float zero[W] = {};
      TT* to = static_cast<TT*>(A.dtable) + static_cast<long long>(id) * A.n;
      for (int c = lane * W; c < A.n; c += kWave * W) store_n<TT, W>(to + (c < A.n - W ? c : A.n - W), zero);
      continue;
    }
    wave_fence();   // the list is read by the wave's other lanes
    for (int c = lane * V; c < A.n; c += kWave * V) {
      const int base = c < A.n - V ? c : A.n - V;
      const T* dy = static_cast<const T*>(A.dy) + base;
      constexpr int U = 8;   // loads in flight
      float acc[V], v[U][V];
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = 0.0f;
      for (int i = 0; i < found; i += U) {
#pragma unroll
        for (int u = 0; u < U; ++u) load_n<T, V>(dy + static_cast<long long>(tokens[w][i + u < found ? i + u : i]) * A.lddy, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] += i + u < found ? v[u][e] : 0.0f;
      }
      put<TT, V>(A, id, base, c - base, acc);
    }
    wave_fence();
  }
}

template <typename T, typename TT, int V>
hipError_t few(const EmbedGradLaunch& A, hipStream_t st) {
  const int range = static_cast<int>((static_cast<long long>(A.vocab) + 4095) / 4096);   // sixteen workgroups a compute unit
  hipLaunchKernelGGL((embed_few_kernel<T, TT, V>), grid_of((static_cast<long long>(A.vocab) + range - 1) / range), dim3(kThreads), 0, st, A, range);
  return hipGetLastError();
}

template <typename T, typename TT, int V>
hipError_t sums(const EmbedGradLaunch& A, int chunk, hipStream_t st) {
  const long long chunks = (static_cast<long long>(A.tokens) + chunk - 1) / chunk;
  const uint32_t pieces = (static_cast<uint32_t>(A.n) + V - 1) / V;
  const uint32_t slices = (pieces + kWave - 1) / kWave;
  hipLaunchKernelGGL((embed_sum_kernel<T, TT, V>), grid_of((chunks * slices + kThreads / kWave - 1) / (kThreads / kWave)), dim3(kThreads), 0, st, A,
                     A.sorted, A.count, chunk, slices);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || chunks < 3) return e;   // no run spans two borders
  constexpr int W = V < 4 ? V : 4;
  dim3 grid = grid_of((chunks + kJoinChunks - 1) / kJoinChunks);
  grid.z = (A.n + kWave * W - 1) / (kWave * W);   // 2^13 at most
  hipLaunchKernelGGL((embed_join_kernel<TT, W>), grid, dim3(kJoinThreads), 0, st, A, chunk);
  return hipGetLastError();
}

template <typename T, typename TT>
hipError_t embed_grad(const EmbedGradLaunch& A, hipStream_t st) {
  constexpr int V = Vec<T>::n;
  if (A.tokens <= kFew) return A.n >= V ? few<T, TT, V>(A, st) : few<T, TT, 1>(A, st);
  const int range = range_of(A.vocab), sorters = (A.vocab + range - 1) / range;
  const long long bytes = A.accumulate ? 0 : static_cast<long long>(A.vocab) * A.n * static_cast<long long>(sizeof(TT));
  const long long fill = (bytes + 16LL * kFillPerThread * kSortThreads - 1) / (16LL * kFillPerThread * kSortThreads);
  const dim3 grid = grid_of(sorters + fill), block(kSortThreads);
  hipError_t e;
  if (mapped(A.tokens, A.vocab)) {
    const uint32_t padded = kSortWaves * wave_span(A.tokens, kMapUnit);
    hipLaunchKernelGGL(embed_map_kernel, dim3((padded + kMapBlock - 1) / kMapBlock), block, 0, st, A.ids, A.tokens, A.vocab, sorters,
                       A.by_range, padded, A.map, A.table);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((embed_sort_kernel<TT, true>), grid, block, 0, st, A, range, sorters, bytes);
  } else {
    hipLaunchKernelGGL((embed_sort_kernel<TT, false>), grid, block, 0, st, A, range, sorters, bytes);
  }
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int chunk = embed_grad_chunk(A.tokens);
  return A.n >= V ? sums<T, TT, V>(A, chunk, st) : sums<T, TT, 1>(A, chunk, st);
}

}  // namespace

EmbedMapSizes embed_map_sizes(uint32_t tokens, int vocab) {
  if (!mapped(tokens, vocab)) return {0, 0, 1};
  const int range = range_of(vocab);
  const size_t padded = static_cast<size_t>(kSortWaves) * wave_span(tokens, kMapUnit), ranges = (vocab + range - 1) / range;
  return {padded * sizeof(uint16_t), (padded + kMapBlock - 1) / kMapBlock * ranges * sizeof(int), range};
}

// Sorted tokens of a chunk: 16,384 tokens of 768 take 13 + 6 us (sums and joins) in
// chunks of 16, 13 + 8 of 8 and 16 + 5 of 32; 131,071 of 515 take 59 + 13 of 32,
// 61 + 23 of 16 and 71 + 40 of 8.
int embed_grad_chunk(uint32_t tokens) { return tokens > 1u << 16 ? 32 : 16; }

hipError_t launch_embed(const EmbedLaunch& A, bool table_bf16, bool bf16, hipStream_t st) {
  if (table_bf16) return bf16 ? embed_any<bf16_t, bf16_t>(A, st) : embed_any<bf16_t, float>(A, st);
  return bf16 ? embed_any<float, bf16_t>(A, st) : embed_any<float, float>(A, st);
}
hipError_t launch_embed_grad(const EmbedGradLaunch& A, bool bf16, bool table_bf16, hipStream_t st) {
  if (bf16) return table_bf16 ? embed_grad<bf16_t, bf16_t>(A, st) : embed_grad<bf16_t, float>(A, st);
  return table_bf16 ? embed_grad<float, bf16_t>(A, st) : embed_grad<float, float>(A, st);
}

}  // namespace muon
