// The gated scan: for every sequence and head
//   S_t = e^{g_t} S_{t-1} + b_t v_t k_t^T   (P x N),   y_t = S_t q_t.
// With c the inclusive sums of g inside a chunk of kQ tokens that starts from
// S_in, the chunk is
//   y_i   = sum_{j <= i} e^{c_i - c_j} b_j (q_i . k_j) v_j + e^{c_i} S_in q_i
//   S_out = e^{c_end} S_in + sum_j e^{c_end - c_j} b_j v_j k_j^T,
// matrix products all.  One workgroup walks the chunks of a sequence, head and
// block of kPB state rows with the state in its registers (float32, so it
// crosses HBM only at the ends): each of its four waves holds 16 rows of S.
// Held as S^T with n along the accumulator rows, the state is the operand of
// S_in q without leaving the registers.
//
// Rounding, bfloat16 operands: the weights e^{c_i - c_j} b_j (q_i . k_j) and
// the copy of S_in that is read are rounded to bfloat16 once, which leaves y
// within its own rounding; the weighted values that enter the state are split
// into three bfloat16 pieces, so the state keeps float32 accuracy.
//
// In reversed time the same walk with (dy, q) for (v, k), weights e^{c_i} and
// no reads gives the gradients of the states (muon_gated_scan_backward).
#include "scan_tiles.cuh"

namespace muon {
namespace {

using namespace scan;

constexpr int kWalkThreads = 512;
constexpr int kStepThreads = 256;

template <typename T, int NT>
struct WalkLds {
  static constexpr int kLdN = NT + Ops<T>::kPad;
  static constexpr int kLdP = kPB + Ops<T>::kPad;
  static constexpr int kLdM = kQ + Ops<T>::kPad;
  static constexpr int k = 0;                                   // k [kQ][NT]
  static constexpr int x = k + kQ * kLdN * (int)sizeof(T);      // x [kQ][kPB]
  static constexpr int gates = x + kQ * kLdP * (int)sizeof(T);  // Gates[2]
  static constexpr int states_bytes = gates + 2 * (int)sizeof(Gates<kQ>);
  static constexpr int q = states_bytes;                        // q [kQ][NT]
  static constexpr int m = q + kQ * kLdN * (int)sizeof(T);      // weights M [i][j]
  static constexpr int y = m + kQ * kLdM * (int)sizeof(T);      // halves of y that waves hand over [8][2][64] float4
  static constexpr int read_bytes = y + 8 * 2 * 64 * 16;
};

struct WalkPair {
  ScanWalk w[2];
};

// READ: y is computed (q is read); else only states move.
//
// Wave w holds rows p = 16 (w % 4) + 0..15 of S and columns n of half w / 4:
// the tokens' products with the halves are partial sums of y, which the two
// waves of the same rows exchange through LDS, each finishing half of the
// tokens.  Eight waves a workgroup rather than four (160 -> ... us).
template <typename T, int NT, bool READ, bool VEC>
__global__ void __launch_bounds__(kWalkThreads, sizeof(T) == 2 ? 4 : 2) scan_walk_kernel(WalkPair W) {
  typedef Ops<T> O;
  typedef typename O::Frag Frag;
  typedef WalkLds<T, NT> L;
  constexpr int kT = NT / 32;       // state tiles of a wave
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const ScanWalk A = W.w[blockIdx.y];
  T* lk = reinterpret_cast<T*>(lds + L::k);
  T* lx = reinterpret_cast<T*>(lds + L::x);
  T* lq = reinterpret_cast<T*>(lds + L::q);
  T* lm = reinterpret_cast<T*>(lds + L::m);
  f32x4_t* ly = reinterpret_cast<f32x4_t*>(lds + L::y);
  Gates<kQ>* gates = reinterpret_cast<Gates<kQ>*>(lds + L::gates);

  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, g4 = lane >> 4;
  const int pw = w & 3, nh = w >> 2, nbase = nh * (NT / 2);
  const int vheads = A.heads * A.pblocks;
  const int seg = static_cast<int>(blockIdx.x) % A.nseg;
  const int vh = static_cast<int>(blockIdx.x) / A.nseg % vheads;
  const long long bi = static_cast<int>(blockIdx.x) / A.nseg / vheads;
  const int h = vh / A.pblocks, pb = vh - h * A.pblocks, grp = h / (A.heads / A.groups);
  const int rows_p = A.P - pb * kPB < kPB ? A.P - pb * kPB : kPB;
  if (A.totals && seg + 1 == A.nseg) return;   // nothing starts after the last segment
  const long long vrow = bi * vheads + vh;
  const bool reverse = A.reverse != 0;
  const int cc0 = seg * A.seg_chunks;
  const int cc1 = cc0 + A.seg_chunks < A.nchunks ? cc0 + A.seg_chunks : A.nchunks;

  const int N = A.N, last_chunk = A.nchunks - 1;
  const long long tokens = A.tokens, xst = A.x.st, kst = A.k.st, qst = A.q.st, gst = A.g.st, bst = A.b.st;
  const T* xp = static_cast<const T*>(A.x.p) + bi * A.x.sb + h * A.x.sh + pb * kPB;
  const T* kp = static_cast<const T*>(A.k.p) + bi * A.k.sb + grp * A.k.sh;
  const T* qp = READ ? static_cast<const T*>(A.q.p) + bi * A.q.sb + grp * A.q.sh : nullptr;
  const float* gp = static_cast<const float*>(A.g.p) + bi * A.g.sb + h * A.g.sh;
  const float* bp = A.b.p == nullptr ? nullptr : static_cast<const float*>(A.b.p) + bi * A.b.sb + h * A.b.sh;
  T* yp = READ ? static_cast<T*>(A.y) + (bi * tokens * A.heads + h) * A.P + pb * kPB : nullptr;
  const long long yst = static_cast<long long>(A.heads) * A.P;

  const auto chunk_of = [&](int cc) { return reverse ? last_chunk - cc : cc; };
  const auto rows_of = [&](int chunk) {
    const long long left = tokens - static_cast<long long>(chunk) * kQ;
    return left < kQ ? static_cast<int>(left) : kQ;
  };
  // gates of the cc-th chunk visited, a token a lane (past the end: no decay, no input)
  float gv[1] = {0.0f}, bv[1] = {0.0f};
  const auto load_gates = [&](int cc) {
    const int chunk = chunk_of(cc), rows = rows_of(chunk);
    const long long t = static_cast<long long>(chunk) * kQ + (lane < rows ? lane : rows - 1);
    gv[0] = gp[t * gst];
    bv[0] = bp == nullptr ? 1.0f : bp[t * bst];
    if (lane >= rows) gv[0] = bv[0] = 0.0f;
  };

  TileLoad<T, NT, kQ, kWalkThreads, VEC> tk, tq;
  TileLoad<T, kPB, kQ, kWalkThreads, VEC> tx;
  // (past the last chunk nothing is read: a branch around the prefetch would keep two copies of its registers)
  const auto load_tiles = [&](int cc) {
    const int chunk = chunk_of(cc < cc1 ? cc : cc0), rows = cc < cc1 ? rows_of(chunk) : 0;
    const long long t0 = static_cast<long long>(chunk) * kQ;
    tk.load(kp + t0 * kst, kst, rows, N, tid);
    tx.load(xp + t0 * xst, xst, rows, rows_p, tid);
    if constexpr (READ) tq.load(qp + t0 * qst, qst, rows, N, tid);
  };

  // the state: tile t holds S^T rows n = nbase + 16 t + 4 g4 + 0..3, column p = 16 pw + l16
  f32x4_t st[kT];
  const int prow = pb * kPB + 16 * pw + l16, tile_off = (16 * pw + l16) * NT + nbase + 4 * g4;
  if (A.seg_state != nullptr && !A.totals) {
    const float* sp = A.seg_state + (vrow * A.nseg + seg) * (kPB * NT) + tile_off;
#pragma unroll
    for (int t = 0; t < kT; ++t) st[t] = *reinterpret_cast<const f32x4_t*>(sp + 16 * t);
  } else {
    const bool init = A.init != nullptr && !A.totals;
    const float* sp = A.init + ((bi * A.heads + h) * A.P + prow) * static_cast<long long>(N);
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = nbase + 16 * t + 4 * g4 + r;
        st[t][r] = init && prow < A.P && n < N ? sp[n] : 0.0f;
      }
  }

  if constexpr (READ) {
    // tiles (0, 1) and (2, 3) of M lie above the diagonal inside the 32-wide
    // steps that are multiplied: zero for good
    if (w < 2) {
      const int r0 = 32 * w, c0 = 32 * w + 16;
#pragma unroll
      for (int e = 0; e < 4; ++e) lm[(r0 + l16) * L::kLdM + c0 + 4 * g4 + e] = O::from_f32(0.0f);
    }
  }
  float* states = A.states == nullptr ? nullptr : A.states + vrow * A.nblocks * (kPB * NT);
  const int keep = A.keep;
  double seg_log = 0.0;
  load_tiles(cc0);
  if (w == 7) {
    load_gates(cc0);
    seg_log += write_gates(gates[cc0 & 1], gv, bv, lane, reverse);
    if (cc0 + 1 < cc1) load_gates(cc0 + 1);
  }
  for (int cc = cc0; cc < cc1; ++cc) {
    __syncthreads();   // the last chunk's tiles are done with
    tk.store(lk, tid);
    tx.store(lx, tid);
    if constexpr (READ) tq.store(lq, tid);
    __syncthreads();
    const Gates<kQ>& G = gates[cc & 1];
    load_tiles(cc + 1);
    const int chunk = chunk_of(cc);

    f32x4_t y[4];   // y^T: rows p = 16 pw + 4 g4 + 0..3, column i = 16 it + l16
    if constexpr (READ) {
      // M^T tiles: rows j, columns i, so a lane's four values are neighbours in M
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int e = w + 8 * u;
        if (e < 10) {
          const int it = tile_row(e), jt = tile_col(e, it);
          f32x4_t a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int s = 0; s < NT / 32; ++s)
            a = O::mma(O::row(lk + (16 * jt + l16) * L::kLdN + 32 * s + 8 * g4),
                       O::row(lq + (16 * it + l16) * L::kLdN + 32 * s + 8 * g4), a);
          const int i = 16 * it + l16, j0 = 16 * jt + 4 * g4;
          const float hi = G.hi[i], lo = G.lo[i];
          const f32x4_t jh = *reinterpret_cast<const f32x4_t*>(G.hi + j0), jl = *reinterpret_cast<const f32x4_t*>(G.lo + j0);
          const f32x4_t jb = *reinterpret_cast<const f32x4_t*>(G.b + j0);
#pragma unroll
          for (int r = 0; r < 4; ++r) a[r] = j0 + r <= i ? a[r] * between(hi, lo, jh[r], jl[r]) * jb[r] : 0.0f;
          O::store4(lm + i * L::kLdM + j0, a);
        }
      }
      // what this half of S_in gives: S_in q_i
#pragma unroll
      for (int it = 0; it < 4; ++it) y[it] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < kT / 2; ++s) {
        const Frag f = frag_from_acc<T>(st[2 * s], st[2 * s + 1]);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const T* qr = lq + (16 * it + l16) * L::kLdN + nbase + 32 * s + 4 * g4;
          y[it] = O::mma(f, O::row2(qr, qr + 16), y[it]);
        }
      }
      // token tiles 2 nh and 2 nh + 1 stay, the others go to the other half's wave
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        ly[(w * 2 + u) * 64 + lane] = nh == 0 ? y[2 + u] : y[u];
        y[u] = nh == 0 ? y[u] : y[2 + u];
      }
    } else {
      // the state that a block of `keep` chunks starts from (in reversed time: ends with)
      if (states != nullptr && (reverse ? chunk % keep == keep - 1 || chunk == last_chunk : chunk % keep == 0)) {
        float* sp = states + static_cast<long long>(chunk / keep) * (kPB * NT) + state_offset(nbase + 4 * g4, 16 * pw + l16);
#pragma unroll
        for (int t = 0; t < kT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) sp[t * (kPB / 32) * 512 + r * 8] = st[t][r];
      }
    }
    if (w == 7 && cc + 1 < cc1) {
      seg_log += write_gates(gates[(cc + 1) & 1], gv, bv, lane, reverse);
      if (cc + 2 < cc1) load_gates(cc + 2);
    }

    // the chunk's own part of the state
    const float end = G.end[0];
#pragma unroll
    for (int t = 0; t < kT; ++t) st[t] *= end;
#pragma unroll
    for (int s = 0; s < kQ / 32; ++s) {
      float xv[8], wv[8];
      O::widen(O::col(lx, L::kLdP, 32 * s, 16 * pw, lane), xv);
      load8(G.in + 32 * s + 8 * g4, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) xv[e] *= wv[e];
      Frag f[O::kSplit], kf[kT];
      O::split(xv, f);
#pragma unroll
      for (int t = 0; t < kT; ++t) kf[t] = O::col(lk, L::kLdN, 32 * s, nbase + 16 * t, lane);
#pragma unroll
      for (int u = O::kSplit - 1; u >= 0; --u)
#pragma unroll
        for (int t = 0; t < kT; ++t) st[t] = O::mma(kf[t], f[u], st[t]);
    }

    if constexpr (READ) {
      __syncthreads();   // M and the halves of y are written
#pragma unroll
      for (int u = 0; u < 2; ++u) y[u] = (y[u] + ly[((w ^ 4) * 2 + u) * 64 + lane]) * G.first[32 * nh + 16 * u + l16];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s <= nh) {
          const Frag vf = O::col(lx, L::kLdP, 32 * s, 16 * pw, lane);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            y[u] = O::mma(vf, O::row(lm + (32 * nh + 16 * u + l16) * L::kLdM + 32 * s + 8 * g4), y[u]);
        }
      const TileStore<T, VEC> out(yp + static_cast<long long>(chunk) * kQ * yst, yst, rows_of(chunk), rows_p);
#pragma unroll
      for (int u = 0; u < 2; ++u) out.put(32 * nh + 16 * u + l16, 16 * pw + 4 * g4, y[u]);
    }
  }

  if (A.totals) {
    float* sp = A.seg_state + (vrow * A.nseg + seg) * (kPB * NT) + tile_off;
#pragma unroll
    for (int t = 0; t < kT; ++t) *reinterpret_cast<f32x4_t*>(sp + 16 * t) = st[t];
    if (w == 7 && lane == 0) A.seg_decay[vrow * A.nseg + seg] = __builtin_amdgcn_exp2f(static_cast<float>(seg_log));
  } else if (A.fin != nullptr && cc1 == A.nchunks) {
    float* sp = A.fin + ((bi * A.heads + h) * A.P + prow) * static_cast<long long>(N);
#pragma unroll
    for (int t = 0; t < kT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int n = nbase + 16 * t + 4 * g4 + r;
        if (prow < A.P && n < N) sp[n] = st[t][r];
      }
  }
}

// The state that each segment starts from, out of the segments' own totals
// (in place: a total is read before its slot is overwritten).
__global__ void __launch_bounds__(kStepThreads) scan_segments_kernel(WalkPair W, int nt) {
  const ScanWalk& A = W.w[blockIdx.z];
  const int e = static_cast<int>(blockIdx.y) * kStepThreads + static_cast<int>(threadIdx.x);   // of kPB * nt
  const long long vrow = blockIdx.x;
  const int vheads = A.heads * A.pblocks;
  const int vh = static_cast<int>(vrow % vheads);
  const long long bi = vrow / vheads;
  const int h = vh / A.pblocks, p = (vh - h * A.pblocks) * kPB + e / nt, n = e % nt;
  float cur = A.init != nullptr && p < A.P && n < A.N ? A.init[((bi * A.heads + h) * A.P + p) * static_cast<long long>(A.N) + n]
                                                      : 0.0f;
  float* sp = A.seg_state + vrow * A.nseg * kPB * nt + e;
  const float* dp = A.seg_decay + vrow * A.nseg;
  for (int s = 0; s + 1 < A.nseg; ++s) {
    const float own = sp[static_cast<long long>(s) * kPB * nt];
    sp[static_cast<long long>(s) * kPB * nt] = cur;
    cur = fmaf(dp[s], cur, own);
  }
  sp[static_cast<long long>(A.nseg - 1) * kPB * nt] = cur;
}

template <typename T, int NT, bool READ, bool VEC>
hipError_t walk(const WalkPair& W, int dirs, hipStream_t st) {
  const ScanWalk& a = W.w[0];
  constexpr int bytes = READ ? WalkLds<T, NT>::read_bytes : WalkLds<T, NT>::states_bytes;
  const void* fn = reinterpret_cast<const void*>(scan_walk_kernel<T, NT, READ, VEC>);
  const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  const long long items = static_cast<long long>(a.batch) * a.heads * a.pblocks * a.nseg;
  hipLaunchKernelGGL((scan_walk_kernel<T, NT, READ, VEC>), dim3(static_cast<unsigned>(items), dirs), dim3(kWalkThreads), bytes, st,
                     W);
  return hipGetLastError();
}

template <typename T, int NT>
hipError_t walk_any(const WalkPair& W, int dirs, bool read, bool vec, hipStream_t st) {
  if (read) return vec ? walk<T, NT, true, true>(W, dirs, st) : walk<T, NT, true, false>(W, dirs, st);
  return vec ? walk<T, NT, false, true>(W, dirs, st) : walk<T, NT, false, false>(W, dirs, st);
}
hipError_t walk_any(const WalkPair& W, int dirs, bool read, bool vec, bool bf16, hipStream_t st) {
  if (W.w[0].N <= 64) return bf16 ? walk_any<bf16_t, 64>(W, dirs, read, vec, st) : walk_any<float, 64>(W, dirs, read, vec, st);
  return bf16 ? walk_any<bf16_t, 128>(W, dirs, read, vec, st) : walk_any<float, 128>(W, dirs, read, vec, st);
}

}  // namespace

hipError_t launch_scan_walk(const ScanWalk* walks, int dirs, bool read, bool vec, bool bf16, hipStream_t st) {
  WalkPair W{{walks[0], walks[dirs - 1]}};
  const ScanWalk& a = walks[0];
  if (a.nseg > 1) {
    WalkPair S = W;
    for (ScanWalk& x : S.w) {
      x.totals = 1;
      x.states = nullptr;
    }
    hipError_t e = walk_any(S, dirs, false, vec, bf16, st);
    if (e != hipSuccess) return e;
    const int nt = scan_padded_n(a.N);
    const long long vrows = static_cast<long long>(a.batch) * a.heads * a.pblocks;
    hipLaunchKernelGGL(scan_segments_kernel, dim3(static_cast<unsigned>(vrows), kScanRows * nt / kStepThreads, dirs),
                       dim3(kStepThreads), 0, st, W, nt);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return walk_any(W, dirs, read, vec, bf16, st);
}

// ---------------------------------------------------------------------------
// one token: S' = e^g S + b v k^T, y = S' q.  Reads and writes the state once;
// a half-wave holds a row's N <= 128 elements, 4 consecutive ones a lane.
// ---------------------------------------------------------------------------
namespace {

constexpr int kStepRows = 16;   // state rows per workgroup: 8 half-waves, 2 rows each

template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<bf16_t>(const bf16_t* p) { return bf16_to_f32(*p); }
template <>
__device__ __forceinline__ float load1<float>(const float* p) { return *p; }

template <typename T>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(ScanStep A) {
  const int half = threadIdx.x >> 5, l = threadIdx.x & 31, n0 = 4 * l;
  const int pblocks = (A.P + kStepRows - 1) / kStepRows;
  const int pb = static_cast<int>(blockIdx.x) % pblocks;
  const long long bh = blockIdx.x / pblocks;
  const int h = static_cast<int>(bh % A.heads), grp = h / (A.heads / A.groups);
  const long long bi = bh / A.heads;
  const T* vp = static_cast<const T*>(A.v.p) + bi * A.v.sb + h * A.v.sh;
  const T* kp = static_cast<const T*>(A.k.p) + bi * A.k.sb + grp * A.k.sh;
  const T* qp = static_cast<const T*>(A.q.p) + bi * A.q.sb + grp * A.q.sh;
  const bool vec = A.N % 4 == 0;   // rows of the state stay 16-byte aligned
  f32x4_t s[2];
  bool live[2];
  const float* sp[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int p = pb * kStepRows + 8 * u + half;
    live[u] = p < A.P;
    sp[u] = A.S + (bh * A.P + p) * A.N + n0;
    s[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (live[u] && n0 < A.N) {
      if (vec) {
        s[u] = *reinterpret_cast<const f32x4_t*>(sp[u]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n0 + r < A.N) s[u][r] = sp[u][r];
      }
    }
  }
  f32x4_t k, q;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    k[r] = n0 + r < A.N ? load1<T>(kp + n0 + r) : 0.0f;
    q[r] = n0 + r < A.N ? load1<T>(qp + n0 + r) : 0.0f;
  }
  const float decay = expf(static_cast<const float*>(A.g.p)[bi * A.g.sb + h * A.g.sh]);
  const float gate = A.b.p == nullptr ? 1.0f : static_cast<const float*>(A.b.p)[bi * A.b.sb + h * A.b.sh];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int p = pb * kStepRows + 8 * u + half;
    const float v = live[u] ? gate * load1<T>(vp + p) : 0.0f;
    float y = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[u][r] = fmaf(decay, s[u][r], v * k[r]);
      y = fmaf(s[u][r], q[r], y);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) y += __shfl_xor(y, off, kWave);
    if (!live[u]) continue;
    float* op = A.S_out + (bh * A.P + p) * A.N + n0;
    if (n0 < A.N) {
      if (vec) {
        *reinterpret_cast<f32x4_t*>(op) = s[u];
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n0 + r < A.N) op[r] = s[u][r];
      }
    }
    if (l == 0) static_cast<T*>(A.y)[bh * A.P + p] = Ops<T>::from_f32(y);
  }
}

}  // namespace

hipError_t launch_scan_step(const ScanStep& A, bool bf16, hipStream_t st) {
  const long long blocks = static_cast<long long>(A.batch) * A.heads * ((A.P + kStepRows - 1) / kStepRows);
  if (bf16) hipLaunchKernelGGL(scan_step_kernel<bf16_t>, dim3(static_cast<unsigned>(blocks)), dim3(kStepThreads), 0, st, A);
  else hipLaunchKernelGGL(scan_step_kernel<float>, dim3(static_cast<unsigned>(blocks)), dim3(kStepThreads), 0, st, A);
  return hipGetLastError();
}

namespace {
__global__ void __launch_bounds__(kStepThreads) scan_copy_kernel(const float* src, float* dst, long long n) {
  for (long long i = static_cast<long long>(blockIdx.x) * kStepThreads + threadIdx.x; i < n; i += static_cast<long long>(gridDim.x) * kStepThreads)
    dst[i] = src == nullptr ? 0.0f : src[i];
}
}  // namespace

hipError_t launch_copy_f32(const float* src, float* dst, long long n, hipStream_t st) {
  const long long blocks = (n + kStepThreads - 1) / kStepThreads;
  hipLaunchKernelGGL(scan_copy_kernel, dim3(static_cast<unsigned>(blocks < 2048 ? blocks : 2048)), dim3(kStepThreads), 0, st, src, dst, n);
  return hipGetLastError();
}

}  // namespace muon
