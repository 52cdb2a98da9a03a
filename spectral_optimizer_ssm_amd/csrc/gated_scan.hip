// The gated scan: for every sequence and head
//   S_t = e^{g_t} S_{t-1} + b_t v_t k_t^T   (P x N),   y_t = S_t q_t.
// With c the inclusive sums of g inside a chunk of kQ tokens that starts from
// S_in, the chunk is
//   y_i   = sum_{j <= i} e^{c_i - c_j} b_j (q_i . k_j) v_j + e^{c_i} S_in q_i
//   S_out = e^{c_end} S_in + sum_j e^{c_end - c_j} b_j v_j k_j^T,
// matrix products all.  One workgroup walks the chunks of a sequence, head and
// block of kPB state rows with the state in its registers (float32, so it
// crosses HBM only at the ends): eight waves, each with 16 rows of S and half
// of its columns.  Held as S^T with n along the accumulator rows, the state is
// the operand of S_in q without leaving the registers.
//
// Rounding, bfloat16 operands: the weights e^{c_i - c_j} b_j (q_i . k_j) and
// the copy of S_in that is read are two bfloat16 pieces (16 bits), so that y is
// off by its own rounding alone, at any length and from a sequence's first token
// on; in one piece y would be off by 1.4 times that, and by 2.2 times where a row
// sums few tokens, and eight sequences of 2,048 tokens would take 92 us for 103.  The weighted values that enter the state are three pieces, so the state
// keeps float32 accuracy.  Gates are float64 sums, kept as two floats.
//
// In reversed time the same walk with (dy, q) for (v, k), weights e^{c_i} and
// no reads gives the gradients of the states (muon_gated_scan_backward).
#include <climits>

#include "scan_tiles.cuh"

namespace muon {
namespace {

using namespace scan;

// Waves that multiply, and one more that prepares the gates of the next chunk
// while they do (not in the float32 forward walk).
constexpr int kReadWaves = 8, kStatesWaves = 4;
constexpr int kReadThreads = kReadWaves * kWave, kStatesThreads = kStatesWaves * kWave;
constexpr int kStateCols = 64;   // columns n of S per workgroup of the states' walk
constexpr int kStepThreads = kScanStepThreads;

struct WalkPair {
  ScanWalk w[2];
};

// The gates of a chunk on their way into LDS: a token a lane, past the end no
// decay and no input.
struct GateLoad {
  float g[1], b[1];
  template <typename W>
  __device__ __forceinline__ void load(const W& w, int cc) {
    const ScanWalk& A = w.A;
    const float* gp = static_cast<const float*>(A.g.p) + w.bi * A.g.sb + w.h * A.g.sh;
    const float* bp = A.b.p == nullptr ? nullptr : static_cast<const float*>(A.b.p) + w.bi * A.b.sb + w.h * A.b.sh;
    const int rows = w.rows_of(cc);
    const long long t = w.token_of(cc) + (w.lane < rows ? w.lane : 0);
    g[0] = gp[t * A.g.st];
    b[0] = bp == nullptr ? 1.0f : bp[t * A.b.st];
    if (w.lane >= rows) g[0] = b[0] = 0.0f;
  }
};

// One sequence (segment), head and block of kPB state rows.  A wave holds rows
// p = 16 pw + 0..15 of S and KT 16-column tiles from column nbase: of S^T where
// it reads (READ), where the tiles are operands; of S where it stores states,
// whose neighbours p then lie in one lane.
template <typename T, int NT, int KT, bool READ>
struct Walk {
  typedef Ops<T> O;
  typedef typename O::Frag Frag;

  const ScanWalk& A;
  int tid, lane, w, l16, g4, pw, nbase;
  int seg, h, pb, grp, rows_p, cc0, cc1, last_chunk, tail;   // tail: tokens of the last chunk
  long long bi, vrow;
  bool reverse;
  f32x4_t st[KT];

  __device__ __forceinline__ Walk(const ScanWalk& A, int item) : A(A) {
    tid = threadIdx.x;
    lane = tid & 63;
    w = __builtin_amdgcn_readfirstlane(tid >> 6);
    l16 = lane & 15;
    g4 = lane >> 4;
    pw = w & 3;
    nbase = 0;
    const int vheads = A.heads * A.pblocks;
    // the heads that share keys are neighbours, for every segment
    const int vh = item % vheads;
    seg = item / vheads % A.nseg;
    bi = item / vheads / A.nseg;
    h = vh / A.pblocks;
    pb = vh - h * A.pblocks;
    grp = h / (A.heads / A.groups);
    rows_p = A.P - pb * kPB < kPB ? A.P - pb * kPB : kPB;
    vrow = bi * vheads + vh;
    reverse = A.reverse != 0;
    last_chunk = A.nchunks - 1;
    tail = static_cast<int>(A.tokens - static_cast<long long>(last_chunk) * kQ);
    cc0 = seg * A.seg_chunks;
    cc1 = cc0 + A.seg_chunks < A.nchunks ? cc0 + A.seg_chunks : A.nchunks;
  }
  // the cc-th chunk visited, and its tokens (none past the segment: a branch
  // around a prefetch would keep two copies of its registers)
  __device__ __forceinline__ int chunk_of(int cc) const { return reverse ? last_chunk - cc : cc; }
  __device__ __forceinline__ int rows_of(int cc) const { return cc >= cc1 ? 0 : chunk_of(cc) == last_chunk ? tail : kQ; }
  __device__ __forceinline__ long long token_of(int cc) const { return static_cast<long long>(chunk_of(cc < cc1 ? cc : cc0)) * kQ; }
  // elements from a chunk to the next one visited, of rows `st` apart
  __device__ __forceinline__ long long step(long long st) const { return (reverse ? -kQ : kQ) * st; }
  // Columns from n on, or tokens from t of a chunk with `rows`, are padding:
  // float32 products, which their matrix instructions bound, leave it out (77
  // tokens, 12 heads, N = 72: 24 -> 19 us).
  __device__ __forceinline__ bool padding(int n) const { return sizeof(T) == 4 && n >= A.N; }
  static __device__ __forceinline__ bool ended(int t, int rows) { return sizeof(T) == 4 && t >= rows; }
  // element r of tile t
  __device__ __forceinline__ int n_of(int t, int r) const { return nbase + (READ ? state_row(t, 4 * g4) + r : 16 * t + l16); }
  __device__ __forceinline__ int p_of(int r) const { return 16 * pw + (READ ? l16 : 4 * g4 + r); }

  // The gate wave's part: gates of every chunk, one ahead of the others, who
  // meet it at two barriers a chunk (the gates are needed after the second).
  __device__ __forceinline__ void gate_wave(Gates<kQ>* gates) const {
    GateLoad gl;
    gl.load(*this, cc0);
    double log = write_gates(gates[0], gl.g, gl.b, lane, reverse);
    gl.load(*this, cc0 + 1);
    for (int cc = cc0; cc < cc1; ++cc) {
      __syncthreads();
      __syncthreads();
      log += write_gates(gates[(cc - cc0 + 1) & 1], gl.g, gl.b, lane, reverse);   // past the segment: 0
      gl.load(*this, cc + 2);
    }
    if (A.totals && lane == 0) A.seg_decay[vrow * A.nseg + seg] = __builtin_amdgcn_exp2f(static_cast<float>(log));
  }

  __device__ __forceinline__ void load_state() {
    if (A.seg_state != nullptr && !A.totals) {
      const float* sp = A.seg_state + (vrow * A.nseg + seg) * (kPB * NT);
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) st[t][r] = sp[p_of(r) * NT + n_of(t, r)];
    } else {
      const bool init = A.init != nullptr && !A.totals;
      const float* sp = A.init + ((bi * A.heads + h) * A.P + pb * kPB) * static_cast<long long>(A.N);
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          st[t][r] = init && p_of(r) < rows_p && n_of(t, r) < A.N ? sp[p_of(r) * A.N + n_of(t, r)] : 0.0f;
    }
  }
  __device__ __forceinline__ void store_state() const {
    if (A.totals) {
      float* sp = A.seg_state + (vrow * A.nseg + seg) * (kPB * NT);
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) sp[p_of(r) * NT + n_of(t, r)] = st[t][r];
    } else if (A.fin != nullptr && cc1 == A.nchunks) {
      float* sp = A.fin + ((bi * A.heads + h) * A.P + pb * kPB) * static_cast<long long>(A.N);
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (p_of(r) < rows_p && n_of(t, r) < A.N) sp[p_of(r) * A.N + n_of(t, r)] = st[t][r];
    }
  }
  // S = e^{c_end} S + sum_j in_j x_j k_j^T; this wave's columns: from row n0 of
  // lkt.  The weighted values, in pieces: `values(s, f)` for tokens 32 s + 0..31.
  template <typename F>
  __device__ __forceinline__ void update(const Gates<kQ>& G, const T* lkt, int n0, int rows, F values) {
    const float end = G.end[0];
#pragma unroll
    for (int t = 0; t < KT; ++t) st[t] = decayed(st[t], end);
#pragma unroll
    for (int s = 0; s < kQ / 32; ++s) {
      if (ended(32 * s, rows)) continue;
      Frag f[O::kSplit], kf[KT];
      values(s, f);
#pragma unroll
      for (int t = 0; t < KT; ++t) kf[t] = transposed_row(lkt, n0 + (READ ? state_row(t, l16) : 16 * t + l16), 32 * s + 8 * g4);
#pragma unroll
      for (int u = O::kSplit - 1; u >= 0; --u)
#pragma unroll
        for (int t = 0; t < KT; ++t)
          if (!padding(nbase + (READ ? 32 * (t / 2) : 16 * t))) st[t] = READ ? O::mma(kf[t], f[u], st[t]) : O::mma(f[u], kf[t], st[t]);
    }
  }
  // ... weighted and split here
  __device__ __forceinline__ void update_from(const Gates<kQ>& G, const T* lkt, int n0, int rows, const T* lxt) {
    update(G, lkt, n0, rows, [&](int s, Frag (&f)[O::kSplit]) {
      float xv[8], wv[8];
      O::widen(transposed_row(lxt, 16 * pw + l16, 32 * s + 8 * g4), xv);
      load8(G.in + 32 * s + 8 * g4, wv);
#pragma unroll
      for (int e = 0; e < 8; ++e) xv[e] *= wv[e];
      O::split(xv, f);
    });
  }
};

// States only: the state before every block of 2^keep_log2 chunks (in reversed
// time: after it), or a segment's total.  The columns of S are independent, so
// a workgroup takes kStateCols of them: several fit a compute unit and fill the
// chip more evenly than ones of twice the size (125 -> 117 us where both
// directions of eight sequences of 2,048 tokens, 24 heads, bfloat16, are walked).
// S is held by rows, so that a lane stores 16 adjacent bytes of a state (117 ->
// 97 us).  Without the stores of 201 MB of float32 states it took 67; the rest
// is issue: a wave's step is 190 vector, 24 matrix and 130 scalar instructions,
// and splitting the values is half of the first.
template <typename T, int NT, bool VEC>
__global__ void __launch_bounds__(kStatesThreads + kWave, VEC && sizeof(T) == 2 ? 5 : 3) scan_states_kernel(WalkPair P) {
  constexpr int kParts = NT / kStateCols, KT = kStateCols / 16;
  __shared__ __attribute__((aligned(16))) T lkt[kStateCols * kQ], lxt[kPB * kQ];   // k^T, x^T
  __shared__ Gates<kQ> gates[2];
  const ScanWalk A = P.w[blockIdx.y];
  const int block = xcd_item(blockIdx.x, gridDim.x), part = block % kParts;
  Walk<T, NT, KT, false> W(A, block / kParts);
  W.nbase = kStateCols * part;
  if (A.totals && W.seg + 1 == A.nseg) return;   // nothing starts after the last segment
  if (W.w == kStatesWaves) {
    W.gate_wave(gates);
    return;
  }
  const T* xp = static_cast<const T*>(A.x.p) + W.bi * A.x.sb + W.h * A.x.sh + W.pb * kPB;
  const T* kp = static_cast<const T*>(A.k.p) + W.bi * A.k.sb + W.grp * A.k.sh + W.nbase;
  PairLoad<T, kStateCols, kStatesThreads, VEC> tk;
  PairLoad<T, kPB, kStatesThreads, VEC> tx;
  kp += W.token_of(W.cc0) * A.k.st;
  xp += W.token_of(W.cc0) * A.x.st;
  const auto load_tiles = [&](int cc) {   // chunk after chunk
    const int rows = W.rows_of(cc);
    tk.load(kp, A.k.st, rows, A.N - W.nbase, W.tid);
    tx.load(xp, A.x.st, rows, W.rows_p, W.tid);
    kp += W.step(A.k.st);
    xp += W.step(A.x.st);
  };
  W.load_state();
  float* states = A.states == nullptr ? nullptr : A.states + W.vrow * A.nblocks * (kPB * NT);
  load_tiles(W.cc0);
  for (int cc = W.cc0; cc < W.cc1; ++cc) {
    __syncthreads();   // the last chunk's tiles are done with
    tk.store_transposed(lkt, W.tid);
    tx.store_transposed(lxt, W.tid);
    __syncthreads();
    load_tiles(cc + 1);
    const int chunk = W.chunk_of(cc), within = chunk & ((1 << A.keep_log2) - 1);
    if (states != nullptr && (W.reverse ? within + 1 == 1 << A.keep_log2 || chunk == W.last_chunk : within == 0)) {
      float* sp = states + static_cast<long long>(chunk >> A.keep_log2) * (kPB * NT);
#pragma unroll
      for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4_t*>(sp + state_offset(W.n_of(t, 0), W.p_of(0))) = W.st[t];
    }
    W.update_from(gates[(cc - W.cc0) & 1], lkt, 0, W.rows_of(cc), lxt);
  }
  W.store_state();
}

// Outputs and states.  Between two barriers: the tiles of M, what S_in gives
// (partial sums over the two halves of n, which the two waves of the same rows
// exchange through LDS, each finishing half of the tokens), and the next S; then
// what the chunk's own tokens give, and the next chunk's tiles go to LDS.
//
// Eight sequences of 2,048 tokens, 24 heads of 64 x 128, bfloat16: 98 to 104 us
// (192 workgroups, 32 steps of about 7,500 clocks); HBM needs 112 MB, 22 us.
// Bound by issue and LDS together: a step is 2,900 clocks of vector and 1,600 of
// matrix instructions a SIMD and 2,500 of LDS, and two waves a SIMD that meet
// at barriers overlap little of it.  What made the step short: 16-byte LDS reads
// without bank conflicts everywhere (107 -> 94 us, with two barriers instead of
// three and the weighted values split once for all waves), the gates, whose
// float64 prefix sum is a long chain, and two of the ten tiles of M on a wave of
// their own.  Four waves that hold all columns, in one piece, took 123 us against 107.
template <typename T, int NT, bool VEC>
__global__ void __launch_bounds__(sizeof(T) == 2 ? kReadThreads + kWave : kReadThreads, sizeof(T) == 2 ? 3 : 2) scan_read_kernel(WalkPair P) {
  typedef Ops<T> O;
  typedef typename O::Frag Frag;
  typedef Tile<T, NT> TN;
  typedef Tile<T, kQ> TM;
  constexpr int KT = NT / 32, kPieces = O::kRounded;   // of M and of the copy of S_in that is read
  // bfloat16: the weighted values of a chunk are split once for all waves, and
  // x^T, which a chunk reads last, is double, so that the next chunk's tiles need
  // no third barrier.  float32 values are not split, and its tiles fill the LDS.
  // (Arrays of their own: the compiler may move reads of one across writes to another.)
  constexpr bool kPlanes = sizeof(T) == 2;
  __shared__ __attribute__((aligned(16))) T lkt[NT * kQ], lk[kQ * NT], lq[kQ * NT], lxts[kPlanes ? 2 : 1][kPB * kQ];
  __shared__ __attribute__((aligned(16))) T lxw[kPlanes ? 3 * kPB * kQ : 8];   // weighted x^T in three pieces
  __shared__ __attribute__((aligned(16))) T lm[kPieces * kQ * kQ];            // the weights M [i][j], in pieces
  __shared__ f32x4_t ly[kReadWaves * 2 * kWave];   // halves of y that waves hand over
  __shared__ Gates<kQ> gates[2];
  const ScanWalk A = P.w[0];
  Walk<T, NT, KT, true> W(A, xcd_item(blockIdx.x, gridDim.x));
  // wave w of eight: rows 16 (w % 4) + 0..15, the columns of half w / 4
  const int tid = W.tid, lane = W.lane, w = W.w, l16 = W.l16, g4 = W.g4, pw = W.pw, nh = w >> 2, nbase = nh * (NT / 2);
  W.nbase = nbase;
  // tile e of M, rows i and columns j
  const auto weights = [&](int e, int rows, const Gates<kQ>& G) {
    const int it = tile_row(e), jt = tile_col(e, it);
    if (W.ended(16 * it, rows)) return;
    f32x4_t a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < NT / 32; ++s)
      if (!W.padding(32 * s)) a = O::mma(TN::row(lq, 16 * it + l16, 32 * s + 8 * g4), TN::row(lk, 16 * jt + l16, 32 * s + 8 * g4), a);
    const int i0 = 16 * it + 4 * g4, j = 16 * jt + l16;
    a *= between4(G, it, jt, i0, j) * G.b[j];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const T hi = O::from_f32(a[r]);
      lm[TM::at(i0 + r, j)] = hi;
      if constexpr (kPieces == 2) lm[kQ * kQ + TM::at(i0 + r, j)] = O::from_f32(a[r] - bf16_to_f32(hi));
    }
  };
  if (kPlanes && w == kReadWaves) {
    // the ninth wave: two of the ten tiles of M, then the next chunk's gates
    GateLoad gl;
    gl.load(W, W.cc0);
    write_gates(gates[0], gl.g, gl.b, lane, false);
    gl.load(W, W.cc0 + 1);
    __syncthreads();
    for (int cc = W.cc0; cc < W.cc1; ++cc) {
      const int slot = (cc - W.cc0) & 1;
      __syncthreads();
      weights(kReadWaves, kQ, gates[slot]);
      weights(kReadWaves + 1, kQ, gates[slot]);
      write_gates(gates[slot ^ 1], gl.g, gl.b, lane, false);
      gl.load(W, cc + 2);
      __syncthreads();
    }
    return;
  }
  const T* xp = static_cast<const T*>(A.x.p) + W.bi * A.x.sb + W.h * A.x.sh + W.pb * kPB;
  const T* kp = static_cast<const T*>(A.k.p) + W.bi * A.k.sb + W.grp * A.k.sh;
  const T* qp = static_cast<const T*>(A.q.p) + W.bi * A.q.sb + W.grp * A.q.sh;
  T* yp = static_cast<T*>(A.y) + (W.bi * A.tokens * A.heads + W.h) * A.P + W.pb * kPB;
  const long long yst = static_cast<long long>(A.heads) * A.P;

  PairLoad<T, NT, kReadThreads, VEC, NT == 64 ? 4 : O::kVec> tk;
  PairLoad<T, kPB, kReadThreads, VEC, 4> tx;
  TileLoad<T, NT, kQ, kReadThreads, VEC> tq;
  kp += W.token_of(W.cc0) * A.k.st;
  qp += W.token_of(W.cc0) * A.q.st;
  xp += W.token_of(W.cc0) * A.x.st;
  yp += W.token_of(W.cc0) * yst;
  const auto load_tiles = [&](int cc) {   // chunk after chunk
    const int rows = W.rows_of(cc);
    tk.load(kp, A.k.st, rows, A.N, tid);
    tq.load(qp, A.q.st, rows, A.N, tid);
    tx.load(xp, A.x.st, rows, W.rows_p, tid);
    kp += W.step(A.k.st);
    qp += W.step(A.q.st);
    xp += W.step(A.x.st);
  };

  W.load_state();
  // tiles (0, 1) and (2, 3) of M lie above the diagonal inside the 32-wide
  // steps that are multiplied: zero for good
  if (w < 2) {
    const int r0 = 32 * w, c0 = r0 + 16;
#pragma unroll
    for (int e = 0; e < 4 * kPieces; ++e) lm[e / 4 * kQ * kQ + TM::at(r0 + l16, c0 + 4 * g4 + e % 4)] = O::from_f32(0.0f);
  }
  const auto store_tiles = [&](int slot) {
    tk.store(lk, tid);
    tk.store_transposed(lkt, tid);
    tq.store(lq, tid);
    tx.store_transposed(lxts[kPlanes ? slot : 0], tid);
    if constexpr (kPlanes) tx.store_split(lxw, gates[slot].in, tid);
  };
  load_tiles(W.cc0);
  // float32: no ninth wave, whose registers the others need (77 tokens, 12 heads, N = 72, padding multiplied: 28 us
  // with it, 23 without)
  GateLoad gl;
  const bool gate_wave = !kPlanes && w == kReadWaves - 1;
  if (gate_wave) {
    gl.load(W, W.cc0);
    write_gates(gates[0], gl.g, gl.b, lane, false);
    gl.load(W, W.cc0 + 1);
  }
  __syncthreads();   // the first gates are written
  store_tiles(0);
  load_tiles(W.cc0 + 1);
  for (int cc = W.cc0; cc < W.cc1; ++cc) {
    const int slot = (cc - W.cc0) & 1;
    const Gates<kQ>& G = gates[slot];
    const T* lxt = lxts[kPlanes ? slot : 0];
    const int rows = W.rows_of(cc);
    __syncthreads();   // the tiles are written
    weights(w, rows, G);
    if (!kPlanes && w < 2) weights(kReadWaves + w, rows, G);
    if (gate_wave) {
      write_gates(gates[slot ^ 1], gl.g, gl.b, lane, false);
      gl.load(W, cc + 2);
    }
    // what this half of S_in gives, e^{c_i} S_in q_i: y^T rows p = 16 pw + 4 g4 + 0..3, column i = 16 it + l16
    f32x4_t y[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) y[it] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < KT / 2; ++s) {
      if (W.padding(nbase + 32 * s)) continue;
      const f32x4_t a = W.st[2 * s], b = W.st[2 * s + 1];
      const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      Frag f[kPieces];
      O::split(v, f);
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        if (W.ended(16 * it, rows)) continue;
        const Frag qf = TN::row(lq, 16 * it + l16, nbase + 32 * s + 8 * g4);
#pragma unroll
        for (int u = kPieces - 1; u >= 0; --u) y[it] = O::mma(f[u], qf, y[it]);
      }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) y[it] = decayed(y[it], G.first[16 * it + l16]);
    // token tiles 2 nh and 2 nh + 1 stay, the others go to the other half's wave
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      ly[(w * 2 + u) * 64 + lane] = nh == 0 ? y[2 + u] : y[u];
      y[u] = nh == 0 ? y[u] : y[2 + u];
    }
    if constexpr (kPlanes)
      W.update(G, lkt, nbase, rows, [&](int s, Frag (&f)[O::kSplit]) {
#pragma unroll
        for (int u = 0; u < O::kSplit; ++u) f[u] = transposed_row(lxw + u * kPB * kQ, 16 * pw + l16, 32 * s + 8 * g4);
      });
    else
      W.update_from(G, lkt, nbase, rows, lxt);
    __syncthreads();   // M, the halves of y and the next gates are written; the tiles but x^T are done with
    // what the chunk's own tokens give
#pragma unroll
    for (int u = 0; u < 2; ++u) y[u] += ly[((w ^ 4) * 2 + u) * 64 + lane];
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (s <= nh && !W.ended(32 * nh, rows)) {
        const Frag vf = transposed_row(lxt, 16 * pw + l16, 32 * s + 8 * g4);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int z = kPieces - 1; z >= 0; --z)
            y[u] = O::mma(vf, TM::row(lm + z * kQ * kQ, 32 * nh + 16 * u + l16, 32 * s + 8 * g4), y[u]);
      }
    const TileStore<T, VEC> out(yp, yst, rows, W.rows_p);
    yp += W.step(yst);
#pragma unroll
    for (int u = 0; u < 2; ++u) out.put(32 * nh + 16 * u + l16, 16 * pw + 4 * g4, y[u]);
    if constexpr (!kPlanes) __syncthreads();
    store_tiles(slot ^ 1);
    load_tiles(cc + 2);
  }
  W.store_state();
}

// The state that each segment starts from, out of the segments' own totals
// (in place: a total is read before its slot is overwritten).  A thread an
// element, segment after segment: 6 us for 24 heads of 64 x 128 and ten segments,
// bound by the chain of loads.
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
    cur = own + decayed(cur, dp[s]);
  }
  sp[static_cast<long long>(A.nseg - 1) * kPB * nt] = cur;
}

template <typename T, int NT, bool VEC>
hipError_t states(const WalkPair& W, int dirs, long long items, hipStream_t st) {
  hipLaunchKernelGGL((scan_states_kernel<T, NT, VEC>), dim3(static_cast<unsigned>(items * (NT / kStateCols)), dirs),
                     dim3(kStatesThreads + kWave), 0, st, W);
  return hipGetLastError();
}
template <typename T, int NT, bool VEC>
hipError_t read(const WalkPair& W, long long items, hipStream_t st) {
  hipLaunchKernelGGL((scan_read_kernel<T, NT, VEC>), dim3(static_cast<unsigned>(items)),
                     dim3(kReadThreads + (sizeof(T) == 2 ? kWave : 0)), 0, st, W);
  return hipGetLastError();
}
template <typename T, int NT, bool VEC>
hipError_t walk(const WalkPair& W, int dirs, bool reads, hipStream_t st) {
  const ScanWalk& a = W.w[0];
  const long long items = static_cast<long long>(a.batch) * a.heads * a.pblocks * a.nseg;
  if (!reads) return states<T, NT, VEC>(W, dirs, items, st);
  return read<T, NT, VEC>(W, items, st);
}
template <typename T, int NT>
hipError_t walk_any(const WalkPair& W, int dirs, bool reads, bool vec, hipStream_t st) {
  return vec ? walk<T, NT, true>(W, dirs, reads, st) : walk<T, NT, false>(W, dirs, reads, st);
}
hipError_t walk_any(const WalkPair& W, int dirs, bool reads, bool vec, bool bf16, hipStream_t st) {
  if (W.w[0].N <= 64) return bf16 ? walk_any<bf16_t, 64>(W, dirs, reads, vec, st) : walk_any<float, 64>(W, dirs, reads, vec, st);
  return bf16 ? walk_any<bf16_t, 128>(W, dirs, reads, vec, st) : walk_any<float, 128>(W, dirs, reads, vec, st);
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
// one token: S' = e^g S + b v k^T, y = S' q.  Reads and writes the state once,
// which is what bounds it: 160 sequences of 24 heads, 64 x 128, take 49 us for
// 252 MB (5.1 TB/s, the rate of a large copy); one sequence is 4.5 us of launch
// and latency.  The state is next read a token later, by when other layers'
// states have passed, so it goes past the caches (such batches in turn: 62 us
// with stores past them, 71 without; 49 and 52 with loads past them or not).  A
// half-wave holds a row's N <= 128 elements, 4 consecutive ones a lane.
// ---------------------------------------------------------------------------
namespace {

constexpr int kStepHalves = kStepThreads / 32;   // half-waves of a workgroup, a row of the state at a time

template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<bf16_t>(const bf16_t* p) { return bf16_to_f32(*p); }
template <>
__device__ __forceinline__ float load1<float>(const float* p) { return *p; }

// EACH: rows of a half-wave, whose loads are under way together.
template <typename T, int EACH>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(ScanStep A) {
  constexpr int kRows = EACH * kStepHalves;
  const int half = threadIdx.x >> 5, l = threadIdx.x & 31, n0 = 4 * l;
  const int pblocks = (A.P - 1) / kRows + 1;
  const int pb = static_cast<int>(blockIdx.x) % pblocks;
  const long long bh = blockIdx.x / pblocks;
  const int h = static_cast<int>(bh % A.heads), grp = h / (A.heads / A.groups);
  const long long bi = bh / A.heads;
  const T* vp = static_cast<const T*>(A.v.p) + bi * A.v.sb + h * A.v.sh;
  const T* kp = static_cast<const T*>(A.k.p) + bi * A.k.sb + grp * A.k.sh;
  const T* qp = static_cast<const T*>(A.q.p) + bi * A.q.sb + grp * A.q.sh;
  const bool vec = A.N % 4 == 0;   // rows of the state stay 16-byte aligned
  f32x4_t s[EACH];
  bool live[EACH];
  const float* sp[EACH];
#pragma unroll
  for (int u = 0; u < EACH; ++u) {
    const int p = pb * kRows + kStepHalves * u + half;
    live[u] = p < A.P;
    sp[u] = A.S + (bh * A.P + p) * A.N + n0;
    s[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (live[u] && n0 < A.N) {
      if (vec) {
        s[u] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(sp[u]));
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
  for (int u = 0; u < EACH; ++u) {
    const int p = pb * kRows + kStepHalves * u + half;
    const float v = live[u] ? gate * load1<T>(vp + p) : 0.0f;
    float y = 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      s[u][r] = fmaf(decay, decay == 0.0f ? 0.0f : s[u][r], v * k[r]);
      y = fmaf(s[u][r], q[r], y);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) y += __shfl_xor(y, off, kWave);
    if (!live[u]) continue;
    float* op = A.S_out + (bh * A.P + p) * A.N + n0;
    if (n0 < A.N) {
      if (vec) {
        __builtin_nontemporal_store(s[u], reinterpret_cast<f32x4_t*>(op));
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n0 + r < A.N) op[r] = s[u][r];
      }
    }
    if (l == 0) static_cast<T*>(A.y)[bh * A.P + p] = Ops<T>::from_f32(y);
  }
}

template <int EACH>
hipError_t step(const ScanStep& A, bool bf16, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(scan_step_blocks(A.batch, A.heads, A.P)));
  if (bf16) hipLaunchKernelGGL((scan_step_kernel<bf16_t, EACH>), grid, dim3(kStepThreads), 0, st, A);
  else hipLaunchKernelGGL((scan_step_kernel<float, EACH>), grid, dim3(kStepThreads), 0, st, A);
  return hipGetLastError();
}

// Four rows a half-wave where that leaves two workgroups to each of 256 compute
// units, two where it does not: 192 heads of 64 x 128 take 6.6 us by four and
// 5.9 by two (24 heads 5.4 and 4.4), 384 heads 8.0 and 8.6, 1,536 heads 20 and 26.
int step_rows(int batch, int heads, int P) {
  return static_cast<double>(batch) * heads * P >= 2.0 * 256 * 4 * kStepHalves ? 4 : 2;
}

}  // namespace

long long scan_step_blocks(int batch, int heads, int P) {
  const int rows = step_rows(batch, heads, P) * kStepHalves, pblocks = (P - 1) / rows + 1;
  const long long bh = static_cast<long long>(batch) * heads;
  return bh > LLONG_MAX / pblocks ? LLONG_MAX : bh * pblocks;
}
hipError_t launch_scan_step(const ScanStep& A, bool bf16, hipStream_t st) {
  return step_rows(A.batch, A.heads, A.P) == 4 ? step<4>(A, bf16, st) : step<2>(A, bf16, st);
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
