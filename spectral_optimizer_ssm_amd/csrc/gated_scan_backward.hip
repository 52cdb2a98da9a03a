// Gradients of the gated scan (gated_scan.hip), chunk by chunk.  With
//   A_ij = q_i . k_j,  E_ij = dy_i . v_j,  L_ij = e^{c_i - c_j} for i >= j (else 0)
// and the states S_in before and dS_out after the chunk (scan_walk_kernel, in
// forward and in reversed time):
//   z_j  = sum_i L_ij A_ij dy_i + e^{c_end - c_j} dS_out k_j,  dv_j = b_j z_j,  db_j = v_j . z_j
//   dq_i = sum_h [ sum_j L_ij b_j E_ij k_j + e^{c_i} S_in^T dy_i ]
//   dk_j = sum_h b_j [ sum_i L_ij E_ij q_i + e^{c_end - c_j} dS_out^T v_j ]
// over the heads h that share the keys and queries.  The log decay of t scales
// whatever crosses t: with W_ij = L_ij b_j A_ij E_ij,
//   dg_t = sum_{i >= t} (sum_j W_ij - sum_j W_ji + dy_i . e^{c_i} S_in q_i)
//        + sum_{j < t} b_j e^{c_end - c_j} v_j . dS_out k_j + e^{c_end} <S_in, dS_out>,
// where no sum leaves the chunk, so nothing large cancels.
//
// One workgroup takes a chunk and walks the heads that share its keys and
// queries: A, and the sum over heads of L b E, stay in registers, so the
// chunk's products with k and q are done once for all heads, and dq and dk are
// summed in float32 registers without atomics.  Where that leaves too few
// workgroups the heads are split and the parts added by a second kernel in
// fixed order.
//
// Rounding, bfloat16 operands: L A, the sum of L b E and the copy of dS_out
// that dv reads are rounded to bfloat16 once; dq and dk take the states as
// three bfloat16 pieces (float32 accuracy), since db and dg, which are
// float32, are dot products of them.
#include "scan_tiles.cuh"

namespace muon {
namespace {

using namespace scan;

template <typename T, int NT>
struct GradLds {
  static constexpr int kLdN = NT + Ops<T>::kPad;
  static constexpr int kLdP = kPB + Ops<T>::kPad;
  static constexpr int kLdM = kQ + Ops<T>::kPad;
  static constexpr int q = 0;                                     // [kQ][NT]
  static constexpr int k = q + kQ * kLdN * (int)sizeof(T);        // [kQ][NT]
  static constexpr int v = k + kQ * kLdN * (int)sizeof(T);        // [kQ][kPB]; at the end D [i][j]
  static constexpr int dy = v + kQ * kLdP * (int)sizeof(T);       // [kQ][kPB]; at the end D^T [j][i]
  static constexpr int m = dy + kQ * kLdP * (int)sizeof(T);       // (L A)^T [j][i]
  static constexpr int gates = m + kQ * kLdM * (int)sizeof(T);    // Gates
  static constexpr int rows = gates + (int)sizeof(Gates);         // row sums of W by column block [4][kQ]
  static constexpr int cols = rows + 4 * kQ * 4;                  // column sums of L A E by row block [4][kQ]
  static constexpr int qs = cols + 4 * kQ * 4;                    // e^{c_i} q_i . S_in^T dy_i by wave [4][kQ]
  static constexpr int ks = qs + 4 * kQ * 4;                      // e^{c_end - c_j} k_j . dS_out^T v_j by wave [4][kQ]
  static constexpr int through = ks + 4 * kQ * 4;                 // <S_in, dS_out> by wave [4]
  static constexpr int bytes = through + 16;
};

// Sum over the 16 lanes of a row.
__device__ __forceinline__ float row_sum(float v) {
  v += dpp_f<kDppXor1>(v);
  v += dpp_f<kDppXor2>(v);
  v += dpp_f<0x141>(v);   // row_half_mirror
  v += dpp_f<0x140>(v);   // row_mirror
  return v;
}

template <typename T, int NT>
__global__ void __launch_bounds__(kThreads, 2) scan_grad_kernel(ScanGrad A) {
  typedef Ops<T> O;
  typedef typename O::Frag Frag;
  typedef GradLds<T, NT> L;
  constexpr int kNW = NT / 64;   // 16-wide blocks of n per wave
  extern __shared__ __attribute__((aligned(16))) char lds[];
  T* lq = reinterpret_cast<T*>(lds + L::q);
  T* lk = reinterpret_cast<T*>(lds + L::k);
  T* lv = reinterpret_cast<T*>(lds + L::v);
  T* ldy = reinterpret_cast<T*>(lds + L::dy);
  T* lm = reinterpret_cast<T*>(lds + L::m);
  Gates& G = *reinterpret_cast<Gates*>(lds + L::gates);
  float* lrow = reinterpret_cast<float*>(lds + L::rows);
  float* lcol = reinterpret_cast<float*>(lds + L::cols);
  float* lqs = reinterpret_cast<float*>(lds + L::qs);
  float* lks = reinterpret_cast<float*>(lds + L::ks);
  float* lthrough = reinterpret_cast<float*>(lds + L::through);

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l16 = lane & 15, g4 = lane >> 4;
  const int split = static_cast<int>(blockIdx.x % A.nsplit);
  const long long rest = blockIdx.x / A.nsplit;
  const int grp = static_cast<int>(rest % A.groups);
  const int c = static_cast<int>(rest / A.groups % A.nchunks);
  const long long bi = rest / A.groups / A.nchunks;
  const long long t0 = static_cast<long long>(c) * kQ;
  const int rows = A.tokens - t0 < kQ ? static_cast<int>(A.tokens - t0) : kQ;
  const int per_group = A.heads / A.groups;
  const int per_split = (per_group + A.nsplit - 1) / A.nsplit;
  const int h0 = grp * per_group + split * per_split;
  const int h1 = grp * per_group + (split * per_split + per_split < per_group ? split * per_split + per_split : per_group);
  const int nvirt = (h1 - h0) * A.pblocks;   // (head, block of kPB value components), heads outermost
  const int vheads = A.heads * A.pblocks;

  const auto rows_p_of = [&](int pb) { return A.P - pb * kPB < kPB ? A.P - pb * kPB : kPB; };
  TileLoad<T, kPB> tv, tdy;
  float gv = 0.0f, bv = 0.0f;
  const auto load_head = [&](int i) {
    const int h = h0 + i / A.pblocks, pb = i % A.pblocks, rp = rows_p_of(pb);
    const T* vp = static_cast<const T*>(A.v.p) + bi * A.v.sb + h * A.v.sh + t0 * A.v.st + pb * kPB;
    const T* dp = static_cast<const T*>(A.dy.p) + bi * A.dy.sb + h * A.dy.sh + t0 * A.dy.st + pb * kPB;
    tv.load(vp, A.v.st, rows, rp, A.v.vec && rp % O::kVec == 0);
    tdy.load(dp, A.dy.st, rows, rp, A.dy.vec && rp % O::kVec == 0);
    if (w == 3) {
      gv = 0.0f;
      bv = 0.0f;
      if (lane < rows) {
        gv = (static_cast<const float*>(A.g.p) + bi * A.g.sb + h * A.g.sh)[(t0 + lane) * A.g.st];
        bv = A.b.p == nullptr ? 1.0f : (static_cast<const float*>(A.b.p) + bi * A.b.sb + h * A.b.sh)[(t0 + lane) * A.b.st];
      }
    }
  };

  {
    TileLoad<T, NT> tq, tk;
    tq.load(static_cast<const T*>(A.q.p) + bi * A.q.sb + grp * A.q.sh + t0 * A.q.st, A.q.st, rows, A.N, A.q.vec);
    tk.load(static_cast<const T*>(A.k.p) + bi * A.k.sb + grp * A.k.sh + t0 * A.k.st, A.k.st, rows, A.N, A.k.vec);
    if (nvirt > 0) load_head(0);
    tq.store(lq);
    tk.store(lk);
  }
  // tiles of (L A)^T and of the sums that no wave writes
  for (int i = tid; i < kQ * L::kLdM; i += kThreads) lm[i] = O::from_f32(0.0f);
  for (int i = tid; i < 4 * kQ; i += kThreads) {
    lrow[i] = 0.0f;
    lcol[i] = 0.0f;
  }
  __syncthreads();

  // A and the sum of L b E: tiles on and below the diagonal, rows i, columns j
  const int ntile = tile_count(w);
  f32x4_t sc[kMaxTiles], dsum[kMaxTiles];
#pragma unroll
  for (int t = 0; t < kMaxTiles; ++t) {
    sc[t] = dsum[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    if (t < ntile)
#pragma unroll
      for (int s = 0; s < NT / 32; ++s)
        sc[t] = O::mma(O::row(lq + (16 * tile_row(w, t) + l16) * L::kLdN + 32 * s + 8 * g4),
                       O::row(lk + (16 * tile_col(w, t) + l16) * L::kLdN + 32 * s + 8 * g4), sc[t]);
  }
  // dq^T and dk^T: rows n = 16 (w kNW + b) + 4 g4 + 0..3, column i (j) = 16 it + l16
  f32x4_t dq[kNW][4], dk[kNW][4];
#pragma unroll
  for (int b = 0; b < kNW; ++b)
#pragma unroll
    for (int it = 0; it < 4; ++it) dq[b][it] = dk[b][it] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  float acc_in = 0.0f, acc_leave = 0.0f, acc_db = 0.0f, acc_z = 0.0f;   // wave 0: token = lane, over a head's blocks
  for (int i = 0; i < nvirt; ++i) {
    const int h = h0 + i / A.pblocks, pb = i % A.pblocks;
    const long long srow = ((bi * vheads + h * A.pblocks + pb) * A.nchunks + c) * static_cast<long long>(kPB * NT);
    const float* sp = A.states + srow;
    const float* dsp = A.dstates + srow;
    tv.store(lv);
    tdy.store(ldy);
    if (w == 3) write_gates(G, gv, bv, lane);
    __syncthreads();
    if (i + 1 < nvirt) load_head(i + 1);

#pragma unroll
    for (int t = 0; t < kMaxTiles; ++t) {
      if (t < ntile) {
        const int it = tile_row(w, t), jt = tile_col(w, t);
        f32x4_t e = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kPB / 32; ++s)
          e = O::mma(O::row(ldy + (16 * it + l16) * L::kLdP + 32 * s + 8 * g4),
                     O::row(lv + (16 * jt + l16) * L::kLdP + 32 * s + 8 * g4), e);
        const int j = 16 * jt + l16, i0 = 16 * it + 4 * g4;
        const float hi = G.hi[j], lo = G.lo[j], b = G.b[j];
        const f32x4_t ih = *reinterpret_cast<const f32x4_t*>(G.hi + i0), il = *reinterpret_cast<const f32x4_t*>(G.lo + i0);
        f32x4_t mm;
        float col = 0.0f;
        float rsum[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float d = i0 + r >= j ? between(ih[r], il[r], hi, lo) : 0.0f;
          mm[r] = d * sc[t][r];
          const float le = d * e[r];
          dsum[t][r] = fmaf(le, b, dsum[t][r]);
          const float we = mm[r] * e[r];
          col += we;
          rsum[r] = row_sum(we * b);
        }
        O::store4(lm + j * L::kLdM + i0, mm);
        col += __shfl_xor(col, 16, kWave);
        col += __shfl_xor(col, 32, kWave);
        if (g4 == 0) lcol[it * kQ + j] = col;
        if (l16 == 0) *reinterpret_cast<f32x4_t*>(lrow + jt * kQ + i0) = f32x4_t{rsum[0], rsum[1], rsum[2], rsum[3]};
      }
    }

    // the states' part of dq and dk, and the states' product
    float qs[4] = {0.0f, 0.0f, 0.0f, 0.0f}, ks[4] = {0.0f, 0.0f, 0.0f, 0.0f}, through = 0.0f;
#pragma unroll
    for (int b = 0; b < kNW; ++b) {
      const int n0 = 16 * (w * kNW + b);
      f32x4_t aq[4], ak[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) aq[it] = ak[it] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < kPB / 32; ++s) {
        float x[8], y[8];
        const long long off = static_cast<long long>(32 * s + 8 * g4) * NT + n0 + l16;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = sp[off + e * NT];
          y[e] = dsp[off + e * NT];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) through = fmaf(x[e], y[e], through);
        Frag fx[O::kSplit], fy[O::kSplit];
        O::split(x, fx);
        O::split(y, fy);
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          const Frag d = O::row(ldy + (16 * it + l16) * L::kLdP + 32 * s + 8 * g4);
          const Frag v = O::row(lv + (16 * it + l16) * L::kLdP + 32 * s + 8 * g4);
#pragma unroll
          for (int u = O::kSplit - 1; u >= 0; --u) {
            aq[it] = O::mma(fx[u], d, aq[it]);
            ak[it] = O::mma(fy[u], v, ak[it]);
          }
        }
      }
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int t = 16 * it + l16;
        const float first = G.first[t], last = G.last[t], bt = G.b[t];
        const f32x4_t qv = O::load4(lq + t * L::kLdN + n0 + 4 * g4), kv = O::load4(lk + t * L::kLdN + n0 + 4 * g4);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float a = aq[it][r] * first, d = ak[it][r] * last;
          qs[it] = fmaf(a, qv[r], qs[it]);
          ks[it] = fmaf(d, kv[r], ks[it]);
          dq[b][it][r] += a;
          dk[b][it][r] = fmaf(d, bt, dk[b][it][r]);
        }
      }
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      qs[it] += __shfl_xor(qs[it], 16, kWave);
      qs[it] += __shfl_xor(qs[it], 32, kWave);
      ks[it] += __shfl_xor(ks[it], 16, kWave);
      ks[it] += __shfl_xor(ks[it], 32, kWave);
      if (g4 == 0) {
        lqs[w * kQ + 16 * it + l16] = qs[it];
        lks[w * kQ + 16 * it + l16] = ks[it];
      }
    }
    through = wave_sum(through);
    if (lane == 0) lthrough[w] = through;

    // z^T: rows p = 16 w + 4 g4 + 0..3, column j = 16 jt + l16; the states' part first
    f32x4_t z[4];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) z[jt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < NT / 32; ++s) {
      const float* dp = dsp + (16 * w + l16) * NT + 32 * s + 8 * g4;
      const f32x4_t a = *reinterpret_cast<const f32x4_t*>(dp), b = *reinterpret_cast<const f32x4_t*>(dp + 4);
      const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
      const Frag f = O::narrow(x);
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) z[jt] = O::mma(f, O::row(lk + (16 * jt + l16) * L::kLdN + 32 * s + 8 * g4), z[jt]);
    }
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) z[jt] *= G.last[16 * jt + l16];
    __syncthreads();   // (L A)^T and the sums are written
#pragma unroll
    for (int s = 0; s < kQ / 32; ++s) {
      const Frag f = O::col(ldy, L::kLdP, 32 * s, 16 * w, lane);
#pragma unroll
      for (int jt = 0; jt < 2 * s + 2; ++jt) z[jt] = O::mma(f, O::row(lm + (16 * jt + l16) * L::kLdM + 32 * s + 8 * g4), z[jt]);
    }
    const int rp = rows_p_of(pb), p0 = 16 * w + 4 * g4;
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      const int j = 16 * jt + l16;
      if (j < rows && p0 < rp) {
        const f32x4_t o = z[jt] * G.b[j];
        T* op = static_cast<T*>(A.dv) + ((bi * A.tokens + t0 + j) * A.heads + h) * A.P + pb * kPB + p0;
        if (A.dvvec) {
          O::store4(op, o);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (p0 + r < rp) op[r] = O::from_f32(o[r]);
        }
      }
    }

    if (w == 0) {
      const float b = G.b[lane];
      const float rs = (lrow[lane] + lrow[kQ + lane]) + (lrow[2 * kQ + lane] + lrow[3 * kQ + lane]);
      const float cs = (lcol[lane] + lcol[kQ + lane]) + (lcol[2 * kQ + lane] + lcol[3 * kQ + lane]);
      const float us = (lqs[lane] + lqs[kQ + lane]) + (lqs[2 * kQ + lane] + lqs[3 * kQ + lane]);
      const float ws = (lks[lane] + lks[kQ + lane]) + (lks[2 * kQ + lane] + lks[3 * kQ + lane]);
      acc_in += rs - b * cs + us;
      acc_leave = fmaf(b, ws, acc_leave);
      acc_db += cs + ws;
      acc_z += (lthrough[0] + lthrough[1]) + (lthrough[2] + lthrough[3]);
      if (pb + 1 == A.pblocks) {
        const double pin = wave_prefix_d(static_cast<double>(acc_in));
        const double pl = wave_prefix_d(static_cast<double>(acc_leave));
        const double suffix = read_lane_d(pin, 63) - pin + static_cast<double>(acc_in);
        const double before = pl - static_cast<double>(acc_leave);
        if (lane < rows) {
          const long long o = (bi * A.tokens + t0 + lane) * A.heads + h;
          const double d = suffix + before + static_cast<double>(G.end[0]) * static_cast<double>(acc_z);
          // nothing crosses a token whose decay is 0: what the sums leave there is rounding
          A.dg[o] = G.own[lane] == 0.0f ? 0.0f : static_cast<float>(d);
          if (A.db != nullptr) A.db[o] = acc_db;
        }
        acc_in = acc_leave = acc_db = acc_z = 0.0f;
      }
    }
    __syncthreads();   // the tiles, gates and sums are done with
  }

  // D = sum over heads of L b E, once as D [i][j] and once as D^T [j][i]
  T* ld = lv;
  T* ldt = ldy;
  for (int i = tid; i < kQ * L::kLdP; i += kThreads) ld[i] = ldt[i] = O::from_f32(0.0f);
  __syncthreads();
#pragma unroll
  for (int t = 0; t < kMaxTiles; ++t) {
    if (t < ntile) {
      const int j = 16 * tile_col(w, t) + l16, i0 = 16 * tile_row(w, t) + 4 * g4;
      O::store4(ldt + j * L::kLdP + i0, dsum[t]);
#pragma unroll
      for (int r = 0; r < 4; ++r) ld[(i0 + r) * L::kLdP + j] = O::from_f32(dsum[t][r]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int b = 0; b < kNW; ++b) {
    const int n0 = 16 * (w * kNW + b);
#pragma unroll
    for (int s = 0; s < kQ / 32; ++s) {
      const Frag fk = O::col(lk, L::kLdN, 32 * s, n0, lane), fq = O::col(lq, L::kLdN, 32 * s, n0, lane);
#pragma unroll
      for (int it = 2 * s; it < 4; ++it) dq[b][it] = O::mma(fk, O::row(ld + (16 * it + l16) * L::kLdP + 32 * s + 8 * g4), dq[b][it]);
#pragma unroll
      for (int it = 0; it < 2 * s + 2; ++it) dk[b][it] = O::mma(fq, O::row(ldt + (16 * it + l16) * L::kLdP + 32 * s + 8 * g4), dk[b][it]);
    }
    const int n = n0 + 4 * g4;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int t = 16 * it + l16;
      if (t >= rows || n >= A.N) continue;
      const long long o = ((bi * A.tokens + t0 + t) * A.groups + grp) * A.N + n;
      if (A.nsplit > 1) {
        const long long half = static_cast<long long>(A.batch) * A.tokens * A.groups * A.N;
        float* pq = A.parts + (2LL * split) * half + o;
        float* pk = pq + half;
        if (A.N % 4 == 0) {
          *reinterpret_cast<f32x4_t*>(pq) = dq[b][it];
          *reinterpret_cast<f32x4_t*>(pk) = dk[b][it];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < A.N) {
              pq[r] = dq[b][it][r];
              pk[r] = dk[b][it][r];
            }
        }
      } else if (A.dkvec) {
        O::store4(static_cast<T*>(A.dq) + o, dq[b][it]);
        O::store4(static_cast<T*>(A.dk) + o, dk[b][it]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < A.N) {
            static_cast<T*>(A.dq)[o + r] = O::from_f32(dq[b][it][r]);
            static_cast<T*>(A.dk)[o + r] = O::from_f32(dk[b][it][r]);
          }
      }
    }
  }
}

// dq and dk out of the head splits' parts, added in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) scan_parts_kernel(const float* parts, int nsplit, long long half, T* dq, T* dk) {
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= 2 * half) return;
  float s = 0.0f;
  for (int u = 0; u < nsplit; ++u) s += parts[2LL * u * half + i];
  if (i < half) dq[i] = Ops<T>::from_f32(s);
  else dk[i - half] = Ops<T>::from_f32(s);
}

template <typename T, int NT>
hipError_t grad(const ScanGrad& A, hipStream_t st) {
  constexpr int bytes = GradLds<T, NT>::bytes;
  const void* fn = reinterpret_cast<const void*>(scan_grad_kernel<T, NT>);
  hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  const long long items = static_cast<long long>(A.batch) * A.nchunks * A.groups * A.nsplit;
  hipLaunchKernelGGL((scan_grad_kernel<T, NT>), dim3(static_cast<unsigned>(items)), dim3(kThreads), bytes, st, A);
  e = hipGetLastError();
  if (e != hipSuccess || A.nsplit == 1) return e;
  const long long half = static_cast<long long>(A.batch) * A.tokens * A.groups * A.N;
  hipLaunchKernelGGL((scan_parts_kernel<T>), dim3(static_cast<unsigned>((2 * half + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                     st, A.parts, A.nsplit, half, static_cast<T*>(A.dq), static_cast<T*>(A.dk));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_grad(const ScanGrad& A, bool bf16, hipStream_t st) {
  if (A.N <= 64) return bf16 ? grad<bf16_t, 64>(A, st) : grad<float, 64>(A, st);
  return bf16 ? grad<bf16_t, 128>(A, st) : grad<float, 128>(A, st);
}

}  // namespace muon
