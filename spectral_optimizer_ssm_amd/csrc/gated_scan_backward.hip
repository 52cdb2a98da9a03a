// Gradients of the gated scan (gated_scan.hip), by blocks of tokens.  With
//   A_ij = q_i . k_j,  E_ij = dy_i . v_j,  L_ij = e^{c_i - c_j} for i >= j (else 0)
// and the states S_in before and dS_out after the block (scan_states_kernel,
// in forward and in reversed time):
//   z_j  = sum_i L_ij A_ij dy_i + e^{c_end - c_j} dS_out k_j,  dv_j = b_j z_j,  db_j = v_j . z_j
//   dq_i = sum_h [ sum_j L_ij b_j E_ij k_j + e^{c_i} S_in^T dy_i ]
//   dk_j = sum_h b_j [ sum_i L_ij E_ij q_i + e^{c_end - c_j} dS_out^T v_j ]
// over the heads h that share the keys and queries.  The log decay of t scales
// whatever crosses t: with W_ij = L_ij b_j A_ij E_ij,
//   dg_t = sum_{j < t <= i} W_ij + sum_{i >= t} dy_i . e^{c_i} S_in q_i
//        + sum_{j < t} b_j e^{c_end - c_j} v_j . dS_out k_j + e^{c_end} <S_in, dS_out>.
// Only what crosses t is added, so its float32 accuracy holds where a strong
// decay leaves little of it.  With t in token tile T, the pairs are those of T's
// own tile, whose rows are summed up to each column; the rest of T's columns
// before t (tiles below) and of its rows from t on (tiles to the left); and the
// whole tiles below T and to its left.
//
// One workgroup takes a block of tokens and walks the heads that share its keys
// and queries: A, and the sum over heads of L b E, stay in registers, so the
// block's products with k and q are done once for all heads, and dq and dk are
// summed in float32 registers without atomics.  Where that leaves too few
// workgroups the heads are split and the parts added by a second kernel in
// fixed order.
//
// Eight sequences of 2,048 tokens, 24 heads of 64 x 128 sharing keys, bfloat16:
// 174 us, of which the two states' 201 MB alone need 40 at the rate of a large
// copy.  Bound by issue: of about 400,000 clocks a SIMD has 180,000 of vector
// instructions (the weights and sums of E's tiles, the states' splits) and 64,000
// of matrix ones, with two waves to overlap them and the LDS.  Blocks of
// 64 tokens would read and write twice the states.
//
// Rounding, bfloat16 operands: L A, the sum of L b E and the copy of dS_out
// that dv reads are two bfloat16 pieces (16 bits), so that dv, dq and dk are off by
// their own rounding alone (by 1.2 to 1.4 times that in one piece, which would save
// 15 us); dq and dk take the states as three pieces (float32 accuracy), since
// db and dg, which are float32, are dot products of them.  The pieces of L A and
// of the sums are kept as the tiles on one side of the diagonal, or they would not
// fit the LDS beside the block's operands.
#include <type_traits>

#include "scan_tiles.cuh"

namespace muon {
namespace {

using namespace scan;

// A block of Q tokens by 4 Q threads.
template <typename T, int NT, int Q, bool VEC>
__global__ void __launch_bounds__(4 * Q, Q / 64) scan_grad_kernel(ScanGrad A) {
  typedef Ops<T> O;
  typedef typename O::Frag Frag;
  typedef Tile<T, NT> TN;
  typedef Tile<T, kPB> TP;
  typedef Triangle<T, Q / 16> TM;
  constexpr int kThreads = 4 * Q, kTiles = Q / 16, kU = Q / 64, kPieces = O::kRounded;
  // a wave has one of the diagonal's tiles, first, and a run of those below it
  constexpr int kBelow = kTiles * (kTiles - 1) / 2, kMaxTiles = 1 + (kBelow + kTiles - 1) / kTiles;
  // dq and dk: 16-wide blocks of n per wave, groups of waves that share a block's tokens
  constexpr int kBlocks = NT / 16, kNW = kBlocks > kTiles ? kBlocks / kTiles : 1;
  constexpr int kTG = kTiles > kBlocks ? kTiles / kBlocks : 1, kTT = kTiles / kTG;
  // dv: four blocks of value rows, the tokens dealt to kTiles / 4 groups of waves
  constexpr int kZG = kTiles / 4;
  // dS_out [n][p] as the operand of dv goes where v was, if it fits, its second piece where dy was
  constexpr bool kStateInV = NT <= Q;
  // arrays of their own: the compiler may move reads of one across writes to another
  __shared__ __attribute__((aligned(16))) T lq[Q * NT], lk[Q * NT], lv[2 * Q * kPB];   // q; k; v and dy
  __shared__ __attribute__((aligned(16))) T lm[TM::kSize];                                       // (L A)^T [j][i], at the end D^T, then D
  __shared__ Gates<Q> gates[2];
  // by token: row sums of W by column tile (in its own tile, what crosses it there),
  // column sums of L A E by row tile, e^{c_i} q_i . S_in^T dy_i and
  // e^{c_end - c_j} k_j . dS_out^T v_j by block of n
  __shared__ float lsums[4][kTiles * Q];
  // <S_in, dS_out> by wave; over a head's blocks of value rows, by token: its own tile's part of dg, and db; by
  // tile: the sums of the last two of lsums (b_j times the second), and of W by column tile
  __shared__ float lthrough[kTiles], lown[Q], ldb[Q], lfrom[kTiles], lupto[kTiles], lpairs[kTiles * kTiles];
  T* ldy = lv + Q * kPB;
  float *lrow = lsums[0], *lcol = lsums[1], *lqs = lsums[2], *lks = lsums[3];

  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, g4 = lane >> 4;
  const int split = static_cast<int>(blockIdx.x % A.nsplit);
  const long long rest = blockIdx.x / A.nsplit;
  const int grp = static_cast<int>(rest % A.groups);
  const int c = static_cast<int>(rest / A.groups % A.nblocks);
  const long long bi = rest / A.groups / A.nblocks;
  const long long t0 = static_cast<long long>(c) * Q;
  const int rows = A.tokens - t0 < Q ? static_cast<int>(A.tokens - t0) : Q;
  const int per_group = A.heads / A.groups;
  const int per_split = (per_group + A.nsplit - 1) / A.nsplit;
  const int h0 = grp * per_group + split * per_split;
  const int h1 = grp * per_group + (split * per_split + per_split < per_group ? split * per_split + per_split : per_group);
  const int nvirt = (h1 - h0) * A.pblocks;   // (head, block of kPB value components), heads outermost
  const int vheads = A.heads * A.pblocks;
  const auto rows_p_of = [&](int pb) { return A.P - pb * kPB < kPB ? A.P - pb * kPB : kPB; };
  // offset of the states of the i-th of them
  const auto state_at = [&](int i) {
    return ((bi * vheads + h0 * A.pblocks + i) * A.nblocks + c) * static_cast<long long>(kPB * NT);
  };

  TileLoad<T, kPB, Q, kThreads, VEC> tv, tdy;
  float gv[kU], bv[kU];
  // (rows_ and bytes 0: nothing is read and zeros come back, so the last pass needs no branch around its prefetch)
  const auto load_head = [&](int h, int pb, int rows_, int tid) {
    const int lane = tid & 63, rp = rows_p_of(pb);
    const T* vp = static_cast<const T*>(A.v.p) + bi * A.v.sb + h * A.v.sh + t0 * A.v.st + pb * kPB;
    const T* dp = static_cast<const T*>(A.dy.p) + bi * A.dy.sb + h * A.dy.sh + t0 * A.dy.st + pb * kPB;
    tv.load(vp, A.v.st, rows_, rp, tid);
    tdy.load(dp, A.dy.st, rows_, rp, tid);
    const float* gp = static_cast<const float*>(A.g.p) + bi * A.g.sb + h * A.g.sh + t0 * A.g.st;
    const float* bp = A.b.p == nullptr ? gp : static_cast<const float*>(A.b.p) + bi * A.b.sb + h * A.b.sh + t0 * A.b.st;
    const long long bst = A.b.p == nullptr ? 0 : A.b.st;
    if (w == kTiles - 1)
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int t = kU * lane + u, in = t < rows ? t : rows - 1;
        gv[u] = gp[in * A.g.st];
        bv[u] = bp[in * bst];
      }
  };
  // by the last wave, of what load_head has brought
  const auto next_gates = [&](Gates<Q>& G) {
    const int lane = fresh(threadIdx.x) & 63;
#pragma unroll
    for (int u = 0; u < kU; ++u) {   // past the end: no decay, no input
      const bool live = kU * lane + u < rows;
      gv[u] = live ? gv[u] : 0.0f;
      bv[u] = !live ? 0.0f : A.b.p == nullptr ? 1.0f : bv[u];
    }
    write_gates(G, gv, bv, lane, false);
  };
  // the states as operands: row n = n0 + l16, 8 components p = 32 s + 8 g4 + 0..7 (the walk's order, state_offset)
  const int nw0 = (w % (kBlocks / kNW)) * kNW, tg = w / (kBlocks / kNW);
  const auto load_columns = [&](const float* base, int bytes, int lane, f32x4_t (&x)[kNW][kPB / 32][2]) {
    const __amdgpu_buffer_rsrc_t r = rsrc(base, bytes);
#pragma unroll
    for (int b = 0; b < kNW; ++b)
#pragma unroll
      for (int s = 0; s < kPB / 32; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u) x[b][s][u] = load_f32x4(r, (nw0 * (kPB / 32) * 128 + lane) * 16, ((b * (kPB / 32) + s) * 2 + u) * 1024);
  };

  {
    TileLoad<T, NT, Q, kThreads, VEC> tq, tk;
    tq.load(static_cast<const T*>(A.q.p) + bi * A.q.sb + grp * A.q.sh + t0 * A.q.st, A.q.st, rows, A.N, tid);
    tk.load(static_cast<const T*>(A.k.p) + bi * A.k.sb + grp * A.k.sh + t0 * A.k.st, A.k.st, rows, A.N, tid);
    tq.store(lq, tid);
    tk.store(lk, tid);
  }
  f32x4_t x[kNW][kPB / 32][2], y[kNW][kPB / 32][2];
  if (nvirt > 0) {
    load_head(h0, 0, rows, tid);
    load_columns(A.states + state_at(0), kPB * NT * 4, lane, x);
    load_columns(A.dstates + state_at(0), kPB * NT * 4, lane, y);
    if (w == kTiles - 1) next_gates(gates[0]);
  }
  // slots of the sums that no wave writes
  TM::clear_zeros(lm, tid);
  for (int i = tid; i < 4 * kTiles * Q; i += kThreads) lsums[0][i] = 0.0f;
  __syncthreads();

  // A and the sum of L b E, by tile: rows i, columns j
  // (a wave with one tile less repeats its neighbour's first, to the same result, and leaves it out of D)
  const int tile0 = w * kBelow / kTiles, ntile = 1 + (w + 1) * kBelow / kTiles - tile0;
  int trow[kMaxTiles], tcol[kMaxTiles];
  f32x4_t sc[kMaxTiles], dsum[kMaxTiles];
#pragma unroll
  for (int t = 0; t < kMaxTiles; ++t) {
    const int r = t == 0 ? 0 : tile_row(tile0 + t - 1);
    trow[t] = t == 0 ? w : r + 1;
    tcol[t] = t == 0 ? w : tile_col(tile0 + t - 1, r);
    sc[t] = dsum[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int s = 0; s < NT / 32; ++s)
        sc[t] = O::mma(TN::row(lq, 16 * trow[t] + l16, 32 * s + 8 * g4),
                       TN::row(lk, 16 * tcol[t] + l16, 32 * s + 8 * g4), sc[t]);
  }
  // dq^T and dk^T: rows n = 16 (nw0 + b) + 4 g4 + 0..3, column i (j) = 16 (u kTG + tg) + l16
  f32x4_t dq[kNW][kTT], dk[kNW][kTT];
#pragma unroll
  for (int b = 0; b < kNW; ++b)
#pragma unroll
    for (int u = 0; u < kTT; ++u) dq[b][u] = dk[b][u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  float acc_z = 0.0f;   // <S_in, dS_out> over a head's blocks
  for (int i = 0, h = h0, pb = 0; i < nvirt; ++i) {
    const int tid = fresh(threadIdx.x), lane = tid & 63, l16 = lane & 15, g4 = lane >> 4;
    const Gates<Q>& G = gates[i & 1];
    tv.store(lv, tid);
    tdy.store(ldy, tid);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    // The next head's tiles, and below its states, each as soon as their registers
    // are free: issued together they would stall the waves, which can have only so
    // many loads under way (173 -> 151 us).  float32 has half the tiles to load
    // beside eight times the matrix instructions, and gains nothing (37 us against
    // 38 for three sequences of 333 tokens, 8 heads of 64 x 64).
    constexpr bool kEarly = sizeof(T) == 2;
    const bool more = i + 1 < nvirt;
    const int next = more ? i + 1 : i;
    const int next_pb = !more ? pb : pb + 1 < A.pblocks ? pb + 1 : 0, next_h = h + (more && next_pb == 0);
    if constexpr (kEarly) {
      load_head(next_h, next_pb, more ? rows : 0, fresh(threadIdx.x));
      __builtin_amdgcn_sched_barrier(0);
    }

    float cols[kMaxTiles];
#pragma unroll
    for (int t = 0; t < kMaxTiles; ++t) {
      {
        const int it = trow[t], jt = tcol[t];
        f32x4_t e = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kPB / 32; ++s)
          e = O::mma(TP::row(ldy, 16 * it + l16, 32 * s + 8 * g4),
                     TP::row(lv, 16 * jt + l16, 32 * s + 8 * g4), e);
        const int j = 16 * jt + l16, i0 = 16 * it + 4 * g4;
        const float b = G.b[j];
        const f32x4_t d = t == 0 ? between4_diagonal(G, i0, j) : between4_below(G, it, i0, j);
        f32x4_t mm, rs;
        cols[t] = 0.0f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          mm[r] = d[r] * sc[t][r];
          dsum[t][r] = fmaf(d[r] * e[r], b, dsum[t][r]);
          const float we = mm[r] * e[r];
          cols[t] += we;
          rs[r] = we * b;
        }
        TM::store4(lm, TM::tile(it, jt), l16, 4 * g4, mm);
        if (t == 0) {
          // rows from token l16 of the tile on, columns before it
          float c = 0.0f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float before = lanes_before(rs[r]);
            c += 4 * g4 + r >= l16 ? before : 0.0f;
          }
          c = sum_rows4(c, c, c, c);
          if (g4 == 0) lrow[jt * Q + j] = c;
        } else {
          const float row = sum_lanes4(rs[0], rs[1], rs[2], rs[3], l16);
          if (l16 < 4) lrow[jt * Q + i0 + l16] = row;
        }
        settle(dsum[t]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }

    // column sums, four tiles at a time (a wave's last group may name its last tile twice)
#pragma unroll
    for (int t = 0; t < kMaxTiles; t += 4) {
      const int a = t, b = t + 1 < kMaxTiles ? t + 1 : a, c = t + 2 < kMaxTiles ? t + 2 : a, d = t + 3 < kMaxTiles ? t + 3 : a;
      const float sum = sum_rows4(cols[a], cols[b], cols[c], cols[d]);
      const int it = g4 == 0 ? trow[a] : g4 == 1 ? trow[b] : g4 == 2 ? trow[c] : trow[d];
      const int jt = g4 == 0 ? tcol[a] : g4 == 1 ? tcol[b] : g4 == 2 ? tcol[c] : tcol[d];
      lcol[it * Q + 16 * jt + l16] = sum;
    }

    // the states' part of dq, then of dk, and the states' product
    float through = 0.0f;
#pragma unroll
    for (int b = 0; b < kNW; ++b)
#pragma unroll
      for (int s = 0; s < kPB / 32; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) through = fmaf(x[b][s][e / 4][e % 4], y[b][s][e / 4][e % 4], through);
    through = wave_total(through);
    if (lane == 0) lthrough[w] = tg == 0 ? through : 0.0f;
    Frag f[kNW][kPB / 32][O::kSplit];
    const auto split = [&](const f32x4_t (&xs)[kNW][kPB / 32][2]) {
#pragma unroll
      for (int b = 0; b < kNW; ++b)
#pragma unroll
        for (int s = 0; s < kPB / 32; ++s) {
          const f32x4_t a = xs[b][s][0], c = xs[b][s][1];
          const float v[8] = {a[0], a[1], a[2], a[3], c[0], c[1], c[2], c[3]};
          O::split(v, f[b][s]);
        }
    };
    // four token tiles at a time, so that their sums and operands leave room for what stays
    const auto products = [&](auto gated, const T* tile, const T* other, const float* scale, f32x4_t (&out)[kNW][kTT],
                              float* slot) {
      const int lane = fresh(threadIdx.x) & 63, l16 = lane & 15, g4 = lane >> 4;
#pragma unroll
      for (int u0 = 0; u0 < kTT; u0 += 4) {
        float sums[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < kNW; ++b) {
          f32x4_t acc[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) acc[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int s = 0; s < kPB / 32; ++s) {
            Frag d[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) d[u] = TP::row(tile, 16 * ((u0 + u) * kTG + tg) + l16, 32 * s + 8 * g4);
#pragma unroll
            for (int z = O::kSplit - 1; z >= 0; --z)
#pragma unroll
              for (int u = 0; u < 4; ++u) acc[u] = O::mma(f[b][s][z], d[u], acc[u]);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int t = 16 * ((u0 + u) * kTG + tg) + l16;
            const float sv = scale[t], gt = gated ? G.b[t] : 1.0f;
            const f32x4_t ov = TN::load4(other, t, 16 * (nw0 + b) + 4 * g4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float a = decayed(acc[u][r], sv);
              sums[u] = fmaf(a, ov[r], sums[u]);
              out[b][u0 + u][r] = gated ? fmaf(a, gt, out[b][u0 + u][r]) : out[b][u0 + u][r] + a;
            }
            settle(out[b][u0 + u]);
          }
        }
        slot[nw0 / kNW * Q + 16 * ((u0 + g4) * kTG + tg) + l16] = sum_rows4(sums[0], sums[1], sums[2], sums[3]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    split(x);
    if constexpr (kEarly) {
      load_columns(A.states + state_at(next), more ? kPB * NT * 4 : 0, lane, x);
      __builtin_amdgcn_sched_barrier(0);
    }
    products(std::false_type(), ldy, lq, G.first, dq, lqs);
    split(y);
    if constexpr (kEarly) {
      load_columns(A.dstates + state_at(next), more ? kPB * NT * 4 : 0, lane, y);
      __builtin_amdgcn_sched_barrier(0);
    }
    products(std::true_type(), lv, lk, G.last, dk, lks);
    __syncthreads();   // (L A)^T and the sums are written, v is done with
    {
      const int lane = fresh(threadIdx.x) & 63, l16 = lane & 15, g4 = lane >> 4;
      // a piece of dS_out [n][p], as the operand of dv
      const auto store_state = [&](T* tile, int piece) {
#pragma unroll
        for (int b = 0; b < kNW; ++b)
#pragma unroll
          for (int s = 0; s < kPB / 32; ++s) TP::store8(tile, 16 * (nw0 + b) + l16, 32 * s + 8 * g4, f[b][s][piece]);
      };
      if constexpr (kStateInV)
        if (tg == 0) store_state(lv, 0);
      const float* dsp = A.dstates + state_at(i);
      if constexpr (!kEarly) {
        load_head(next_h, next_pb, more ? rows : 0, fresh(threadIdx.x));
        load_columns(A.states + state_at(next), more ? kPB * NT * 4 : 0, lane, x);
        load_columns(A.dstates + state_at(next), more ? kPB * NT * 4 : 0, lane, y);
      }
      __builtin_amdgcn_sched_barrier(0);
      // sums of a token: 16 tokens a wave, one of the four kinds each quarter of it
      {
        const int t = 16 * w + l16;
        const float* src = lsums[g4] + t;
        float part[kTiles], a = 0.0f, own = 0.0f;   // own: of its own tile, of rows and columns
#pragma unroll
        for (int e = 0; e < kTiles; ++e) {
          part[e] = src[e * Q];
          if (e == w && g4 < 2) own = part[e];
          else a += part[e];
        }
        const float b = G.b[t];
        const float cs = __shfl_xor(a, 16, kWave), us = __shfl_xor(a, 32, kWave), ws = __shfl_xor(a, 48, kWave);
        const float cs_own = __shfl_xor(own, 16, kWave);
        // (of use in the first quarter, whose a and own are the rows')
        const float within = own + lanes_from(a + us) + lanes_before(b * (cs + ws)), d = cs_own + cs + ws;
        const float ends = sum_lanes4(us, b * ws, us, b * ws, l16);
        const auto keep = [&](float* p, float v) { *p = pb == 0 ? v : *p + v; };
        if (g4 == 0) {
          keep(lown + t, within);
          keep(ldb + t, d);
          if (l16 < 2) keep((l16 == 0 ? lfrom : lupto) + w, ends);
        }
#pragma unroll
        for (int e = 0; e < kTiles; e += 4) {
          const float pairs = sum_lanes4(part[e], part[e + 1], part[e + 2], part[e + 3], l16);
          if (g4 == 0 && l16 < 4) keep(lpairs + w * kTiles + e + l16, pairs);
        }
      }

      // z^T: rows p = 16 (w % 4) + 4 g4 + 0..3, column j = 16 (kZG u + w / 4) + l16
      f32x4_t z[4], zs[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) z[u] = zs[u] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < Q / 32; ++s) {
        const Frag f = TP::col(ldy, 32 * s, 16 * (w & 3), lane);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int jt = kZG * u + (w >> 2);
          if (s >= kZG * u / 2)   // jt / 2: tiles of tokens before j are zero
#pragma unroll
            for (int e = kPieces - 1; e >= 0; --e) z[u] = O::mma(f, TM::row(lm, e, TM::tile(2 * s + (g4 >> 1), jt), l16, 8 * (g4 & 1)), z[u]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kStateInV) {
        __syncthreads();   // dS_out is written, dy is done with
        if constexpr (kPieces == 2)
          if (tg == 0) store_state(ldy, 1);
      }
      const auto state_product = [&](int s, const auto& f, int pieces) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const Frag kf = TN::row(lk, 16 * (kZG * u + (w >> 2)) + l16, 32 * s + 8 * g4);
#pragma unroll
          for (int e = pieces - 1; e >= 0; --e) zs[u] = O::mma(f[e], kf, zs[u]);
        }
      };
#pragma unroll
      for (int s = 0; s < NT / 32; ++s) {
        if constexpr (kStateInV) {
          const Frag f[1] = {TP::col(lv, 32 * s, 16 * (w & 3), lane)};
          state_product(s, f, 1);
        } else {
          float v[8];
          Frag f[kPieces];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = dsp[state_offset(32 * s + 8 * g4 + e, 16 * (w & 3) + l16)];
          O::split(v, f);
          state_product(s, f, kPieces);
        }
      }
      if constexpr (kStateInV && kPieces == 2) {
        __syncthreads();   // its second piece is written
#pragma unroll
        for (int s = 0; s < NT / 32; ++s) {
          const Frag f[1] = {TP::col(ldy, 32 * s, 16 * (w & 3), lane)};
          state_product(s, f, 1);
        }
      }
      const TileStore<T, VEC> out(static_cast<T*>(A.dv) + ((bi * A.tokens + t0) * A.heads + h) * A.P + pb * kPB,
                                  static_cast<long long>(A.heads) * A.P, rows, rows_p_of(pb));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int j = 16 * (kZG * u + (w >> 2)) + l16;
        out.put(j, 16 * (w & 3) + 4 * g4, (z[u] + decayed(zs[u], G.last[j])) * G.b[j]);
      }
    }
    if constexpr (!kStateInV) __syncthreads();   // the tokens' sums are written

    // the last wave has the next head's gates to prepare, the first one this head's dg
    if (w == kTiles - 1 && more) next_gates(gates[(i + 1) & 1]);
    if (w == 0) {
      const int lane = fresh(threadIdx.x) & 63;
#pragma unroll
      for (int e = 0; e < kTiles; ++e) acc_z += lthrough[e];
      if (pb + 1 == A.pblocks) {
        // what crosses the whole tile of this lane's tokens: tile m's share, then all of them
        const int mine = lane / (kWave / kTiles), m = lane % kTiles;
        float a = m > mine ? lfrom[m] : m < mine ? lupto[m] : 0.0f;
#pragma unroll
        for (int e = 0; e + 2 < kTiles; ++e) a += m > mine && e < mine ? lpairs[m * kTiles + e] : 0.0f;
        a += dpp_f<kDppXor1>(a);
        a += dpp_f<kDppXor2>(a);
        if constexpr (kTiles == 8) a += dpp_f<kDppHalfMirror>(a);
        a += decayed(acc_z, G.end[0]);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int t = kU * lane + u;
          if (t < rows) {
            const long long o = (bi * A.tokens + t0 + t) * A.heads + h;
            A.dg[o] = a + lown[t];
            if (A.db != nullptr) A.db[o] = ldb[t];
          }
        }
        acc_z = 0.0f;
      }
    }
    h = next_h;
    pb = next_pb;
    __syncthreads();   // the tiles, gates and sums are done with
  }

  // D = sum over heads of L b E, as D^T [j][i] for dk, then as D [i][j] for dq
  const auto each_tile = [&](auto store) {
#pragma unroll
    for (int t = 0; t < kMaxTiles; ++t)
      if (t + 1 < kMaxTiles || t < ntile) store(TM::tile(trow[t], tcol[t]), dsum[t]);
  };
  each_tile([&](int tile, const f32x4_t& d) { TM::store4(lm, tile, l16, 4 * g4, d); });
  __syncthreads();
  const int hi = g4 >> 1, lo = 8 * (g4 & 1);
#pragma unroll
  for (int s = 0; s < Q / 32; ++s)
#pragma unroll
    for (int b = 0; b < kNW; ++b) {
      const Frag fq = TN::col(lq, 32 * s, 16 * (nw0 + b), lane);
#pragma unroll
      for (int u = 0; u < kTT; ++u)
        if (s >= u * kTG / 2)   // tokens i before j are zero
#pragma unroll
          for (int e = kPieces - 1; e >= 0; --e) dk[b][u] = O::mma(fq, TM::row(lm, e, TM::tile(2 * s + hi, u * kTG + tg), l16, lo), dk[b][u]);
    }
  __syncthreads();   // D^T is done with
  each_tile([&](int tile, const f32x4_t& d) {
#pragma unroll
    for (int r = 0; r < 4; ++r) TM::store1(lm, tile, 4 * g4 + r, l16, d[r]);
  });
  __syncthreads();
#pragma unroll
  for (int s = 0; s < Q / 32; ++s)
#pragma unroll
    for (int b = 0; b < kNW; ++b) {
      const Frag fk = TN::col(lk, 32 * s, 16 * (nw0 + b), lane);
#pragma unroll
      for (int u = 0; u < kTT; ++u)
        if (s <= (u * kTG + kTG - 1) / 2)
#pragma unroll
          for (int e = kPieces - 1; e >= 0; --e) dq[b][u] = O::mma(fk, TM::row(lm, e, TM::tile(u * kTG + tg, 2 * s + hi), l16, lo), dq[b][u]);
    }
#pragma unroll
  for (int b = 0; b < kNW; ++b) {
    const int n0 = 16 * (nw0 + b);
    const int n = n0 + 4 * g4;
#pragma unroll
    for (int u = 0; u < kTT; ++u) {
      const int t = 16 * (u * kTG + tg) + l16;
      if (t >= rows || n >= A.N) continue;
      const long long o = ((bi * A.tokens + t0 + t) * A.groups + grp) * A.N + n;
      if (A.nsplit > 1) {
        const long long half = static_cast<long long>(A.batch) * A.tokens * A.groups * A.N;
        float* pq = A.parts + (2LL * split) * half + o;
        float* pk = pq + half;
        if (A.N % 4 == 0) {
          *reinterpret_cast<f32x4_t*>(pq) = dq[b][u];
          *reinterpret_cast<f32x4_t*>(pk) = dk[b][u];
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (n + r < A.N) {
              pq[r] = dq[b][u][r];
              pk[r] = dk[b][u][r];
            }
        }
      } else if (A.dkvec) {
        O::store4(static_cast<T*>(A.dq) + o, dq[b][u]);
        O::store4(static_cast<T*>(A.dk) + o, dk[b][u]);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (n + r < A.N) {
            static_cast<T*>(A.dq)[o + r] = O::from_f32(dq[b][u][r]);
            static_cast<T*>(A.dk)[o + r] = O::from_f32(dk[b][u][r]);
          }
      }
    }
  }
}

constexpr int kPartThreads = 256;

// dq and dk out of the head splits' parts, added in order: EACH elements a
// thread, four where they are aligned so (two parts of 16,384 x 128 each, 42 MB:
// 7 us, 11 with one).
template <typename T, int EACH>
__global__ void __launch_bounds__(kPartThreads) scan_parts_kernel(const float* parts, int nsplit, long long half, T* dq, T* dk) {
  const long long i = (static_cast<long long>(blockIdx.x) * kPartThreads + threadIdx.x) * EACH;
  if (i >= 2 * half) return;
  T* out = i < half ? dq + i : dk + (i - half);
  if constexpr (EACH == 4) {
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int u = 0; u < nsplit; ++u) s += *reinterpret_cast<const f32x4_t*>(parts + 2LL * u * half + i);
    Ops<T>::store4(out, s);
  } else {
    float s = 0.0f;
    for (int u = 0; u < nsplit; ++u) s += parts[2LL * u * half + i];
    *out = Ops<T>::from_f32(s);
  }
}

template <typename T, int NT, int Q, bool VEC>
hipError_t grad(const ScanGrad& A, hipStream_t st) {
  const long long items = static_cast<long long>(A.batch) * A.nblocks * A.groups * A.nsplit;
  hipLaunchKernelGGL((scan_grad_kernel<T, NT, Q, VEC>), dim3(static_cast<unsigned>(items)), dim3(4 * Q), 0, st, A);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || A.nsplit == 1) return e;
  const long long half = static_cast<long long>(A.batch) * A.tokens * A.groups * A.N;
  const int each = A.dkvec ? 4 : 1;
  const dim3 parts(static_cast<unsigned>((2 * half / each + kPartThreads - 1) / kPartThreads));
  T *dq = static_cast<T*>(A.dq), *dk = static_cast<T*>(A.dk);
  if (each == 4) hipLaunchKernelGGL((scan_parts_kernel<T, 4>), parts, dim3(kPartThreads), 0, st, A.parts, A.nsplit, half, dq, dk);
  else hipLaunchKernelGGL((scan_parts_kernel<T, 1>), parts, dim3(kPartThreads), 0, st, A.parts, A.nsplit, half, dq, dk);
  return hipGetLastError();
}

template <int NT>
hipError_t grad_bf16(const ScanGrad& A, bool vec, hipStream_t st) {
  if (scan_grad_tokens(true, A.tokens) == 64) return vec ? grad<bf16_t, NT, 64, true>(A, st) : grad<bf16_t, NT, 64, false>(A, st);
  return vec ? grad<bf16_t, NT, 128, true>(A, st) : grad<bf16_t, NT, 128, false>(A, st);
}

}  // namespace

hipError_t launch_scan_grad(const ScanGrad& A, bool vec, bool bf16, hipStream_t st) {
  if (bf16) return A.N <= 64 ? grad_bf16<64>(A, vec, st) : grad_bf16<128>(A, vec, st);
  if (A.N <= 64) return vec ? grad<float, 64, 64, true>(A, st) : grad<float, 64, 64, false>(A, st);
  return vec ? grad<float, 128, 64, true>(A, st) : grad<float, 128, 64, false>(A, st);
}

}  // namespace muon
