// Gradients of the group norm (group_norm.hip).  With a = silu(z), xh = (u - mu) r,
// o = xh w + b and, behind the norm, do = dy (gate before), dy a (after) or
// dy act'(o) (none):
//   t = do w,  du = r (t - mean(t) - xh mean(t xh)),  dw = sum_rows do xh,  db = sum_rows do
//   before: dx = du a, dz = du x a'(z);  after: dx = du, dz = dy o a'(z);  none: dx = du.
// Without centering mean(t) leaves du.
//
// Bound by memory where the gate's exponentials leave it so.  Threads keep the sums of
// dw and db for their columns in registers over all the rows that they walk, with the
// next row's loads in flight, and leave them in the workspace, where a second kernel
// adds them in fixed order: 16,384 bfloat16 rows of 1,536 with a gate take 45 + 5 us
// (252 MB, 5.6 TB/s), 2,062 float32 rows of 24 groups of 75, centered, 20 + 4.
#include "group_norm.cuh"

#include <algorithm>

namespace muon {
namespace {

// As group_plan, but no thread holds four pieces, whose sums and rows fill its registers
// (12,288 bfloat16 rows of 2,048: 49 us by workgroups, 60 by waves with four; 6,144 of
// 4,096 50 either way; 3,145 of 8,000 with a bias 61 and 94).
GroupPlan grad_plan(int w, int elems) {
  const long long p = (static_cast<long long>(w) + elems - 1) / elems;
  if (p <= 3 * 64) return group_plan(w, elems);
  if (p <= 2 * 256) return {256, p <= 256 ? 1 : 2, false};
  if (p <= 2 * 512) return {512, 2, false};
  if (p <= 2 * 1024) return {1024, 2, false};
  return {0, 0, false};
}

// FULL: centered, or the bias's gradient is wanted.  Workgroup (b, s) walks `span`
// adjacent groups, from s span on, of `per` rows at a time, a grid apart (groups that
// share a wave lie side by side in memory), and leaves part[b][2][groups w].
template <typename T, NormGate G, bool FULL, int TPR, int PIECES, bool TINY>
__global__ void __launch_bounds__(group_threads<TPR>()) group_norm_grad_kernel(GroupNormGradLaunch A) {
  constexpr int V = Vec<T>::n, kAll = group_threads<TPR>(), kUnits = kAll / TPR;
  __shared__ float red[kAll / kWave];
  __shared__ float cols[kUnits > 1 ? kUnits * TPR * V : 1];
  const int sub = kUnits == 1 ? 0 : threadIdx.x / TPR, t = threadIdx.x % TPR;
  constexpr bool kShared = TPR < kWave;   // groups share a wave
  const int span = kShared ? A.span : 1, per = kShared ? A.per : kUnits, g0 = blockIdx.y * span;
  const int up = kShared ? sub / span : sub;   // this unit's row
  const bool live = !kShared || (up < per && g0 + sub - up * span < A.groups);
  const int g = kShared ? (live ? g0 + sub - up * span : g0) : g0, c0 = g * A.w;
  const float inv_w = 1.0f / static_cast<float>(A.w);
  // parameters in registers: a load in the loop would wait for the next row's as well
  float wv[PIECES][V], bv[G == kGateBefore ? 1 : PIECES][V], dw[PIECES][V], db[FULL ? PIECES : 1][V];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    if constexpr (G != kGateBefore) {
#pragma unroll
      for (int e = 0; e < V; ++e) bv[i][e] = 0.0f;
      if (A.bias != nullptr) group_param<T, TPR, TINY>(A.bias + c0, i, t, A.w, bv[i]);
    }
    if (A.weight != nullptr) group_param<T, TPR, TINY>(A.weight + c0, i, t, A.w, wv[i]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (A.weight == nullptr) wv[i][e] = 1.0f;
      dw[i][e] = 0.0f;
      if constexpr (FULL) db[i][e] = 0.0f;
    }
  }
  const bool center = FULL && A.mean != nullptr;
  u32x4_t xn[PIECES], gn[PIECES], zn[G == kGateNone ? 1 : PIECES];   // the next row's, as they are loaded
  float mun = 0.0f, rn = 0.0f;
  const auto load_row = [&](long long row) {
    const T* x = static_cast<const T*>(A.x) + row * A.ldx + c0;
    const T* dy = static_cast<const T*>(A.dy) + row * A.lddy + c0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      xn[i] = group_raw<T, TPR, TINY>(x, i, t, A.w);
      gn[i] = group_raw<T, TPR, TINY>(dy, i, t, A.w);
      if constexpr (G != kGateNone) zn[i] = group_raw<T, TPR, TINY>(static_cast<const T*>(A.z) + row * A.ldz + c0, i, t, A.w);
    }
    mun = center ? A.mean[row * A.groups + g] : 0.0f;
    rn = A.rstd[row * A.groups + g];
  };
  const long long step = static_cast<long long>(gridDim.x) * per;
  long long row = live ? static_cast<long long>(blockIdx.x) * per + up : A.rows;
  if (row < A.rows) load_row(row);
  for (; row < A.rows; row += step) {
    // h: xh;  d: do, then t;  k: what dx and dz take du times (before), the gate's slope times dy (after)
    float h[PIECES][V], d[PIECES][V];
    u32x4_t xr[G == kGateBefore ? PIECES : 1], zr[G == kGateNone ? 1 : PIECES];
    const float mu = mun, r = rn;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      asm volatile("" : "+v"(xn[i]), "+v"(gn[i]));   // unpacked here, not where they were loaded, in twice the registers
      unpack<T>(xn[i], h[i]);
      unpack<T>(gn[i], d[i]);
      if constexpr (G == kGateBefore) xr[i] = xn[i];
      if constexpr (G != kGateNone) {
        asm volatile("" : "+v"(zn[i]));
        zr[i] = zn[i];
      }
    }
    load_row(row + step < A.rows ? row + step : row);
    T* dz = G == kGateNone ? nullptr : static_cast<T*>(A.dz) + row * A.lddz + c0;
    float s1 = 0.0f, s2 = 0.0f;
    constexpr bool kKeep = G == kGateBefore && PIECES <= 2;   // there are registers for the gate's sigmoids
    float sig[kKeep ? PIECES : 1][V];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const GroupPiece<T, TPR, TINY> p(i, t, A.w);
      float z[V];
      if constexpr (G != kGateNone) unpack<T>(zr[i], z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (G == kGateBefore) {
          const float s = sigmoid<T>(z[e]);
          h[i][e] *= z[e] * s;
          if constexpr (kKeep) sig[i][e] = s;
        }
        h[i][e] = (h[i][e] - mu) * r;
        if constexpr (G == kGateAfter) {
          const float s = sigmoid<T>(z[e]), dy = d[i][e];
          d[i][e] = dy * (z[e] * s);
          z[e] = dy * fmaf(h[i][e], wv[i][e], bv[i][e]) * silu_slope(z[e], s);
        }
        if (G == kGateNone && A.act == kActSilu) {
          const float o = fmaf(h[i][e], wv[i][e], bv[i][e]);
          d[i][e] *= silu_slope(o, sigmoid<T>(o));
        }
        dw[i][e] = fmaf(d[i][e], h[i][e], dw[i][e]);
        if constexpr (FULL) db[i][e] += d[i][e];
        d[i][e] *= wv[i][e];
        const float c = p.counts(e) ? d[i][e] : 0.0f;
        if constexpr (FULL) s1 += c;
        s2 = fmaf(c, h[i][e], s2);
      }
      if constexpr (G == kGateAfter) group_store<T, TPR, TINY>(dz, i, t, A.w, z);
    }
    asm volatile("" : "+v"(s1), "+v"(s2));   // both summed up before the branch: their terms take no registers across it
    s1 = center ? group_total<TPR>(s1, red) * inv_w : 0.0f;
    s2 = group_total<TPR>(s2, red) * inv_w;
    T* dx = static_cast<T*>(A.dx) + row * A.lddx + c0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) d[i][e] = r * (d[i][e] - s1 - h[i][e] * s2);
      if constexpr (G == kGateBefore) {
        float x[V], z[V];
        unpack<T>(xr[i], x);
        unpack<T>(zr[i], z);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float s;
          if constexpr (kKeep) s = sig[i][e];
          else s = sigmoid<T>(z[e]);
          x[e] *= d[i][e] * silu_slope(z[e], s);
          d[i][e] *= z[e] * s;
        }
        group_store<T, TPR, TINY>(dz, i, t, A.w, x);
      }
      group_store<T, TPR, TINY>(dx, i, t, A.w, d[i]);
    }
  }
  const long long n = static_cast<long long>(A.groups) * A.w;
  const auto leave = [&](auto& acc, int k, float* out) {
    if (out == nullptr) return;   // a sum that nobody asked for
    float* to = (gridDim.x == 1 ? out : A.part + (2LL * blockIdx.x + k) * n) + g0 * A.w;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const GroupPiece<T, TPR, TINY> p(i, t, A.w);
      if constexpr (kUnits == 1) {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (p.counts(e)) to[p.base + e] = acc[i][e];
      } else {
        // the units' sums, in order
        __syncthreads();
#pragma unroll
        for (int e = 0; e < V; ++e) cols[(e * kUnits + sub) * TPR + t] = acc[i][e];
        __syncthreads();
        for (int j = threadIdx.x; j < span * TPR * V; j += kAll) {
          const int s = kShared ? j / (TPR * V) : 0, e = j / TPR % V;
          const GroupPiece<T, TPR, TINY> q(i, j % TPR, A.w);
          float sum = 0.0f;
#pragma unroll 4
          for (int u = 0; u < per; ++u) sum += cols[(e * kUnits + u * span + s) * TPR + j % TPR];
          if (g0 + s < A.groups && q.counts(e)) to[s * A.w + q.base + e] = sum;
        }
      }
    }
  };
  leave(dw, 0, A.dw);
  if constexpr (FULL) leave(db, 1, A.db);
}

// Groups of any width, a workgroup a row at a time; column sums in the workspace
// (each element always by the same thread).
template <typename T, NormGate G>
__global__ void __launch_bounds__(kGroupThreads) group_norm_grad_any_kernel(GroupNormGradLaunch A) {
  __shared__ float red[kGroupThreads / kWave];
  const int g = blockIdx.y, c0 = g * A.w;
  const long long n = static_cast<long long>(A.groups) * A.w;
  const float inv_w = 1.0f / static_cast<float>(A.w);
  float* pw = A.part + 2LL * blockIdx.x * n + c0;
  float* pb = pw + n;
  for (int c = threadIdx.x; c < A.w; c += kGroupThreads) pw[c] = pb[c] = 0.0f;
  for (long long row = blockIdx.x; row < A.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(A.x) + row * A.ldx + c0;
    const T* dy = static_cast<const T*>(A.dy) + row * A.lddy + c0;
    const T* z = G == kGateNone ? nullptr : static_cast<const T*>(A.z) + row * A.ldz + c0;
    T* dx = static_cast<T*>(A.dx) + row * A.lddx + c0;
    T* dz = G == kGateNone ? nullptr : static_cast<T*>(A.dz) + row * A.lddz + c0;
    const float mu = A.mean != nullptr ? A.mean[row * A.groups + g] : 0.0f, r = A.rstd[row * A.groups + g];
    struct At {
      float h, d, o, z, s;   // xh, do, o, the gate and its sigmoid
    };
    const auto at = [&](int c) {
      At v;
      float u = element(x[c]);
      v.d = element(dy[c]);
      v.z = v.s = 0.0f;
      if constexpr (G != kGateNone) {
        v.z = element(z[c]);
        v.s = sigmoid<T>(v.z);
      }
      if constexpr (G == kGateBefore) u *= v.z * v.s;
      v.h = (u - mu) * r;
      v.o = v.h * (A.weight != nullptr ? A.weight[c0 + c] : 1.0f) + (A.bias != nullptr ? A.bias[c0 + c] : 0.0f);
      if constexpr (G == kGateAfter) v.d *= v.z * v.s;
      if (G == kGateNone && A.act == kActSilu) v.d *= silu_slope(v.o, sigmoid<T>(v.o));
      return v;
    };
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < A.w; c += kGroupThreads) {
      const At v = at(c);
      const float t = A.weight != nullptr ? v.d * A.weight[c0 + c] : v.d;
      s1 += t;
      s2 = fmaf(t, v.h, s2);
      pw[c] = fmaf(v.d, v.h, pw[c]);
      pb[c] += v.d;
    }
    s1 = A.mean != nullptr ? block_sum(s1, red) * inv_w : 0.0f;
    s2 = block_sum(s2, red) * inv_w;
    for (int c = threadIdx.x; c < A.w; c += kGroupThreads) {
      const At v = at(c);
      const float t = A.weight != nullptr ? v.d * A.weight[c0 + c] : v.d;
      float o = r * (t - s1 - v.h * s2), k = 0.0f;
      if constexpr (G == kGateBefore) {
        k = o * element(x[c]) * silu_slope(v.z, v.s);
        o *= v.z * v.s;
      }
      if constexpr (G == kGateAfter) k = element(dy[c]) * v.o * silu_slope(v.z, v.s);
      if constexpr (sizeof(T) == 2) {
        dx[c] = f32_to_bf16(o);
        if constexpr (G != kGateNone) dz[c] = f32_to_bf16(k);
      } else {
        dx[c] = o;
        if constexpr (G != kGateNone) dz[c] = k;
      }
    }
  }
}

template <typename T, NormGate G, int TPR, int PIECES, bool TINY = false>
hipError_t run(const GroupNormGradLaunch& A, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(A.parts), static_cast<unsigned>((A.groups + A.span - 1) / A.span)), block(group_threads<TPR>());
  if (A.mean == nullptr && A.db == nullptr)
    hipLaunchKernelGGL((group_norm_grad_kernel<T, G, false, TPR, PIECES, TINY>), grid, block, 0, st, A);
  else
    hipLaunchKernelGGL((group_norm_grad_kernel<T, G, true, TPR, PIECES, TINY>), grid, block, 0, st, A);
  return hipGetLastError();
}

template <typename T, NormGate G>
hipError_t run_any(const GroupNormGradLaunch& A, hipStream_t st) {
  const GroupPlan p = grad_plan(A.w, Vec<T>::n);
  hipError_t e;
  switch (p.threads) {
    case 1: e = p.tiny ? run<T, G, 1, 1, true>(A, st) : run<T, G, 1, 1>(A, st); break;
    case 2: e = run<T, G, 2, 1>(A, st); break;
    case 4:
      if constexpr (sizeof(T) == 2)
        if (p.pieces == 3) {
          e = run<T, G, 4, 3>(A, st);
          break;
        }
      e = run<T, G, 4, 1>(A, st);
      break;
    case 8: e = run<T, G, 8, 1>(A, st); break;
    case 16: e = p.pieces == 1 ? run<T, G, 16, 1>(A, st) : run<T, G, 16, 2>(A, st); break;
    case 64: e = p.pieces == 1 ? run<T, G, 64, 1>(A, st) : p.pieces == 2 ? run<T, G, 64, 2>(A, st) : run<T, G, 64, 3>(A, st); break;
    case 256: e = p.pieces == 1 ? run<T, G, 256, 1>(A, st) : run<T, G, 256, 2>(A, st); break;
    case 512: e = run<T, G, 512, 2>(A, st); break;
    case 1024: e = run<T, G, 1024, 2>(A, st); break;
    default:
      hipLaunchKernelGGL((group_norm_grad_any_kernel<T, G>), dim3(static_cast<unsigned>(A.parts), static_cast<unsigned>(A.groups)), dim3(kGroupThreads), 0, st, A);
      e = hipGetLastError();
  }
  if (e != hipSuccess || (A.parts == 1 && p.threads != 0) || (A.dw == nullptr && A.db == nullptr)) return e;
  return launch_norm_parts(A.part, A.parts, A.groups * A.w, A.dw, A.db, st);
}

template <typename T>
hipError_t run_gate(const GroupNormGradLaunch& A, NormGate gate, hipStream_t st) {
  return gate == kGateBefore ? run_any<T, kGateBefore>(A, st) : gate == kGateAfter ? run_any<T, kGateAfter>(A, st) : run_any<T, kGateNone>(A, st);
}

}  // namespace

// What a workgroup walks, and how many walk the rows of a group: enough to fill the
// chip, eight rows a unit where there are that many.  Groups that share a wave are
// walked side by side (65,536 bfloat16 rows of 24 groups of 16: 48 us, 134 if each
// workgroup walks one group; 24 groups of 64: 49 and 58).  At most 512 workgroups, or 256
// of 512 threads or more: twice as many leave twice the sums (196,608 rows of 128: 47 and
// 51 us).  Waves that walk three pieces of three tensors have enough in flight alone on
// their unit.  With a gate, 256 workgroups and 512, a call in a given workspace: 16,384
// bfloat16 rows of 1,536 channels 49 and 53 us (gate behind 46 and 48, centered 52 and 58),
// of 1,032 42 and 45 (40 and 38, 49 and 54), 49,152 of 1,536 141 and 148; 16,384 float32
// rows of 768 45 and 47, 49,152 140 and 149; 2 to 16 groups of 1,536 5 to 9% less by 256,
// of 768 float32 6 to 8%; up to 4,096 rows nothing.  Only 16,384 float32 rows of 516 and
// 600, centered, take more (40 and 37, 42 and 40).  Without a gate 40 and 34; two pieces
// of 1,024 channels 35 either way, of 768 with the gate after 36 and 32.
GroupGradPlan group_norm_grad_plan(int rows, int groups, int w, bool bf16, bool gated) {
  const GroupPlan p = grad_plan(w, bf16 ? Vec<bf16_t>::n : Vec<float>::n);
  const int units = p.threads == 0 || p.threads >= kGroupThreads ? 1 : kGroupThreads / p.threads;
  GroupGradPlan g{1, units, 1};
  if (p.threads != 0 && p.threads < kWave) {
    const int spans = (groups + units - 1) / units;
    g.span = (groups + spans - 1) / spans;
    g.per = units / g.span;
  }
  const long long most = (p.threads >= 512 || (p.pieces == 3 && p.threads == kWave && gated) ? 256 : 512) / ((groups + g.span - 1) / g.span);
  const long long rows_of = static_cast<long long>(g.per) * (units > 1 ? 8 : 4), want = (rows + rows_of - 1) / rows_of;
  g.parts = static_cast<int>(std::max(1LL, std::min(want, most)));
  return g;
}

hipError_t launch_group_norm_grad(const GroupNormGradLaunch& A, NormGate gate, bool bf16, hipStream_t st) {
  return bf16 ? run_gate<bf16_t>(A, gate, st) : run_gate<float>(A, gate, st);
}

}  // namespace muon
