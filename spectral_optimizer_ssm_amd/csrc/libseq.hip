// libmuon C ABI of the sequence operators (the gated scan and the layer norm;
// declared in include/muon.h): argument validation, workspace planning and
// launches.  Nothing is allocated and nothing synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "host.h"
#include "launch.h"

using namespace muon;

namespace {

Span span(const muon_seq& s, int batch, int tokens, int heads, int width, size_t es) {
  const long long last = (batch - 1) * s.sb + (tokens - 1) * s.st + (heads - 1) * s.sh + width;
  return {static_cast<const char*>(s.p), static_cast<size_t>(last) * es};
}
bool seq_ok(const muon_seq& s, int batch, int tokens, int heads, size_t es) {
  return s.p != nullptr && aligned_to(s.p, es) && s.sb >= 0 && s.st >= 0 && s.sh >= 0 &&
         extent_ok({batch - 1, tokens - 1, heads - 1}, {s.sb, s.st, s.sh});
}
// (the token stride of a single token is free: a row's, so that its loads are whole pieces)
SeqOperand operand(const muon_seq& s, int tokens, int width) { return {s.p, s.sb, tokens == 1 ? width : s.st, s.sh}; }

int check_dims(const muon_scan_args* a) {
  if (a == nullptr) return MUON_EINVAL;
  if (a->dtype != MUON_F32 && a->dtype != MUON_BF16) return MUON_EINVAL;
  if (a->batch < 0 || a->tokens < 0 || a->heads <= 0 || a->groups <= 0 || a->heads % a->groups != 0 || a->P <= 0 || a->N <= 0)
    return MUON_EINVAL;
  if (a->N > kScanMaxN) return MUON_EUNSUPPORTED;
  return MUON_OK;
}
int check_operands(const muon_scan_args* a) {
  const size_t es = dtype_size(a->dtype);
  const auto ok = [a](const muon_seq& s, int heads, size_t es) { return seq_ok(s, a->batch, a->tokens, heads, es); };
  if (!ok(a->v, a->heads, es) || !ok(a->k, a->groups, es) || !ok(a->q, a->groups, es) || !ok(a->log_decay, a->heads, 4)) return MUON_EINVAL;
  if (a->gate.p != nullptr && !ok(a->gate, a->heads, 4)) return MUON_EINVAL;
  if (a->S0 != nullptr && !aligned_to(a->S0, 4)) return MUON_EINVAL;
  return MUON_OK;
}

// The product, or LLONG_MAX where it does not fit.
long long times(long long a, long long b, long long c) {
  long long p;
  return __builtin_mul_overflow(a, b, &p) || __builtin_mul_overflow(p, c, &p) ? LLONG_MAX : p;
}

// Where to stop cutting work: one workgroup of the forward walk or of the
// backward pass for each of 256 compute units (their tiles fill its LDS), and
// 384 walks of the states, which are lighter.  Measured with 24 heads of 64 x
// 128 sharing keys, bfloat16: 16,384 tokens forward take 136 us with up to 256
// walks, 146 with 512 and 171 with 170; 8,191 tokens backward 170 us with up to
// 384, 180 with 256, 178 with 512 and 187 with 768; eight sequences of 2,048
// tokens backward 257 us with 256 workgroups, 351 with 128 and 280 with 512.
constexpr long long kReadFill = 256, kStatesFill = 384, kGradFill = 256;

struct ScanPlan {
  int pblocks, nchunks, nblocks, nseg, seg_chunks, nsplit;   // nblocks: of the backward pass
  size_t states, dstates, seg, seg2, decay, decay2, parts, end;   // workspace offsets
};
// The walk of one sequence is serial, so with few sequences and heads the time
// axis is cut into segments: their totals first, then all of them at once.
// Each token is walked over twice, so segments have to fill otherwise idle
// compute units.  Forward, the second walk is the longer one, and two segments
// already win (96 heads of 4,096 tokens: 152 us in two, 180 in one; 24 heads of
// 16,384: 136 in ten, 692 in one).  For the backward pass both are the same
// walk: 24 heads of 16,384 tokens take 352 us in eight and 445 in one, but 48
// of 8,192 take 327 in four and 316 in one, and 96 of 4,096 take 325 in two and
// 281 in one, so fewer than five are not cut.  A segment has at least kSegChunks
// chunks (24 heads of 2,048 tokens forward: 39 us with four, 47 with eight, and
// no less with two).
constexpr int kSegChunks = 4;

int grad_tokens(const muon_scan_args* a) { return scan_grad_tokens(a->dtype == MUON_BF16, a->tokens); }

int plan_scan(const muon_scan_args* a, bool backward, ScanPlan* p) {
  p->pblocks = (a->P - 1) / kScanRows + 1;
  p->nchunks = static_cast<int>((static_cast<long long>(a->tokens) + kScanChunk - 1) / kScanChunk);
  const int block = grad_tokens(a);
  p->nblocks = static_cast<int>((static_cast<long long>(a->tokens) + block - 1) / block);
  const long long vrows = times(a->batch, a->heads, p->pblocks), groups = times(a->batch, p->nblocks, a->groups);
  if (!launchable(vrows, kScanItemThreads) || (backward && !launchable(groups, kScanItemThreads))) return MUON_EUNSUPPORTED;
  const long long walks = backward ? 2 * vrows : vrows;
  if (a->batch == 0 || a->tokens == 0) {
    p->nseg = p->nsplit = 1;
    p->seg_chunks = 0;
    p->end = kAlign;
    return MUON_OK;
  }
  long long nseg = std::min<long long>((backward ? kStatesFill : kReadFill) / walks, p->nchunks / kSegChunks);
  if (nseg < (backward ? 5 : 2)) nseg = 1;
  p->seg_chunks = static_cast<int>((p->nchunks + nseg - 1) / nseg);
  p->nseg = (p->nchunks + p->seg_chunks - 1) / p->seg_chunks;
  p->nsplit = static_cast<int>(std::min<long long>(a->heads / a->groups, std::max<long long>(1, kGradFill / groups)));
  const int per_split = (a->heads / a->groups + p->nsplit - 1) / p->nsplit;
  p->nsplit = (a->heads / a->groups + per_split - 1) / per_split;   // none without heads
  const size_t tile = static_cast<size_t>(kScanRows) * scan_padded_n(a->N) * sizeof(float);
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, kAlign);
    return at;
  };
  const size_t seg_bytes = p->nseg > 1 ? vrows * p->nseg * tile : 0, decay_bytes = p->nseg > 1 ? vrows * p->nseg * 4 : 0;
  p->seg = take(seg_bytes);
  p->decay = take(decay_bytes);
  if (backward) {
    p->seg2 = take(seg_bytes);
    p->decay2 = take(decay_bytes);
    p->states = take(vrows * p->nblocks * tile);
    p->dstates = take(vrows * p->nblocks * tile);
    const size_t half = static_cast<size_t>(a->batch) * a->tokens * a->groups * a->N;
    p->parts = take(p->nsplit > 1 ? static_cast<size_t>(p->nsplit) * 2 * half * 4 : 0);
  }
  p->end = std::max(off, kAlign);
  return MUON_OK;
}

size_t scan_bytes(const muon_scan_args* a, bool backward) {
  ScanPlan p;
  return check_dims(a) == MUON_OK && plan_scan(a, backward, &p) == MUON_OK ? p.end : 0;
}

ScanWalk walk_of(const muon_scan_args* a, const ScanPlan& p) {
  ScanWalk w{};
  w.x = operand(a->v, a->tokens, a->P);
  w.k = operand(a->k, a->tokens, a->N);
  w.q = operand(a->q, a->tokens, a->N);
  w.g = operand(a->log_decay, a->tokens, 1);
  if (a->gate.p != nullptr) w.b = operand(a->gate, a->tokens, 1);
  w.batch = a->batch; w.tokens = a->tokens; w.heads = a->heads; w.groups = a->groups;
  w.P = a->P; w.N = a->N;
  w.pblocks = p.pblocks; w.nchunks = p.nchunks; w.nseg = p.nseg; w.seg_chunks = p.seg_chunks;
  w.keep_log2 = grad_tokens(a) / kScanChunk / 2; w.nblocks = p.nblocks;
  w.init = a->S0;
  return w;
}

bool walk_vec(const ScanWalk& w, int es) { return scan_vec(w.x, w.P, es) && scan_vec(w.k, w.N, es); }
// Rows of an output, `st` elements apart, take 4-element buffer stores.
bool rows_out(const void* p, long long st, int width, int es) {
  return width % 4 == 0 && aligned_to(p, 4 * es) && st * es * 2 * kScanChunk < (1LL << 31) - 256;
}

size_t state_bytes(const muon_scan_args* a) { return static_cast<size_t>(a->batch) * a->heads * a->P * a->N * 4; }
size_t value_bytes(const muon_scan_args* a) {
  return static_cast<size_t>(a->batch) * a->tokens * a->heads * a->P * dtype_size(a->dtype);
}
Span gate_span(const muon_scan_args* a) {
  return a->gate.p == nullptr ? Span{nullptr, 0} : span(a->gate, a->batch, a->tokens, a->heads, 1, 4);
}

// S_out of a call without tokens is S0 (or zero).
int copy_state(const muon_scan_args* a, float* dst, const float* src, hipStream_t st) {
  const size_t n = state_bytes(a);
  if (dst == nullptr || n == 0) return MUON_OK;
  return launch_copy_f32(src, dst, static_cast<long long>(n / 4), st) == hipSuccess ? MUON_OK : MUON_EHIP;
}

}  // namespace

extern "C" {

size_t muon_gated_scan_workspace_size(const muon_scan_args* args) { return scan_bytes(args, false); }

int muon_gated_scan(const muon_scan_args* a, void* Y, float* S_out, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_dims(a);
  if (rc != MUON_OK) return rc;
  ScanPlan p;
  rc = plan_scan(a, false, &p);
  if (rc != MUON_OK) return rc;
  const int es = static_cast<int>(dtype_size(a->dtype));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (S_out != nullptr && !aligned_to(S_out, 4)) return MUON_EINVAL;
  if (a->batch == 0) return MUON_OK;
  const Span s0 = span(a->S0, state_bytes(a)), so = span(S_out, state_bytes(a));
  if (a->tokens == 0) {
    if ((a->S0 != nullptr && !aligned_to(a->S0, 4)) || clash({so}, {s0})) return MUON_EINVAL;
    return copy_state(a, S_out, a->S0, st);
  }
  rc = check_operands(a);
  if (rc != MUON_OK) return rc;
  if (Y == nullptr || !aligned_to(Y, es)) return MUON_EINVAL;
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < p.end) return MUON_EWORKSPACE;
  const Span v = span(a->v, a->batch, a->tokens, a->heads, a->P, es), k = span(a->k, a->batch, a->tokens, a->groups, a->N, es),
             q = span(a->q, a->batch, a->tokens, a->groups, a->N, es),
             g = span(a->log_decay, a->batch, a->tokens, a->heads, 1, 4);
  if (clash({span(Y, value_bytes(a)), so, span(workspace, p.end)}, {v, k, q, g, gate_span(a), s0})) return MUON_EINVAL;
  ScanWalk w = walk_of(a, p);
  char* ws = static_cast<char*>(workspace);
  w.y = Y;
  w.fin = S_out;
  w.seg_state = p.nseg > 1 ? reinterpret_cast<float*>(ws + p.seg) : nullptr;
  w.seg_decay = p.nseg > 1 ? reinterpret_cast<float*>(ws + p.decay) : nullptr;
  const bool vec = walk_vec(w, es) && scan_vec(w.q, a->N, es) && rows_out(Y, static_cast<long long>(a->heads) * a->P, a->P, es);
  return launch_scan_walk(&w, 1, true, vec, a->dtype == MUON_BF16, st) == hipSuccess ? MUON_OK : MUON_EHIP;
}

size_t muon_gated_scan_backward_workspace_size(const muon_scan_args* args) { return scan_bytes(args, true); }

int muon_gated_scan_backward(const muon_scan_args* a, const muon_seq* dY, const float* dS, void* dV, void* dK, void* dQ,
                             float* dlog_decay, float* dgate, float* dS0, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int rc = check_dims(a);
  if (rc != MUON_OK) return rc;
  ScanPlan p;
  rc = plan_scan(a, true, &p);
  if (rc != MUON_OK) return rc;
  const int es = static_cast<int>(dtype_size(a->dtype));
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if ((dS != nullptr && !aligned_to(dS, 4)) || (dS0 != nullptr && !aligned_to(dS0, 4))) return MUON_EINVAL;
  if (a->batch == 0) return MUON_OK;
  const Span ds = span(dS, state_bytes(a)), ds0 = span(dS0, state_bytes(a)), s0 = span(a->S0, state_bytes(a));
  if (a->tokens == 0) {
    if (clash({ds0}, {ds, s0})) return MUON_EINVAL;
    return copy_state(a, dS0, dS, st);
  }
  rc = check_operands(a);
  if (rc != MUON_OK) return rc;
  if (dY == nullptr || !seq_ok(*dY, a->batch, a->tokens, a->heads, es) || dV == nullptr || dK == nullptr || dQ == nullptr || dlog_decay == nullptr ||
      !aligned_to(dV, es) || !aligned_to(dK, es) || !aligned_to(dQ, es) || !aligned_to(dlog_decay, 4) ||
      (dgate != nullptr && !aligned_to(dgate, 4)))
    return MUON_EINVAL;
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < p.end) return MUON_EWORKSPACE;
  const Span v = span(a->v, a->batch, a->tokens, a->heads, a->P, es), k = span(a->k, a->batch, a->tokens, a->groups, a->N, es),
             q = span(a->q, a->batch, a->tokens, a->groups, a->N, es),
             g = span(a->log_decay, a->batch, a->tokens, a->heads, 1, 4),
             dy = span(*dY, a->batch, a->tokens, a->heads, a->P, es);
  const size_t keys = static_cast<size_t>(a->batch) * a->tokens * a->groups * a->N * es;
  const size_t gates = static_cast<size_t>(a->batch) * a->tokens * a->heads * 4;
  if (clash({span(dV, value_bytes(a)), span(dK, keys), span(dQ, keys), span(dlog_decay, gates), span(dgate, gates), ds0,
             span(workspace, p.end)},
            {v, k, q, g, gate_span(a), s0, dy, ds}))
    return MUON_EINVAL;
  const bool bf16 = a->dtype == MUON_BF16;
  char* ws = static_cast<char*>(workspace);
  const auto at = [&](size_t off) { return reinterpret_cast<float*>(ws + off); };
  // 1. the states before every block and the gradients of the states after it
  ScanWalk w[2] = {walk_of(a, p), walk_of(a, p)};
  w[0].states = at(p.states);
  w[1].x = operand(*dY, a->tokens, a->P);
  w[1].k = w[1].q;
  w[1].reverse = 1;
  w[1].init = dS;
  w[1].fin = dS0;
  w[1].states = at(p.dstates);
  if (p.nseg > 1) {
    w[0].seg_state = at(p.seg);
    w[0].seg_decay = at(p.decay);
    w[1].seg_state = at(p.seg2);
    w[1].seg_decay = at(p.decay2);
  }
  const bool vec = walk_vec(w[0], es) && walk_vec(w[1], es) && rows_out(dV, static_cast<long long>(a->heads) * a->P, a->P, es);
  if (launch_scan_walk(w, 2, false, vec, bf16, st) != hipSuccess) return MUON_EHIP;
  // 2. the gradients, block by block
  ScanGrad r{};
  r.v = w[0].x; r.k = w[0].k; r.q = w[0].q; r.dy = w[1].x; r.g = w[0].g; r.b = w[0].b;
  r.batch = a->batch; r.tokens = a->tokens; r.heads = a->heads; r.groups = a->groups; r.P = a->P; r.N = a->N;
  r.pblocks = p.pblocks; r.nblocks = p.nblocks; r.nsplit = p.nsplit;
  r.dkvec = a->N % 4 == 0 && aligned_to(dK, 4 * es) && aligned_to(dQ, 4 * es);
  r.states = at(p.states);
  r.dstates = at(p.dstates);
  r.dv = dV; r.dk = dK; r.dq = dQ; r.dg = dlog_decay; r.db = dgate;
  r.parts = at(p.parts);
  return launch_scan_grad(r, vec, bf16, st) == hipSuccess ? MUON_OK : MUON_EHIP;
}

int muon_gated_scan_step(const muon_scan_args* a, void* Y, float* S_out, void* stream) {
  int rc = check_dims(a);
  if (rc != MUON_OK) return rc;
  if (a->tokens != 1) return MUON_EINVAL;
  if (!launchable(scan_step_blocks(a->batch, a->heads, a->P), kScanStepThreads)) return MUON_EUNSUPPORTED;
  if (a->batch == 0) return MUON_OK;
  rc = check_operands(a);
  if (rc != MUON_OK) return rc;
  const size_t es = dtype_size(a->dtype);
  // whole 16-byte accesses of the states where their rows are
  const size_t sa = a->N % 4 == 0 ? 16 : 4;
  if (Y == nullptr || !aligned_to(Y, es) || a->S0 == nullptr || S_out == nullptr || !aligned_to(a->S0, sa) || !aligned_to(S_out, sa))
    return MUON_EINVAL;
  const Span v = span(a->v, a->batch, 1, a->heads, a->P, es), k = span(a->k, a->batch, 1, a->groups, a->N, es),
             q = span(a->q, a->batch, 1, a->groups, a->N, es), g = span(a->log_decay, a->batch, 1, a->heads, 1, 4);
  const Span s0 = span(a->S0, state_bytes(a)), so = span(S_out, state_bytes(a));
  const bool in_place = a->S0 == S_out;
  if (clash({span(Y, value_bytes(a)), so}, {v, k, q, g, gate_span(a), in_place ? Span{nullptr, 0} : s0})) return MUON_EINVAL;
  ScanStep s{};
  s.v = operand(a->v, a->tokens, a->P);
  s.k = operand(a->k, a->tokens, a->N);
  s.q = operand(a->q, a->tokens, a->N);
  s.g = operand(a->log_decay, a->tokens, 1);
  if (a->gate.p != nullptr) s.b = operand(a->gate, a->tokens, 1);
  s.batch = a->batch; s.heads = a->heads; s.groups = a->groups; s.P = a->P; s.N = a->N;
  s.y = Y;
  s.S = a->S0;
  s.S_out = S_out;
  return launch_scan_step(s, a->dtype == MUON_BF16, static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_EHIP;
}

// ---------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------
namespace {

int check_norm(int dtype, long long rows, int n) {
  if (dtype != MUON_F32 && dtype != MUON_BF16) return MUON_EINVAL;
  if (rows < 0 || n <= 0) return MUON_EINVAL;
  return rows > INT_MAX || n > kNormMaxN ? MUON_EUNSUPPORTED : MUON_OK;
}
}  // namespace

int muon_layer_norm(const void* X, long long ldx, int dtype, long long rows, int n, const float* weight, const float* bias,
                    float eps, int center, void* Y, long long ldy, float* mean, float* rstd, void* stream) {
  const int rc = check_norm(dtype, rows, n);
  if (rc != MUON_OK) return rc;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || (center != 0 && center != 1) || !rows_ok(rows, n, ldx) || !rows_ok(rows, n, ldy)) return MUON_EINVAL;
  if (rows == 0) return MUON_OK;
  const size_t es = dtype_size(dtype);
  if (X == nullptr || Y == nullptr || !aligned_to(X, es) || !aligned_to(Y, es) || !aligned_to(weight, 4) ||
      !aligned_to(bias, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return MUON_EINVAL;
  const size_t params = static_cast<size_t>(n) * 4, stats = static_cast<size_t>(rows) * 4;
  if (clash({rows_span(Y, rows, n, ldy, es), span(mean, stats), span(rstd, stats)},
            {rows_span(X, rows, n, ldx, es), span(weight, params), span(bias, params)}))
    return MUON_EINVAL;
  NormLaunch A{};
  A.x = X; A.y = Y; A.ldx = ldx; A.ldy = ldy; A.rows = rows; A.n = n; A.center = center;
  A.w = weight; A.bias = bias; A.eps = eps; A.mean = mean; A.rstd = rstd;
  return launch_norm(A, dtype == MUON_BF16, static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_EHIP;
}

size_t muon_layer_norm_backward_workspace_size(long long rows, int n, int dtype) {
  if (check_norm(dtype, rows, n) != MUON_OK) return 0;
  return align_up(static_cast<size_t>(norm_grad_parts(rows, n, dtype == MUON_BF16)) * 2 * n * 4, kAlign);
}

int muon_layer_norm_backward(const void* dY, long long lddy, const void* X, long long ldx, int dtype, long long rows, int n,
                             const float* weight, const float* mean, const float* rstd, void* dX, long long lddx,
                             float* dweight, float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_norm(dtype, rows, n);
  if (rc != MUON_OK) return rc;
  if (!rows_ok(rows, n, lddy) || !rows_ok(rows, n, ldx) || !rows_ok(rows, n, lddx)) return MUON_EINVAL;
  const size_t es = dtype_size(dtype), need = muon_layer_norm_backward_workspace_size(rows, n, dtype);
  if (!aligned_to(dweight, 4) || !aligned_to(dbias, 4) || !aligned_to(weight, 4)) return MUON_EINVAL;
  if (rows == 0 && dweight == nullptr && dbias == nullptr) return MUON_OK;
  if (rows > 0 && (dY == nullptr || X == nullptr || dX == nullptr || rstd == nullptr || !aligned_to(dY, es) || !aligned_to(X, es) ||
                   !aligned_to(dX, es) || !aligned_to(mean, 4) || !aligned_to(rstd, 4)))
    return MUON_EINVAL;
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need) return MUON_EWORKSPACE;
  const size_t params = static_cast<size_t>(n) * 4, stats = static_cast<size_t>(rows) * 4;
  if (clash({rows_span(dX, rows, n, lddx, es), span(dweight, params), span(dbias, params), span(workspace, need)},
            {rows_span(dY, rows, n, lddy, es), rows_span(X, rows, n, ldx, es), span(weight, params), span(mean, stats),
             span(rstd, stats)}))
    return MUON_EINVAL;
  NormGradLaunch A{};
  A.dy = dY; A.x = X; A.dx = dX; A.lddy = lddy; A.ldx = ldx; A.lddx = lddx; A.rows = rows; A.n = n;
  A.w = weight; A.mean = mean; A.rstd = rstd; A.dw = dweight; A.dbias = dbias;
  A.part = static_cast<float*>(workspace);
  A.parts = norm_grad_parts(rows, n, dtype == MUON_BF16);
  return launch_norm_grad(A, dtype == MUON_BF16, static_cast<hipStream_t>(stream)) == hipSuccess ? MUON_OK : MUON_EHIP;
}

}  // extern "C"
