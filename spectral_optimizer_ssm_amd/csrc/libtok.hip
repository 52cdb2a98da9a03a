// libmuon C ABI of the token embedding, the group norm and the token log
// probabilities (declared in include/muon.h): argument validation, workspace
// planning and launches.  Nothing is allocated and nothing synchronises.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "host.h"
#include "launch.h"

using namespace muon;

namespace {

constexpr int kMaxTokens = 1 << 30, kEmbedMaxN = 1 << 21;
// Elements of a tensor: no memory holds more, and every grid over that many fits its two dimensions.
constexpr long long kMaxElements = 1LL << 40;

bool known(int dtype) { return dtype == MUON_F32 || dtype == MUON_BF16; }
int launched(hipError_t e) { return e == hipSuccess ? MUON_OK : MUON_EHIP; }

bool ids_ok(const muon_ids* a, long long tokens) {
  if (a == nullptr || a->p == nullptr || (a->bits != 32 && a->bits != 64) || !aligned_to(a->p, a->bits / 8)) return false;
  if (a->run < 1 || a->stride < 0 || a->step < 0) return false;
  return extent_ok({(tokens - 1) / a->run, std::min(tokens, a->run) - 1}, {a->stride, a->step});
}
Span ids_span(const muon_ids& a, long long tokens) {
  const long long last = (tokens - 1) / a.run * a.stride + (std::min(tokens, a.run) - 1) * a.step;
  return span(a.p, static_cast<size_t>(last + 1) * (a.bits / 8));
}
// t / run as a product: exact for t < 2^31 (with l the bits of run - 1, the factor
// 2^(31 + l) / run, rounded up, is off by at most run of 2^(31 + l)).
void divide_by(long long run, IdsOperand* o) {
  const int l = 64 - __builtin_clzll(static_cast<unsigned long long>(run - 1));   // run > 1
  o->run = static_cast<uint32_t>(run);
  o->magic = static_cast<uint32_t>((1ULL << (31 + l)) / static_cast<unsigned long long>(run) + 1);
  o->shift = l - 1;
}
IdsOperand ids_operand(const muon_ids& a, long long tokens) {
  IdsOperand o{};
  o.p = a.p;
  o.wide = a.bits == 64;
  o.stride = a.stride;
  o.step = a.step;
  if (a.run >= tokens) return o;          // one run: the quotient is 0
  if (a.run == 1) {                       // a run for each token: their stride is the step
    o.step = a.stride;
    return o;
  }
  divide_by(a.run, &o);
  return o;
}

// ---------------------------------------------------------------------------
// embedding
// ---------------------------------------------------------------------------
int check_embed(int table_dtype, int dtype, long long tokens, int vocab, int n) {
  if (!known(table_dtype) || !known(dtype) || tokens < 0 || vocab <= 0 || n <= 0) return MUON_EINVAL;
  if (tokens > kMaxTokens || vocab > kMaxTokens || n > kEmbedMaxN) return MUON_EUNSUPPORTED;
  return tokens * n > kMaxElements || static_cast<long long>(vocab) * n > kMaxElements ? MUON_EUNSUPPORTED : MUON_OK;
}

struct EmbedPlan {
  size_t sorted, part, map, table, end;
  int range;
};
EmbedPlan plan_embed(long long tokens, int vocab, int n) {
  EmbedPlan p;
  const int chunk = embed_grad_chunk(static_cast<uint32_t>(tokens));
  const size_t chunks = static_cast<size_t>((tokens + chunk - 1) / chunk);
  p.sorted = kAlign;   // behind the count
  p.part = p.sorted + align_up(static_cast<size_t>(tokens) * 8, kAlign);
  p.map = p.part + align_up(chunks * 2 * n * 4, kAlign);
  const EmbedMapSizes m = embed_map_sizes(static_cast<uint32_t>(tokens), vocab);
  p.table = p.map + align_up(m.map, kAlign);
  p.end = p.table + align_up(m.table, kAlign);
  p.range = m.range;
  return p;
}

// ---------------------------------------------------------------------------
// group norm
// ---------------------------------------------------------------------------
int check_group_norm(int dtype, long long rows, int groups, int width) {
  if (!known(dtype) || rows < 0 || groups <= 0 || width <= 0) return MUON_EINVAL;
  const long long n = static_cast<long long>(groups) * width;
  if (groups > 65535 || n > kNormMaxN || rows > INT_MAX || rows * groups > INT_MAX) return MUON_EUNSUPPORTED;
  return MUON_OK;
}
bool gated(int gate) { return gate == MUON_GATE_BEFORE || gate == MUON_GATE_AFTER; }
NormGate gate_of(int gate) { return gate == MUON_GATE_BEFORE ? kGateBefore : gate == MUON_GATE_AFTER ? kGateAfter : kGateNone; }
int act_of(int gate) { return gate == MUON_ACT_SILU ? kActSilu : kActNone; }

// ---------------------------------------------------------------------------
// log probabilities
// ---------------------------------------------------------------------------
int check_logp(int dtype, long long rows, int vocab, int top) {
  if (!known(dtype) || rows < 0 || vocab <= 0 || top < 0) return MUON_EINVAL;
  return rows > INT_MAX || vocab > kNormMaxN || top > kLogpMaxTop || rows * vocab > kMaxElements ? MUON_EUNSUPPORTED : MUON_OK;
}
struct LogpPlan {
  int splits;
  size_t ranks, end;
};
LogpPlan plan_logp(long long rows, int vocab, int dtype, int top) {
  LogpPlan p;
  p.splits = logp_splits(rows, vocab, dtype == MUON_BF16);
  const size_t parts = p.splits > 1 ? static_cast<size_t>(rows) * p.splits : 0;
  p.ranks = align_up(parts * 3 * 4, kAlign);
  p.end = std::max(p.ranks + align_up(parts * top * 8, kAlign), kAlign);
  return p;
}
// The kernels' exponents are in base 2: their factor has to be finite too.
bool temper_ok(float scale) { return scale > 0.0f && std::isfinite(scale * 1.44269504f); }
bool strided_ok(const float* p, long long rows, long long stride) {
  return aligned_to(p, 4) && stride >= 0 && extent_ok({rows - 1}, {stride});
}
Span strided_span(const float* p, long long rows, long long stride) {
  return span(p, static_cast<size_t>((rows - 1) * stride + 1) * 4);
}

}  // namespace

extern "C" {

int muon_embedding(const void* table, int table_dtype, long long ldt, int vocab, int n, const muon_ids* ids,
                   long long tokens, float scale, void* Y, int dtype, long long ldy, void* stream) {
  const int rc = check_embed(table_dtype, dtype, tokens, vocab, n);
  if (rc != MUON_OK) return rc;
  if (!std::isfinite(scale) || !rows_ok(vocab, n, ldt) || !rows_ok(tokens, n, ldy)) return MUON_EINVAL;
  if (tokens == 0) return MUON_OK;
  const size_t et = dtype_size(table_dtype), es = dtype_size(dtype);
  if (table == nullptr || Y == nullptr || !aligned_to(table, et) || !aligned_to(Y, es) || !ids_ok(ids, tokens)) return MUON_EINVAL;
  if (clash({rows_span(Y, tokens, n, ldy, es)}, {rows_span(table, vocab, n, ldt, et), ids_span(*ids, tokens)})) return MUON_EINVAL;
  EmbedLaunch A{};
  A.table = table; A.y = Y; A.ids = ids_operand(*ids, tokens); A.ldt = ldt; A.ldy = ldy;
  A.tokens = static_cast<uint32_t>(tokens); A.vocab = vocab; A.n = n; A.scale = scale;
  return launched(launch_embed(A, table_dtype == MUON_BF16, dtype == MUON_BF16, static_cast<hipStream_t>(stream)));
}

size_t muon_embedding_backward_workspace_size(long long tokens, int vocab, int n) {
  return check_embed(MUON_F32, MUON_F32, tokens, vocab, n) == MUON_OK ? plan_embed(tokens, vocab, n).end : 0;
}

int muon_embedding_backward(const void* dY, int dtype, long long lddy, const muon_ids* ids, long long tokens, float scale,
                            int vocab, int n, void* dtable, int table_dtype, int accumulate, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const int rc = check_embed(table_dtype, dtype, tokens, vocab, n);
  if (rc != MUON_OK) return rc;
  if (!std::isfinite(scale) || (accumulate != 0 && accumulate != 1) || (accumulate == 1 && table_dtype != MUON_F32)) return MUON_EINVAL;
  const size_t es = dtype_size(dtype), et = dtype_size(table_dtype), bytes = static_cast<size_t>(vocab) * n * et;
  if (!rows_ok(tokens, n, lddy) || dtable == nullptr || !aligned_to(dtable, et)) return MUON_EINVAL;
  if (tokens > 0 && (dY == nullptr || !aligned_to(dY, es) || !ids_ok(ids, tokens))) return MUON_EINVAL;
  const EmbedPlan p = plan_embed(tokens, vocab, n);
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < p.end) return MUON_EWORKSPACE;
  if (tokens > 0 ? clash({span(dtable, bytes), span(workspace, p.end)}, {rows_span(dY, tokens, n, lddy, es), ids_span(*ids, tokens)})
                 : clash({span(dtable, bytes), span(workspace, p.end)}, {}))
    return MUON_EINVAL;
  if (tokens == 0 && accumulate) return MUON_OK;
  EmbedGradLaunch A{};
  char* ws = static_cast<char*>(workspace);
  A.dy = dY; A.dtable = dtable; A.lddy = lddy; A.tokens = static_cast<uint32_t>(tokens); A.vocab = vocab; A.n = n;
  A.accumulate = accumulate; A.scale = scale;
  if (tokens > 0) A.ids = ids_operand(*ids, tokens);
  A.count = reinterpret_cast<int*>(ws);
  A.sorted = reinterpret_cast<int2*>(ws + p.sorted);
  A.part = reinterpret_cast<float*>(ws + p.part);
  A.map = reinterpret_cast<uint16_t*>(ws + p.map);
  A.table = reinterpret_cast<int*>(ws + p.table);
  if (p.range > 1) divide_by(p.range, &A.by_range);
  return launched(launch_embed_grad(A, dtype == MUON_BF16, table_dtype == MUON_BF16, static_cast<hipStream_t>(stream)));
}

int muon_group_norm(const void* X, long long ldx, const void* Z, long long ldz, int dtype, long long rows, int groups, int width,
                    const float* weight, const float* bias, float eps, int center, int gate, void* Y, long long ldy, float* mean,
                    float* rstd, void* stream) {
  const int rc = check_group_norm(dtype, rows, groups, width);
  if (rc != MUON_OK) return rc;
  const int n = groups * width;
  if (!(eps >= 0.0f) || !std::isfinite(eps) || (center != 0 && center != 1) || gate < MUON_GATE_BEFORE || gate > MUON_ACT_NONE ||
      !rows_ok(rows, n, ldx) || !rows_ok(rows, n, ldy) || (gated(gate) && !rows_ok(rows, n, ldz)) || (!gated(gate) && Z != nullptr))
    return MUON_EINVAL;
  if (rows == 0) return MUON_OK;
  const size_t es = dtype_size(dtype);
  if (X == nullptr || Y == nullptr || (gated(gate) && Z == nullptr) || !aligned_to(X, es) || !aligned_to(Z, es) || !aligned_to(Y, es) ||
      !aligned_to(weight, 4) || !aligned_to(bias, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return MUON_EINVAL;
  const size_t params = static_cast<size_t>(n) * 4, stats = static_cast<size_t>(rows) * groups * 4;
  if (clash({rows_span(Y, rows, n, ldy, es), span(mean, stats), span(rstd, stats)},
            {rows_span(X, rows, n, ldx, es), rows_span(Z, rows, n, ldz, es), span(weight, params), span(bias, params)}))
    return MUON_EINVAL;
  GroupNormLaunch A{};
  A.x = X; A.z = Z; A.y = Y; A.ldx = ldx; A.ldz = ldz; A.ldy = ldy;
  A.rows = static_cast<int>(rows); A.groups = groups; A.w = width; A.center = center; A.act = act_of(gate);
  A.weight = weight; A.bias = bias; A.eps = eps; A.mean = mean; A.rstd = rstd;
  return launched(launch_group_norm(A, gate_of(gate), dtype == MUON_BF16, static_cast<hipStream_t>(stream)));
}

size_t muon_group_norm_backward_workspace_size(long long rows, int groups, int width, int dtype) {
  if (check_group_norm(dtype, rows, groups, width) != MUON_OK) return 0;
  const size_t parts = group_norm_grad_plan(static_cast<int>(rows), groups, width, dtype == MUON_BF16, false).parts;   // as many as with a gate, or more
  return align_up(parts * 2 * groups * width * 4, kAlign);
}

int muon_group_norm_backward(const void* dY, long long lddy, const void* X, long long ldx, const void* Z, long long ldz, int dtype,
                             long long rows, int groups, int width, const float* weight, const float* bias, const float* mean,
                             const float* rstd, int gate, void* dX, long long lddx, void* dZ, long long lddz, float* dweight,
                             float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_group_norm(dtype, rows, groups, width);
  if (rc != MUON_OK) return rc;
  const int n = groups * width;
  if (gate < MUON_GATE_BEFORE || gate > MUON_ACT_NONE || !rows_ok(rows, n, lddy) || !rows_ok(rows, n, ldx) || !rows_ok(rows, n, lddx) ||
      (gated(gate) && (!rows_ok(rows, n, ldz) || !rows_ok(rows, n, lddz))) || (!gated(gate) && (Z != nullptr || dZ != nullptr)))
    return MUON_EINVAL;
  const size_t es = dtype_size(dtype), need = muon_group_norm_backward_workspace_size(rows, groups, width, dtype);
  if (!aligned_to(dweight, 4) || !aligned_to(dbias, 4) || !aligned_to(weight, 4) || !aligned_to(bias, 4)) return MUON_EINVAL;
  if (rows == 0 && dweight == nullptr && dbias == nullptr) return MUON_OK;
  if (rows > 0 && (dY == nullptr || X == nullptr || dX == nullptr || rstd == nullptr || (gated(gate) && (Z == nullptr || dZ == nullptr)) ||
                   !aligned_to(dY, es) || !aligned_to(X, es) || !aligned_to(Z, es) || !aligned_to(dX, es) || !aligned_to(dZ, es) ||
                   !aligned_to(mean, 4) || !aligned_to(rstd, 4)))
    return MUON_EINVAL;
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < need) return MUON_EWORKSPACE;
  const size_t params = static_cast<size_t>(n) * 4, stats = static_cast<size_t>(rows) * groups * 4;
  if (clash({rows_span(dX, rows, n, lddx, es), rows_span(dZ, rows, n, lddz, es), span(dweight, params), span(dbias, params),
             span(workspace, need)},
            {rows_span(dY, rows, n, lddy, es), rows_span(X, rows, n, ldx, es), rows_span(Z, rows, n, ldz, es), span(weight, params),
             span(bias, params), span(mean, stats), span(rstd, stats)}))
    return MUON_EINVAL;
  GroupNormGradLaunch A{};
  A.dy = dY; A.x = X; A.z = Z; A.dx = dX; A.dz = dZ;
  A.lddy = lddy; A.ldx = ldx; A.ldz = ldz; A.lddx = lddx; A.lddz = lddz;
  A.rows = static_cast<int>(rows); A.groups = groups; A.w = width; A.act = act_of(gate);
  A.weight = weight; A.bias = bias; A.mean = mean; A.rstd = rstd; A.dw = dweight; A.db = dbias;
  A.part = static_cast<float*>(workspace);
  const GroupGradPlan p = group_norm_grad_plan(A.rows, groups, width, dtype == MUON_BF16, gated(gate));
  A.parts = p.parts; A.span = p.span; A.per = p.per;
  return launched(launch_group_norm_grad(A, gate_of(gate), dtype == MUON_BF16, static_cast<hipStream_t>(stream)));
}

size_t muon_token_logprobs_workspace_size(long long rows, int vocab, int dtype, int top) {
  return check_logp(dtype, rows, vocab, top) == MUON_OK ? plan_logp(rows, vocab, dtype, top).end : 0;
}

int muon_token_logprobs(const void* X, long long ldx, int dtype, long long rows, int vocab, float scale, const muon_ids* tokens,
                        float* logprobs, float* entropy, float* stats, int top, int* top_ids, float* top_logprobs, void* workspace,
                        size_t workspace_bytes, void* stream) {
  const int rc = check_logp(dtype, rows, vocab, top);
  if (rc != MUON_OK) return rc;
  if (!temper_ok(scale) || !rows_ok(rows, vocab, ldx)) return MUON_EINVAL;
  if (rows == 0) return MUON_OK;
  const size_t es = dtype_size(dtype), per = static_cast<size_t>(rows) * 4;
  if (X == nullptr || !aligned_to(X, es) || !aligned_to(logprobs, 4) || !aligned_to(entropy, 4) || !aligned_to(stats, 4) ||
      !aligned_to(top_ids, 4) || !aligned_to(top_logprobs, 4) || (tokens != nullptr && !ids_ok(tokens, rows)) ||
      (logprobs != nullptr && tokens == nullptr) || (top > 0) != (top_ids != nullptr) || (top > 0) != (top_logprobs != nullptr))
    return MUON_EINVAL;
  const LogpPlan p = plan_logp(rows, vocab, dtype, top);
  if (workspace == nullptr || !aligned16(workspace) || workspace_bytes < p.end) return MUON_EWORKSPACE;
  if (clash({span(logprobs, per), span(entropy, per), span(stats, 2 * per), span(top_ids, top * per), span(top_logprobs, top * per),
             span(workspace, p.end)},
            {rows_span(X, rows, vocab, ldx, es), tokens != nullptr ? ids_span(*tokens, rows) : Span{nullptr, 0}}))
    return MUON_EINVAL;
  LogpLaunch A{};
  A.x = X; A.ldx = ldx; A.rows = rows; A.vocab = vocab; A.top = top; A.splits = p.splits; A.scale = scale;
  if (tokens != nullptr) A.ids = ids_operand(*tokens, rows);
  A.logp = logprobs; A.entropy = entropy; A.stats = stats; A.top_ids = top_ids; A.top_logp = top_logprobs;
  char* ws = static_cast<char*>(workspace);
  A.part = reinterpret_cast<float*>(ws);
  A.ranks = reinterpret_cast<unsigned long long*>(ws + p.ranks);
  return launched(launch_logp(A, dtype == MUON_BF16, static_cast<hipStream_t>(stream)));
}

int muon_token_logprobs_backward(const void* X, long long ldx, int dtype, long long rows, int vocab, float scale,
                                 const muon_ids* tokens, const float* stats, const float* dlogprobs, long long sdlp,
                                 const float* entropy, const float* dentropy, long long sdh, void* dX, long long lddx, void* stream) {
  const int rc = check_logp(dtype, rows, vocab, 0);
  if (rc != MUON_OK) return rc;
  if (!temper_ok(scale) || !rows_ok(rows, vocab, ldx) || !rows_ok(rows, vocab, lddx)) return MUON_EINVAL;
  if (rows == 0) return MUON_OK;
  const size_t es = dtype_size(dtype), per = static_cast<size_t>(rows) * 4;
  if (X == nullptr || dX == nullptr || stats == nullptr || !aligned_to(X, es) || !aligned_to(dX, es) || !aligned_to(stats, 4) ||
      !aligned_to(entropy, 4) || (tokens != nullptr && !ids_ok(tokens, rows)) || (dlogprobs != nullptr && tokens == nullptr) ||
      (dentropy != nullptr && entropy == nullptr) || (dlogprobs != nullptr && !strided_ok(dlogprobs, rows, sdlp)) ||
      (dentropy != nullptr && !strided_ok(dentropy, rows, sdh)))
    return MUON_EINVAL;
  const Span none{nullptr, 0};
  const bool in_place = X == dX && ldx == lddx;
  if (clash({rows_span(dX, rows, vocab, lddx, es)},
            {in_place ? none : rows_span(X, rows, vocab, ldx, es), tokens != nullptr ? ids_span(*tokens, rows) : none,
             span(stats, 2 * per), dlogprobs != nullptr ? strided_span(dlogprobs, rows, sdlp) : none,
             dentropy != nullptr ? strided_span(dentropy, rows, sdh) : none, dentropy != nullptr ? span(entropy, per) : none}))
    return MUON_EINVAL;
  LogpGradLaunch A{};
  A.x = X; A.dx = dX; A.ldx = ldx; A.lddx = lddx; A.rows = rows; A.vocab = vocab; A.scale = scale;
  if (tokens != nullptr) A.ids = ids_operand(*tokens, rows);
  A.stats = stats; A.dlogp = dlogprobs; A.dentropy = dentropy; A.entropy = entropy; A.sdlogp = sdlp; A.sdentropy = sdh;
  return launched(launch_logp_grad(A, dtype == MUON_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
