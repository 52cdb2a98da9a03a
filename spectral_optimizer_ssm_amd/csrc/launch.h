// Internal interface between the C-ABI host code and the kernel launchers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace muon {

// Fused momentum / Nesterov / Frobenius-partials pass (one launch covers up to
// kMaxTable matrices of one shape group).
struct MomentumLaunch {
  PtrTable G;          // user gradients (m x n)
  MutPtrTable M;       // user momentum (m x n, float), entries may be null: U = G
  void* X;             // oriented iterate of the first matrix, s_pad x ld
  long long xstride;   // elements between consecutive matrices of X
  int m, n, s_pad, ld, count, P;
  int ldg;             // row stride of G (elements, >= n); M is contiguous (n)
  bool tall, grad_bf16, x_bf16;
  float beta;
  int nesterov;
  float* partials;     // [count][P] sums of squares
};

struct ApplyLaunch {
  const void* X;       // final iterate (oriented), s_pad x ld
  long long xstride;
  int m, n, ld, count;
  int ldo;             // row stride of O (elements, >= n); W is contiguous (n)
  bool tall, x_bf16;
  MutPtrTable W;       // entries may be null (no apply)
  MutPtrTable O;       // entries may be null (no copy-out); element type = X's
  const float* partials;  // non-null: scale by 1/(nu+eps) (zero Newton-Schulz steps)
  int P;
  float eps;
  float neg_lr_scale;
  // spectral cap (cap_part null: none): O <- O - gamma u v^T with
  // c = sum of the cap_P partials, gamma = c if sigma >= cap and c < 0, else 0
  const float* cap_part;
  int cap_P;
  const float* cap_sigma;
  float cap;
  PtrTable cu, cv;     // u (m floats), v (n floats) per matrix
};

// Spectral cap: partials of u^T O v over the oriented final iterate.
struct CapCoefLaunch {
  const void* X;       // [count][s_pad][ld], bf16 or float
  long long xstride;
  int s, l, ld, count;
  bool tall;           // X = O^T
  PtrTable u, v;       // float[m], float[n] per matrix
  float* part;         // [count][P]
  int P;
};
int cap_coef_blocks(int s);
hipError_t launch_cap_coef(const CapCoefLaunch& L, bool x_bf16, hipStream_t st);

// One simultaneous power step on the updated weights.
struct PowerLaunch {
  PtrTable W;          // float m x n per matrix
  MutPtrTable u, v;    // in: current estimates; out: the next ones
  float* sigma;        // [count]: ||W v||
  float* ybuf;         // [count][m]   W v
  float* zbuf;         // [count][n]   W^T u
  float* zpart;        // [count][nrc][n] partials of W^T u over row blocks
  float* ynorm;        // [count][nrc] partial sums of (W v)_r^2
  float* znorm;        // [count][ncb] partial sums of (W^T u)_j^2
  int m, n, count, nrc, ncb;
};
int power_row_blocks(int m);
int power_col_blocks(int n);
hipError_t launch_power_step(const PowerLaunch& L, hipStream_t st);

// One batched Newton-Schulz GEMM over `count` matrices of one shape, laid out
// contiguously: X [count][s_pad][ld], A [count][s_pad][s_pad].
struct NsGemmLaunch {
  const void* X;       // iterate in
  void* Y;             // iterate out (combine only)
  void* A;             // Gram matrix (out for gram, in for combine)
  long long xstride, astride;
  int s_pad, ld, count;
  // step-1 normalisation folded into the epilogues: when partials is non-null
  // the Gram scales by inv^2 and the combine multiplies alpha, beta by inv,
  // with inv = 1 / (sqrt(sum of partials) + eps).
  const float* partials;
  int P;
  float eps;
  float alpha, beta;   // combine coefficients (a, b)
};

int momentum_blocks_per_matrix(bool tall, int s_pad, int ld);
hipError_t launch_momentum(const MomentumLaunch& L, hipStream_t st);
hipError_t launch_apply(const ApplyLaunch& L, hipStream_t st);
hipError_t launch_norms(const float* partials, int P, int count, float* out, hipStream_t st);
// flag = 1 if any of the n partial sums of squares is not finite, else 0
// (one workgroup; a plain store)
hipError_t launch_flags(const float* partials, long long n, unsigned* flag, hipStream_t st);

// bf16 matrix-core path.  One launch covers up to kMaxSeg shape groups
// (segments) of one Newton-Schulz step.
constexpr int kTileS = 256;   // s_pad multiple for the bf16 tiled path
constexpr int kTileL = 256;   // ld multiple for the bf16 tiled path
constexpr int kMaxSeg = 4;
struct GemmSeg {
  const bf16_t* X;     // iterate in  [count][s_pad][ld]
  bf16_t* Y;           // iterate out (combine)
  bf16_t* A;           // Gram out 1 / combine's left operand  [count][s_pad][s_pad]
  bf16_t* A2;          // Gram out 2 (null: none)
  long long xstride, astride;
  int s_pad, ld, kdim, count, tiles_per_mat;
  // Gram outputs: A = a inv^pa I + b inv^pb X X^T and A2 = a2 I + b2 A (from
  // A's rounded values), inv = 1 / (sqrt(sum of partials) + eps), or 1 when
  // partials is null.
  const float* partials;
  int P;
  float eps;
  float a, b, a2, b2;
  int pa, pb;
  // Combine with the apply fused (the final product of the iteration): Y is
  // not written; with o the bf16 rounding of the result at (i, k) of the
  // oriented iterate (i < s, k < l), matrix z of the segment updates
  // W = GemmArgs.W[tab0 + z] (m x n float32, entry (i, k) wide, (k, i) tall)
  // to fmaf(neg_lr_scale, o, W) and stores o to GemmArgs.O[tab0 + z]
  // (m x n bf16); null table entries skip that output.
  int fuse;
  int tab0, m, n, s, l, tall;
  float neg_lr_scale;
};
struct GemmArgs {
  GemmSeg seg[kMaxSeg];
  int nseg;
  MutPtrTable W, O;    // fused apply: per-matrix outputs of the segments
};
int combine_tiles_per_matrix(int s_pad, int ld);
hipError_t launch_combine_bf16(const GemmArgs& G, hipStream_t st);

// Products L R^T whose result is symmetric: the Gram X X^T (L = R = X, the
// iterate), and products of two symmetric, commuting s_pad x s_pad bf16
// matrices (polynomials in the same Gram matrix, where R^T = R):
// O1 = a1 inv^pa I + b1 inv^pb L R and (optional) O2 = a2 I + b2 O1 from
// O1's rounded values.  Only tiles on or above the diagonal are computed;
// each is stored in place and mirrored.
struct SymSeg {
  const bf16_t* L;     // left factor   [count][s_pad][ld], contraction over kdim columns
  const bf16_t* R;     // right factor  (may equal L)
  bf16_t* O1;          // [count][s_pad][s_pad]
  bf16_t* O2;          // null: none
  long long stride;    // elements between consecutive outputs
  long long in_stride; // elements between consecutive operands
  int ld, kdim;        // operand row stride; contraction length (multiple of 32)
  int s_pad, count, tiles_per_mat;
  const float* partials;
  int P;
  float eps;
  float a1, b1, a2, b2;
  int pa, pb;
  int zip_next;        // 1: the next segment has the same count and s_pad and
                       // runs matrix by matrix together with this one
  int tile;            // 0: symprod_tile(s_pad); else 128 or 192 (dividing s_pad)
  float* F;            // non-null: O1 = a1 inv^pa I + b1 inv^pb L R as float32 here
                       // [count][s_pad][s_pad] (stride), exactly symmetric; O1, O2 unused
  int tri_in;          // 1: L and R hold only their upper block triangle (tile-sized
                       // blocks on and above the diagonal); the others are read transposed
  int tri_out;         // 1: O1 and O2 get only their upper block triangle
  int kseg;            // float32-output runs: > 0 splits the contraction into kdim / kseg
                       // segments of kseg columns; segment g of L reads columns
                       // [lmap_g kseg, (lmap_g + 1) kseg) of the rows, of R those of
                       // rmap_g (4 bits per segment); 0: the columns in order
  unsigned lmap, rmap;
};
struct SymArgs {
  SymSeg seg[kMaxSeg];
  int nseg;
};
int symprod_tile(int s_pad);  // 192 when it divides s_pad, else 128
int symprod_tiles_per_matrix(int s_pad, int tile = 0);
hipError_t launch_symprod_bf16(const SymArgs& G, hipStream_t st);

// float32 path (tile multiples: s_pad % 64 == 0, ld % 64 == 0).
constexpr int kTileF32 = 64;
hipError_t launch_gram_f32(const NsGemmLaunch& L, hipStream_t st);
hipError_t launch_combine_f32(const NsGemmLaunch& L, hipStream_t st);

// Whole Newton-Schulz on chip for small matrices.
struct NsSmallLaunch {
  const void* X;       // [count] matrices, row stride ld_in
  void* Y;             // [count] matrices, row stride ld_out
  long long in_stride, out_stride;
  int s, l, ld_in, ld_out;
  long long count;
  bool transposed;     // X stored as l x s (tall); the kernel orients it
  int steps;
  float a[64], b[64];  // per-step coefficients (passed by value)
  const float* partials;  // non-null: nu from the momentum pass partials
  int P;
  float eps;
};
bool ns_small_supported(bool bf16, int s, int l);
hipError_t launch_ns_small(const NsSmallLaunch& L, bool bf16, hipStream_t st);

// Newton-Schulz of factored matrices X = V K^T (bf16 factors, r <= 8): the
// r x r core and optionally the dense result.
struct FactLaunch {
  const bf16_t* V;     // [batch][m][r]
  const bf16_t* K;     // [batch][n][r]
  float* C;            // [batch][r][r], or null
  bf16_t* O;           // [batch][m][n] or null
  long long batch;
  int m, n, r, m_pad, n_pad;  // pads: multiples of 16
  int vec;             // r == 8 and 16-byte aligned factors: 16-byte row loads
  int waves;           // wavefronts per workgroup
  int per_wave, f_off; // LDS bytes per wavefront; offset of the r x r work matrices in it
  int steps;
  float eps;
  float a[64], b[64], c[64];
};
int factored_lds_per_wave(int m_pad, int n_pad, bool dense, int* f_off = nullptr);
hipError_t launch_ns_factored(const FactLaunch& F, hipStream_t st);

// Padded sides, rank and Newton-Schulz coefficients of a factored core.
struct FactCoreArgs {
  int m_pad, n_pad, r, steps;
  float eps;
  float a[64], b[64], c[64];
};

// Momentum pathway over sequences of factored injections (ssm_momentum.hip):
// one workgroup per (sequence, chunk of kSsmMomQ tokens) forms the NS cores
// of the chunk's tokens and the chunk's float32 partial sums; then the chunk
// maps are applied in token order to the caller's states.
constexpr int kSsmMomQ = 256;
struct SsmMomLaunch {
  const bf16_t* V;     // [nseq][T][m][8]
  const bf16_t* K;     // [nseq][T][n][8]
  const float* a;      // [nseq][T] decays (with S), else null
  float beta;
  int m, n, T, Q, nchunks;  // m <= 64, n <= 128, Q tokens per chunk
  long long nseq;
  float* part;         // [nseq][nchunks][1 or 2][64][128] partial sums
  float* coef;         // [nseq][nchunks][4]: beta^L, prod a, B, 0
  float* M;            // [nseq][m][n] in/out
  float* S;            // null, or [nseq][m][n] in/out
  FactCoreArgs ns;     // m_pad 64, n_pad 128, r 8
};
// phase 0: cores and partial sums; phase 1: combine into M (and S)
hipError_t launch_ssm_momentum(const SsmMomLaunch& P, hipStream_t st, int phase);

// Spectral diagnostics (a chunk of `count` matrices per launch).
struct DiagPackLaunch {
  const void* A;       // [count][m][n], float32 or bf16 (f32)
  long long astride;   // m * n
  int n, s, l;         // row stride of A; short and long side
  bool tall, f32;
  bf16_t* L;           // [count][s_pad][ld] operand rows: X, or for float32 inputs its
                       // three bf16 pieces side by side [h | d | e]
  long long ostride;   // s_pad * ld
  int s_pad, kdim, ld; // s_pad % 128 == 0, kdim % 64 == 0, ld = kdim (bf16) or 3 kdim
  long long count;
  unsigned* clr;       // split run: the first clr_words words of each matrix's scratch
  long long cstride;   //   (stride cstride) are zeroed; or null
  long long clr_words;
};
hipError_t launch_diag_pack(const DiagPackLaunch& P, hipStream_t st);
struct DiagLaunch {
  const float* H;      // [count][s_pad][s_pad] Gram matrices (exactly symmetric)
  long long hstride;
  float* Q;            // [count][kmax][s_pad] Lanczos basis, or the split run's scratch
  long long qstride;
  int s, s_pad, iters, kmax;
  int split_p, split_r, split_nb;  // split run (set by the planner): blocks per side, row ranges, workgroups
  unsigned spin_limit;             // split run: polls before a wait is given up (set by the launcher)
  float* orth;         // [count] or null
  float* smax;         // [count] or null
  float* smin;         // [count] or null
  long long count;
};
size_t diag_lanczos_lds(int s_pad, int kmax);
// Plans the launch (split run or one workgroup per matrix); returns the
// 32-bit words of each matrix's scratch to zero beforehand (0: none).
long long diag_split_clear_words(DiagLaunch& D);
hipError_t launch_diag_lanczos(const DiagLaunch& D, hipStream_t st);

// AdamW over a list of float32 tensors (one launch: up to kAdamwMax tensors).
constexpr int kAdamwMax = 80;      // 40 bytes each: the table fits the kernel arguments
constexpr int kAdamwBlock = 4096;  // elements per workgroup
struct AdamwTensor {
  float* p;
  float* m;
  float* v;
  const void* g;       // float32 or bf16
  int n;               // elements (< 2^31)
  int block0;          // first workgroup of this tensor
};
struct AdamwLaunch {
  AdamwTensor t[kAdamwMax];
  int nt;
  float beta1, beta2, one_m_b1, one_m_b2, eps;
  float decay;         // 1 - lr * weight_decay
  float lr_bc;         // lr / (1 - beta1^t)
  float inv_sqrt_bc2;  // 1 / sqrt(1 - beta2^t)
};
hipError_t launch_adamw(const AdamwLaunch& A, bool grad_bf16, int blocks, hipStream_t st);

// Gated scan (gated_scan.hip, gated_scan_backward.hip).
constexpr int kScanChunk = 64;     // tokens per chunk
// Tokens per workgroup of the backward pass: as many as the tiles in LDS allow,
// 128 bfloat16 or 64 float32 ones; sequences of up to 64 tokens are one block of
// 64, half of whose tiles would be padding otherwise (64 of them, 24 heads: 112 us, 124
// in blocks of 128).
inline int scan_grad_tokens(bool bf16, int tokens) { return bf16 && tokens > kScanChunk ? 2 * kScanChunk : kScanChunk; }
// Work items that a launch has at most for a walk (sequence, head, kScanRows state
// rows: two workgroups of the states' walk) or a block of the backward pass; cut
// walks and split blocks are few.
constexpr int kScanItemThreads = 640;
constexpr int kScanRows = 64;      // state rows (value components) per workgroup
constexpr int kScanMaxN = 128;     // largest key length
// Kernels for up to 64 and up to 128 columns of the state: eight sequences of
// 2,048 tokens with 24 heads and N = 64 take 89 us forward and 176 backward with
// 64 columns, 95 and 239 padded to 128 (float32: 167 and 417, 190 and 634).
inline int scan_padded_n(int n) { return n <= 64 ? 64 : 128; }
struct SeqOperand {    // [batch][tokens][heads or groups][width], innermost stride 1
  const void* p;
  long long sb, st, sh;   // strides in elements
};
struct ScanWalk {
  SeqOperand x, k, q;  // values, keys, queries; in reversed time dy and queries (q unused)
  SeqOperand g, b;     // float32 log decays and input gates (b.p null: 1); st, sh per token, head
  int batch, tokens, heads, groups, P, N;
  int pblocks, nchunks;       // ceil(P / kScanRows), ceil(tokens / kScanChunk)
  int nseg, seg_chunks;       // segments of the time axis and their chunks
  int reverse;                // chunks from the last to the first, weights e^{c_i}
  int totals;                 // set by the launcher: segments from a zero state, into seg_state
  void* y;                    // [batch][tokens][heads][P]
  const float* init;          // null, or [batch][heads][P][N]: the state before the first chunk visited
  float* fin;                 // null, or the state after the last
  int keep_log2, nblocks;     // blocks of 2^keep_log2 chunks
  float* states;              // null, or [batch][heads * pblocks][nblocks][kScanRows x padded N]: the
                              // state that each block is visited with, in the order of state_offset
  float* seg_state;           // nseg > 1: [batch][heads * pblocks][nseg][kScanRows][padded N]
  float* seg_decay;           //           [batch][heads * pblocks][nseg]
};
// One walk, or two (dirs = 2, of equal sizes) in one launch; vec: see scan_vec.
hipError_t launch_scan_walk(const ScanWalk* W, int dirs, bool read, bool vec, bool bf16, hipStream_t st);
// Whether 16-byte buffer loads of rows of `width` elements fit an operand (es
// bytes an element): rows hold whole pieces, do not overlap, and a tile's lie
// within 32-bit offsets.  They may start anywhere: the memory takes 16 bytes at
// any address (eight sequences of 2,048 tokens, 24 heads, at an odd element: 99 us
// forward and 263 backward, 98 and 257 aligned, 329 and 638 element by element).
inline bool scan_vec(const SeqOperand& s, int width, int es) {
  return width % (16 / es) == 0 && s.st >= width && s.st * es * 2 * kScanChunk < (1LL << 31) - 256;
}
struct ScanGrad {
  SeqOperand v, k, q, dy, g, b;
  int batch, tokens, heads, groups, P, N, pblocks;
  int nblocks;                // blocks of scan_grad_tokens
  int nsplit;                 // workgroups that share a block's heads
  int dkvec;                  // rows of dq and dk: 4-element stores
  const float* states;        // as ScanWalk.states: before each block
  const float* dstates;       // gradients of the states after each block
  void *dv, *dk, *dq;
  float *dg, *db;             // [batch][tokens][heads]; db may be null
  float* parts;               // nsplit > 1: [nsplit][2][batch * tokens * groups * N]
};
hipError_t launch_scan_grad(const ScanGrad& A, bool vec, bool bf16, hipStream_t st);
struct ScanStep {
  SeqOperand v, k, q, g, b;
  int batch, heads, groups, P, N;
  void* y;                    // [batch][heads][P]
  const float* S;             // [batch][heads][P][N]
  float* S_out;               // may be S
};
constexpr int kScanStepThreads = 256;
long long scan_step_blocks(int batch, int heads, int P);
hipError_t launch_scan_step(const ScanStep& A, bool bf16, hipStream_t st);

// dst = src, or 0 where src is null (the final state of a scan without tokens).
hipError_t launch_copy_f32(const float* src, float* dst, long long n, hipStream_t st);

// Layer norm (layer_norm.hip).  Longest row: its columns count in int, and 1,024
// threads for 64 of them below 2^32.
constexpr int kNormMaxN = 1 << 27;
struct NormLaunch {
  const void* x;
  void* y;
  long long ldx, ldy, rows;
  int n, center;
  const float *w, *bias;   // may be null
  float eps;
  float *mean, *rstd;      // [rows], may be null
};
hipError_t launch_norm(const NormLaunch& A, bool bf16, hipStream_t st);
struct NormGradLaunch {
  const void *dy, *x;
  void* dx;
  long long lddy, ldx, lddx, rows;
  int n;
  const float* w;          // may be null
  const float *mean, *rstd;   // mean null: no centering
  float *dw, *dbias;       // may be null
  float* part;             // [parts][2][n]
  int parts;
};
int norm_grad_parts(long long rows, int n, bool bf16);
hipError_t launch_norm_grad(const NormGradLaunch& A, bool bf16, hipStream_t st);

// Token numbers (embedding.hip, token_logprobs.hip): token t is element
// (t / run) stride + (t % run) step of p; t / run = umulhi(t, magic) >> shift for
// t < 2^31 (magic 0: one run).
struct IdsOperand {
  const void* p;
  int wide;                  // int64, else int32
  uint32_t run, magic;
  int shift;
  long long stride, step;
};

// Embedding (embedding.hip): y_t = scale table[id_t], zero for ids outside the table.
struct EmbedLaunch {
  const void* table;
  void* y;
  IdsOperand ids;
  long long ldt, ldy;
  uint32_t tokens;
  int vocab, n;
  float scale;
};
hipError_t launch_embed(const EmbedLaunch& A, bool table_bf16, bool bf16, hipStream_t st);
struct EmbedGradLaunch {
  const void* dy;
  void* dtable;              // [vocab][n]
  IdsOperand ids;
  long long lddy;
  uint32_t tokens;
  int vocab, n, accumulate;
  float scale;
  // workspace
  int* count;                // of the tokens inside the table
  int2* sorted;              // those by id, in their order: token, id
  float* part;               // [chunks][2][n]
  uint16_t* map;             // many tokens: their ranges of ids
  int* table;                // and how many each block of tokens has of each
  IdsOperand by_range;       // id / ids of a range, as ids' runs
};
struct EmbedMapSizes {
  size_t map, table;         // bytes
  int range;                 // ids of a range
};
EmbedMapSizes embed_map_sizes(uint32_t tokens, int vocab);   // of no bytes where the map is not used
int embed_grad_chunk(uint32_t tokens);   // sorted tokens that a wave adds up, a piece of their columns a lane
hipError_t launch_embed_grad(const EmbedGradLaunch& A, bool bf16, bool table_bf16, hipStream_t st);

// Group norm (group_norm.hip, group_norm_backward.hip): each group of w channels of a
// row is normalised by itself.
enum NormGate { kGateBefore, kGateAfter, kGateNone };   // norm(x silu(z)) w + b; (norm(x) w + b) silu(z); silu(norm(x) w + b)
enum NormAct { kActNone, kActSilu };                    // of kGateNone
struct GroupNormLaunch {
  const void *x, *z;       // z null: kGateNone
  void* y;
  long long ldx, ldz, ldy;
  int rows, groups, w, center, act;
  const float *weight, *bias;   // may be null
  float eps;
  float *mean, *rstd;      // [rows][groups], may be null
};
hipError_t launch_group_norm(const GroupNormLaunch& A, NormGate gate, bool bf16, hipStream_t st);
struct GroupNormGradLaunch {
  const void *dy, *x, *z;
  void *dx, *dz;
  long long lddy, ldx, ldz, lddx, lddz;
  int rows, groups, w, act;
  const float *weight, *bias;   // may be null
  const float *mean, *rstd;     // [rows][groups]; mean null: no centering
  float *dw, *db;          // may be null
  float* part;             // [parts][2][groups w]
  int parts, span, per;    // see GroupGradPlan
};
// Groups and rows that a workgroup takes at a time, and workgroups that share the rows.
struct GroupGradPlan {
  int span, per, parts;
};
GroupGradPlan group_norm_grad_plan(int rows, int groups, int w, bool bf16, bool gated);
hipError_t launch_group_norm_grad(const GroupNormGradLaunch& A, NormGate gate, bool bf16, hipStream_t st);
// dw and db (null: not wanted) from part[parts][2][n] (layer_norm.hip).
hipError_t launch_norm_parts(const float* part, int parts, int n, float* dw, float* db, hipStream_t st);

// Log probabilities of tokens from rows of logits (token_logprobs.hip).
constexpr int kLogpMaxTop = 64;
struct LogpLaunch {
  const void* x;
  IdsOperand ids;            // p null: no tokens
  long long ldx, rows;
  int vocab, top, splits;    // workgroups that share a row
  float scale;
  float *logp, *entropy;     // [rows], may be null
  float* stats;              // [rows][2]: the largest logit, the log of the sum around it; may be null
  int* top_ids;              // [rows][top]
  float* top_logp;
  // workspace of splits > 1
  float* part;               // [rows][splits][3]
  unsigned long long* ranks; // [rows][splits][top]
};
int logp_splits(long long rows, int vocab, bool bf16);
hipError_t launch_logp(const LogpLaunch& A, bool bf16, hipStream_t st);
struct LogpGradLaunch {
  const void* x;
  void* dx;                  // may be x
  IdsOperand ids;            // p null: no tokens
  long long ldx, lddx, rows;
  int vocab;
  float scale;
  const float* stats;
  const float *dlogp, *dentropy, *entropy;   // dlogp or dentropy may be null
  long long sdlogp, sdentropy;               // their strides
};
hipError_t launch_logp_grad(const LogpGradLaunch& A, bool bf16, hipStream_t st);

}  // namespace muon
