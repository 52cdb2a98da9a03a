// Tiles, fragments and gates of the gated scan kernels (gated_scan.hip,
// gated_scan_backward.hip).
//
// Products run on 16 x 16 matrix-core tiles with 32 contraction terms a step.
// Lane l of the wave (g = l / 16) holds, of either operand, row l % 16 at the
// 8 contraction indices 8 g + 0..7, and of the result column l % 16 (the
// second operand's row), rows 4 g + 0..3 (the first operand's).  Any
// permutation of the contraction indices that both operands share gives the
// same product, so a result kept in registers can be the next product's
// operand without a trip through LDS (state_row).  bfloat16 operands
// take one v_mfma_f32_16x16x32_bf16 per step, float32 ones eight
// v_mfma_f32_16x16x4f32.
#pragma once
#include "launch.h"

namespace muon {
namespace scan {

constexpr int kQ = kScanChunk;   // tokens per chunk
constexpr int kPB = kScanRows;   // state rows (value components) per workgroup
// log decays below this are taken as this: e^-10000 is 0 in float32 and in
// float64 alike, and sums of 64 of them stay finite
constexpr float kMinLogDecay = -1.0e4f;

struct FragF32 {
  float v[8];
};

template <typename T>
struct Ops;

template <>
struct Ops<bf16_t> {
  typedef bf16x8_t Frag;
  static constexpr int kVec = 8;      // elements per 16 bytes
  static constexpr int kSplit = 3;    // bf16 pieces that carry a float32's 24 bits
  static constexpr int kRounded = 2;  // and 16 bits, for operands of results that are rounded to bf16 themselves
  __device__ static __forceinline__ f32x4_t mma(Frag a, Frag b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  // 8 consecutive elements
  __device__ static __forceinline__ Frag row(const bf16_t* p) {
    return __builtin_bit_cast(Frag, *reinterpret_cast<const u32x4_t*>(p));
  }
  __device__ static __forceinline__ void widen(Frag f, float (&o)[8]) {
    const u32x4_t w = __builtin_bit_cast(u32x4_t, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = lo_bf16(w[i]);
      o[2 * i + 1] = hi_bf16(w[i]);
    }
  }
  __device__ static __forceinline__ Frag narrow(const float (&v)[8]) {
    return __builtin_bit_cast(Frag, u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7])});
  }
  // a float32 operand as PIECES bfloat16 ones (rounded, then the remainder, then
  // its remainder): kSplit for all of its 24 bits
  template <int PIECES>
  __device__ static __forceinline__ void split(const float (&v)[8], Frag (&f)[PIECES]) {
    float r[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = v[i];
#pragma unroll
    for (int u = 0; u < PIECES; ++u) {
      f[u] = narrow(r);
      widen(f[u], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = r[i] - w[i];
    }
  }
  __device__ static __forceinline__ void store4(bf16_t* p, f32x4_t v) {
    *reinterpret_cast<u32x2_t*>(p) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
  __device__ static __forceinline__ f32x4_t load4(const bf16_t* p) {
    const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
    return f32x4_t{lo_bf16(w[0]), hi_bf16(w[0]), lo_bf16(w[1]), hi_bf16(w[1])};
  }
  __device__ static __forceinline__ f32x4_t rounded4(f32x4_t v) {
    const uint32_t a = pack_bf16x2(v[0], v[1]), b = pack_bf16x2(v[2], v[3]);
    return f32x4_t{lo_bf16(a), hi_bf16(a), lo_bf16(b), hi_bf16(b)};
  }
  __device__ static __forceinline__ bf16_t from_f32(float v) { return f32_to_bf16(v); }
};

template <>
struct Ops<float> {
  typedef FragF32 Frag;
  static constexpr int kVec = 4;
  static constexpr int kSplit = 1, kRounded = 1;
  __device__ static __forceinline__ f32x4_t mma(const Frag& a, const Frag& b, f32x4_t c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], c, 0, 0, 0);
    return c;
  }
  // two runs of 4 consecutive elements
  __device__ static __forceinline__ Frag row2(const float* p, const float* q) {
    const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(q);
    return Frag{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
  }
  __device__ static __forceinline__ void widen(const Frag& f, float (&o)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = f.v[i];
  }
  __device__ static __forceinline__ Frag narrow(const float (&v)[8]) {
    Frag f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f.v[i] = v[i];
    return f;
  }
  template <int PIECES>
  __device__ static __forceinline__ void split(const float (&v)[8], Frag (&f)[PIECES]) { f[0] = narrow(v); }
  __device__ static __forceinline__ f32x4_t rounded4(f32x4_t v) { return v; }
  __device__ static __forceinline__ void store4(float* p, f32x4_t v) { *reinterpret_cast<f32x4_t*>(p) = v; }
  __device__ static __forceinline__ f32x4_t load4(const float* p) { return *reinterpret_cast<const f32x4_t*>(p); }
  __device__ static __forceinline__ float from_f32(float v) { return v; }
};

// A row-major tile of rows of WIDTH elements in LDS.  The 16-byte pieces of a
// row are permuted by XOR with its number, so that the 16 rows that a fragment
// reads at once cover all banks; 128-byte rows, two to a sweep of the banks,
// take half of it.
template <typename T, int WIDTH>
struct Tile {
  typedef Ops<T> O;
  typedef typename O::Frag Frag;
  static constexpr int kVec = O::kVec, kBytes = WIDTH * static_cast<int>(sizeof(T));
  static_assert(kBytes == 128 || kBytes % 256 == 0, "rows of whole sweeps of the banks, or half a sweep");
  // of column col; what lies in its 16 bytes is contiguous
  __device__ static __forceinline__ int at(int row, int col) {
    const int x = kBytes == 128 ? (row >> 1) & 7 : row & 15;
    return row * WIDTH + ((col / kVec) ^ x) * kVec + col % kVec;
  }
  // 8 elements from column col, a multiple of 8
  __device__ static __forceinline__ Frag row(const T* tile, int row, int col) {
    if constexpr (sizeof(T) == 2) return O::row(tile + at(row, col));
    else return O::row2(tile + at(row, col), tile + at(row, col + 4));
  }
  __device__ static __forceinline__ void store8(T* tile, int row, int col, Frag f) {
    if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<Frag*>(tile + at(row, col)) = f;
    } else {
      O::store4(tile + at(row, col), f32x4_t{f.v[0], f.v[1], f.v[2], f.v[3]});
      O::store4(tile + at(row, col + 4), f32x4_t{f.v[4], f.v[5], f.v[6], f.v[7]});
    }
  }
  // column col0 + l % 16 of rows row0 + 8 g + 0..7 (bfloat16: ds_read_b64_tr_b16,
  // where in each 16-lane group the lanes address a 4 x 16 block, 4 elements
  // each, and receive one column)
  __device__ static __forceinline__ Frag col(const T* tile, int row0, int col0, int lane) {
    if constexpr (sizeof(T) == 2) {
      const int r = row0 + 8 * (lane >> 4) + ((lane & 15) >> 2), c = col0 + 4 * (lane & 3);
      const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(tile + at(r, c)));
      const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(tile + at(r + 4, c)));
      const u32x2_t ua = __builtin_bit_cast(u32x2_t, a), ub = __builtin_bit_cast(u32x2_t, b);
      return __builtin_bit_cast(Frag, u32x4_t{ua[0], ua[1], ub[0], ub[1]});
    } else {
      Frag f;
#pragma unroll
      for (int e = 0; e < 8; ++e) f.v[e] = tile[at(row0 + 8 * (lane >> 4) + e, col0 + (lane & 15))];
      return f;
    }
  }
  __device__ static __forceinline__ f32x4_t load4(const T* tile, int row, int col) { return O::load4(tile + at(row, col)); }
};

// The 16 x 16 tiles on one side of the diagonal of a matrix of TILES x TILES of
// them, and one of zeros for those on the other side: the weights of a block, in
// kRounded pieces.  A tile's 16-byte pieces lie column by column, so that what
// 16 lanes read or 32 lanes write at once is contiguous.
template <typename T, int TILES>
struct Triangle {
  typedef Ops<T> O;
  typedef typename O::Frag Frag;
  static constexpr int kVec = O::kVec, kTiles = TILES * (TILES + 1) / 2, kPiece = (kTiles + 1) * 256, kSize = O::kRounded * kPiece;
  // of the tile at `far` tiles from the matrix' corner along one side and `near` along the other
  static __device__ __forceinline__ int tile(int far, int near) { return far >= near ? far * (far + 1) / 2 + near : kTiles; }
  static __device__ __forceinline__ int at(int tile, int row, int col) { return tile * 256 + ((col / kVec) * 16 + row) * kVec + col % kVec; }
  // 8 elements from column col, a multiple of 8
  static __device__ __forceinline__ Frag row(const T* m, int piece, int tile, int row, int col) {
    m += piece * kPiece;
    if constexpr (sizeof(T) == 2) return O::row(m + at(tile, row, col));
    else return O::row2(m + at(tile, row, col), m + at(tile, row, col + 4));
  }
  static __device__ __forceinline__ void store4(T* m, int tile, int row, int col, f32x4_t v) {
#pragma unroll
    for (int e = 0; e < O::kRounded; ++e) {
      O::store4(m + e * kPiece + at(tile, row, col), v);
      if (e + 1 < O::kRounded) v -= O::rounded4(v);
    }
  }
  static __device__ __forceinline__ void store1(T* m, int tile, int row, int col, float v) {
    const T hi = O::from_f32(v);
    m[at(tile, row, col)] = hi;
    if constexpr (O::kRounded == 2) m[kPiece + at(tile, row, col)] = O::from_f32(v - bf16_to_f32(hi));
  }
  static __device__ __forceinline__ void clear_zeros(T* m, int tid) {
#pragma unroll
    for (int e = 0; e < O::kRounded; ++e)
      if (tid < 256) m[e * kPiece + kTiles * 256 + tid] = O::from_f32(0.0f);
  }
};

// A value that the compiler takes for new: what depends on it is computed where
// it is used, and not once before a long loop, in registers that the loop's
// accumulators need.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Keeps the computation of an accumulator where it is written: sums that are read
// only after a long loop are otherwise moved behind the phases that follow, and
// everything they add is kept until there.
__device__ __forceinline__ void settle(f32x4_t& v) { asm volatile("" : "+v"(v)); }

// Workgroups go to the eight XCDs in turn; this gives each XCD a run of
// neighbouring items instead, whose shared operands its L2 then holds once.
__device__ __forceinline__ int xcd_item(int block, int items) {
  const int x = block & 7, i = block >> 3, each = items >> 3, more = items & 7;
  return x * each + (x < more ? x : more) + i;
}

// Buffer resources: an access at or past `bytes` reads 0 and stores nothing,
// so ragged tiles need no branches.  kNowhere is such an offset.
constexpr int kNowhere = 0x7ffffff0;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0), bytes, 0x00020000);
}
__device__ __forceinline__ f32x4_t load_f32x4(__amdgpu_buffer_rsrc_t r, int offset, int base) {
  return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, offset, base, 0));
}

// A [ROWS][WIDTH] tile of a sequence operand on its way into LDS: 16-byte
// pieces held in the registers of THREADS threads.  Rows past the last token
// and columns past `width` are zero.  VEC (chosen by the host, scan_vec): rows
// hold whole pieces, do not overlap and lie within 2 GiB of each other; otherwise
// element by element.
template <typename T, int WIDTH, int ROWS, int THREADS, bool VEC>
struct TileLoad {
  static constexpr int kVec = Ops<T>::kVec;
  static constexpr int kRowPieces = WIDTH / kVec;
  static constexpr int kPieces = ROWS * kRowPieces / THREADS;
  static_assert(ROWS * kRowPieces % THREADS == 0, "whole pieces");
  u32x4_t r[kPieces];

  // p: element (first token, column 0); rows: tokens left, at most ROWS
  __device__ __forceinline__ void load(const T* p, long long st, int rows, int width, int tid) {
    if constexpr (VEC) {
      const __amdgpu_buffer_rsrc_t b = rsrc(p, static_cast<int>(rows * st) * static_cast<int>(sizeof(T)));
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int idx = i * THREADS + tid, row = idx / kRowPieces, col = (idx % kRowPieces) * kVec;
        const int off = (row * static_cast<int>(st) + col) * static_cast<int>(sizeof(T));
        r[i] = __builtin_amdgcn_raw_buffer_load_b128(b, col < width ? off : kNowhere, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int idx = i * THREADS + tid, row = idx / kRowPieces, col = (idx % kRowPieces) * kVec;
        const T* e = p + row * st + col;
        r[i] = u32x4_t{0u, 0u, 0u, 0u};
        if (row >= rows) continue;
#pragma unroll
        for (int j = 0; j < kVec; ++j)
          if (col + j < width) {
            if constexpr (sizeof(T) == 2) r[i][j / 2] |= static_cast<uint32_t>(e[j]) << (16 * (j & 1));
            else r[i][j] = __float_as_uint(e[j]);
          }
      }
    }
  }
  __device__ __forceinline__ void store(T* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int idx = i * THREADS + tid, row = idx / kRowPieces, col = (idx % kRowPieces) * kVec;
      *reinterpret_cast<u32x4_t*>(lds + Tile<T, WIDTH>::at(row, col)) = r[i];
    }
  }
};

// The 16-byte pieces of row n of a transposed tile [WIDTH][kQ] are permuted by
// XOR with this.  The 16 rows that a fragment reads at once (neighbours, or those
// of state_row) cover all LDS banks, and so do the rows 8 (float32: 4) apart
// that half a wave writes at once.
template <typename T>
__device__ __forceinline__ constexpr int pieces_order(int n) {
  const auto bit = [n](int i) { return n >> i & 1; };
  return sizeof(T) == 2 ? (bit(1) ^ bit(5)) | bit(3) << 1 | (bit(2) ^ bit(4)) << 2
                        : (bit(0) ^ bit(4)) | (bit(1) ^ bit(5)) << 1 | bit(3) << 2 | (bit(2) ^ bit(4)) << 3;
}
// The column of the state that row r of a wave's 16-row tile t of S^T holds: the
// two tiles of 32 columns give a lane, which has rows 4 g + 0..3 of each, 8
// neighbours, as the operand of S q wants them.
__device__ __forceinline__ constexpr int state_row(int t, int r) { return 32 * (t >> 1) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3); }

// A [kQ][WIDTH] tile that is (also) needed transposed: a thread holds the same
// PIECE columns of two neighbouring tokens, so that it writes both tokens of a
// transposed row at once.
template <typename T, int WIDTH, int THREADS, bool VEC, int PIECE = Ops<T>::kVec>
struct PairLoad {
  static constexpr int kVec = Ops<T>::kVec;
  static constexpr int kWords = PIECE * static_cast<int>(sizeof(T)) / 4;
  static constexpr int kRowPieces = WIDTH / PIECE;
  static constexpr int kAll = kQ / 2 * kRowPieces;
  static constexpr int kPairs = kAll / THREADS;
  // half a wave: kNear pieces of 32 / kNear pairs of tokens
  static constexpr int kNear = sizeof(T) == 2 ? 8 : 16;
  static_assert(kAll % THREADS == 0, "whole pairs");
  static_assert(kRowPieces % kNear == 0, "whole half waves");
  typedef uint32_t Piece __attribute__((ext_vector_type(kWords)));
  Piece r[kPairs][2];

  // (pieces of 4 bfloat16: of 0..3 and 8..11, whose order differs)
  static __device__ __forceinline__ int piece_of(int idx) {
    const int i = idx % kNear + kNear * (idx / 32 % (kRowPieces / kNear));
    return sizeof(T) == 2 && PIECE == 4 ? (i & ~12) | (i & 4) << 1 | (i & 8) >> 1 : i;
  }
  static __device__ __forceinline__ int pair_of(int idx) {
    return idx % 32 / kNear + 32 / kNear * (idx / 32 / (kRowPieces / kNear));
  }

  __device__ __forceinline__ void load(const T* p, long long st, int rows, int width, int tid) {
    const __amdgpu_buffer_rsrc_t b = rsrc(p, VEC ? static_cast<int>(rows * st) * static_cast<int>(sizeof(T)) : 0);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int idx = i * THREADS + tid, col = piece_of(idx) * PIECE;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = 2 * pair_of(idx) + u;
        if constexpr (VEC) {
          const int off = col < width ? (row * static_cast<int>(st) + col) * static_cast<int>(sizeof(T)) : kNowhere;
          if constexpr (kWords == 4) r[i][u] = __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0);
          else r[i][u] = __builtin_amdgcn_raw_buffer_load_b64(b, off, 0, 0);
        } else {
          const T* e = p + row * st + col;
          r[i][u] = Piece(0u);
          if (row >= rows) continue;
#pragma unroll
          for (int j = 0; j < PIECE; ++j)
            if (col + j < width) {
              if constexpr (sizeof(T) == 2) r[i][u][j / 2] |= static_cast<uint32_t>(e[j]) << (16 * (j & 1));
              else r[i][u][j] = __float_as_uint(e[j]);
            }
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* lds, int tid) const {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int idx = i * THREADS + tid;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        *reinterpret_cast<Piece*>(lds + Tile<T, WIDTH>::at(2 * pair_of(idx) + u, piece_of(idx) * PIECE)) = r[i][u];
    }
  }
  // f(row n of the transposed tile, offset in it, the two tokens' element n, index of the first token)
  template <typename F>
  __device__ __forceinline__ void each_transposed(int tid, F f) const {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int idx = i * THREADS + tid, n0 = piece_of(idx) * PIECE, j = 2 * pair_of(idx);
      const int c = (j / kVec) ^ pieces_order<T>(n0), at = n0 * kQ + j % kVec;
#pragma unroll
      for (int e = 0; e < PIECE; ++e)   // n0 is a multiple of PIECE: the order of n0 + e is theirs together
        f(at + e * kQ + (c ^ pieces_order<T>(e)) * kVec, r[i][0], r[i][1], e, j);
    }
  }
  __device__ __forceinline__ void store_transposed(T* lds, int tid) const {
    each_transposed(tid, [&](int at, Piece a, Piece b, int e, int) {
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint32_t*>(lds + at) =
            e % 2 == 0 ? (a[e / 2] & 0xffffu) | (b[e / 2] << 16) : (a[e / 2] >> 16) | (b[e / 2] & 0xffff0000u);
      else
        *reinterpret_cast<u32x2_t*>(lds + at) = u32x2_t{a[e], b[e]};
    });
  }
  // (bfloat16) The elements by their tokens' weights, transposed, as three
  // tiles of pieces that carry the products' 24 bits.
  __device__ __forceinline__ void store_split(T* lds, const float* weights, int tid) const {
    static_assert(sizeof(T) == 2, "bfloat16 operands");
    each_transposed(tid, [&](int at, Piece a, Piece b, int e, int j) {
      const uint32_t p = a[e / 2], q = b[e / 2];
      float u = (e % 2 == 0 ? lo_bf16(p) : hi_bf16(p)) * weights[j], v = (e % 2 == 0 ? lo_bf16(q) : hi_bf16(q)) * weights[j + 1];
#pragma unroll
      for (int z = 0; z < 3; ++z) {
        const uint32_t w = pack_bf16x2(u, v);
        *reinterpret_cast<uint32_t*>(lds + z * WIDTH * kQ + at) = w;
        u -= lo_bf16(w);
        v -= hi_bf16(w);
      }
    });
  }
};
// Row n, tokens j0..j0 + 7 (j0 a multiple of 8) of a transposed tile.
template <typename T>
__device__ __forceinline__ typename Ops<T>::Frag transposed_row(const T* tile, int n, int j0) {
  constexpr int kVec = Ops<T>::kVec;
  const T* row = tile + n * kQ;
  const int x = pieces_order<T>(n), c = j0 / kVec;
  if constexpr (sizeof(T) == 2) return Ops<T>::row(row + (c ^ x) * kVec);
  else return Ops<T>::row2(row + (c ^ x) * kVec, row + ((c + 1) ^ x) * kVec);
}

// Four neighbours of an output row (columns col..col + 3 of `width`) at element
// offset `off` of a tile of rows at p; rows < `rows` are written.
template <typename T, bool VEC>
struct TileStore {
  T* p;
  __amdgpu_buffer_rsrc_t b;
  long long st;
  int rows, width;
  __device__ __forceinline__ TileStore(T* p, long long st, int rows, int width)
      : p(p), b(rsrc(p, VEC ? static_cast<int>(rows * st) * static_cast<int>(sizeof(T)) : 0)), st(st), rows(rows), width(width) {}
  __device__ __forceinline__ void put(int row, int col, f32x4_t v) const {
    if constexpr (VEC) {
      const int off = col < width ? (row * static_cast<int>(st) + col) * static_cast<int>(sizeof(T)) : kNowhere;
      if constexpr (sizeof(T) == 2)
        __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}, b, off, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), b, off, 0, 0);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (row < rows && col + r < width) p[row * st + col + r] = Ops<T>::from_f32(v[r]);
    }
  }
};

// Inclusive sums over the lanes of a wave, in float64.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_rows_d(double v) {
  const long long b = __double_as_longlong(v);
  const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xf, false);
  return __longlong_as_double((static_cast<long long>(hi) << 32) | static_cast<unsigned>(lo));
}
__device__ __forceinline__ double wave_prefix_d(double v) {
  v += dpp_rows_d<kDppShr1, 0xf>(v);
  v += dpp_rows_d<kDppShr2, 0xf>(v);
  v += dpp_rows_d<kDppShr4, 0xf>(v);
  v += dpp_rows_d<kDppShr8, 0xf>(v);
  v += dpp_rows_d<kDppBcast15, 0xa>(v);
  v += dpp_rows_d<kDppBcast31, 0xc>(v);
  return v;
}
__device__ __forceinline__ double read_lane_d(double v, int lane) {
  const long long b = __double_as_longlong(v);
  const int lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
  const int hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
  return __longlong_as_double((static_cast<long long>(hi) << 32) | static_cast<unsigned>(lo));
}

// The gates of a chunk of Q tokens.  c is the inclusive prefix sum of the log2
// decays, summed in float64 and kept as two floats, so that e^{c_i - c_j}
// keeps float32 accuracy after a reset (log decay -inf) has made both sums
// large.
template <int Q>
struct Gates {
  float hi[Q], lo[Q];   // c
  float b[Q];           // input gates
  float first[Q];       // e^{c_i}
  float last[Q];        // e^{c_end - c_j}
  float row[Q];         // e^{c_t - c_r}, r the first token of t's 16
  float in[Q];          // weights of what enters a state: e^{c_end - c_j} b_j, in reversed time e^{c_i}
  float end[4];         // e^{c_end}
};

// By one wave: lane l brings the gates of tokens U l..U l + U - 1.  Returns c_end.
template <int Q>
__device__ __forceinline__ double write_gates(Gates<Q>& G, const float (&log_decay)[Q / 64], const float (&gate)[Q / 64],
                                              int lane, bool reverse) {
  constexpr int U = Q / 64;
  double own[U], sum = 0.0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float ld = log_decay[u] < kMinLogDecay ? kMinLogDecay : log_decay[u];   // keeps NaN
    own[u] = static_cast<double>(ld) * static_cast<double>(1.44269504088896340736);
    sum += own[u];
  }
  const double upto = wave_prefix_d(sum), e = read_lane_d(upto, 63);
  double c = upto - sum, first16 = 0.0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = U * lane + u;
    c = u + 1 == U ? upto : c + own[u];
    if (u == 0) first16 = __shfl(c, lane & ~(16 / U - 1), kWave);
    const float hi = static_cast<float>(c);
    G.hi[t] = hi;
    G.lo[t] = static_cast<float>(c - static_cast<double>(hi));
    G.b[t] = gate[u];
    const float first = __builtin_amdgcn_exp2f(static_cast<float>(c)), last = __builtin_amdgcn_exp2f(static_cast<float>(e - c));
    G.first[t] = first;
    G.last[t] = last;
    G.in[t] = reverse ? first : last * gate[u];
    G.row[t] = __builtin_amdgcn_exp2f(static_cast<float>(c - first16));
  }
  if (lane == 0) G.end[0] = __builtin_amdgcn_exp2f(static_cast<float>(e));
  return e;
}

// e^{c_i - c_j} for the four rows i = i0..i0 + 3 and the column j of a tile in
// rows i of 16-token block it.  Below the diagonal block it is taken by way of
// the block's first token, one exponential for the four (its two factors are at
// most 1 where the log decays are); on it, one by one, 0 for j > i.
template <int Q>
__device__ __forceinline__ f32x4_t between4_below(const Gates<Q>& G, int it, int i0, int j) {
  const float to = __builtin_amdgcn_exp2f((G.hi[16 * it] - G.hi[j]) + (G.lo[16 * it] - G.lo[j]));
  return *reinterpret_cast<const f32x4_t*>(G.row + i0) * to;
}
template <int Q>
__device__ __forceinline__ f32x4_t between4_diagonal(const Gates<Q>& G, int i0, int j) {
  const float hi = G.hi[j], lo = G.lo[j];
  const f32x4_t ih = *reinterpret_cast<const f32x4_t*>(G.hi + i0), il = *reinterpret_cast<const f32x4_t*>(G.lo + i0);
  f32x4_t d;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float e = __builtin_amdgcn_exp2f((ih[r] - hi) + (il[r] - lo));
    d[r] = i0 + r >= j ? e : 0.0f;
  }
  return d;
}
template <int Q>
__device__ __forceinline__ f32x4_t between4(const Gates<Q>& G, int it, int jt, int i0, int j) {
  return it != jt ? between4_below(G, it, i0, j) : between4_diagonal(G, i0, j);
}

// By a decay: nothing is left of what has decayed to 0, whatever it was, so a
// sequence that starts is not reached by a NaN or an infinity of the last one's
// state.
__device__ __forceinline__ float decayed(float v, float by) { return by == 0.0f ? 0.0f : v * by; }
__device__ __forceinline__ f32x4_t decayed(f32x4_t v, float by) {
  return f32x4_t{decayed(v[0], by), decayed(v[1], by), decayed(v[2], by), decayed(v[3], by)};
}

// Sums over the four 16-lane rows of a wave, for four values at once: row g of
// the result holds the sum of s_g (v_permlane16_swap, v_permlane32_swap: no
// LDS).
__device__ __forceinline__ float sum_rows4(float s0, float s1, float s2, float s3) {
  const auto swap_add16 = [](float a, float b) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  const float a = swap_add16(s0, s1), b = swap_add16(s2, s3);
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Sums over the 16 lanes of a row, for four values at once: lane l of the row
// holds the sum of s_{l % 4}.
__device__ __forceinline__ float sum_lanes4(float s0, float s1, float s2, float s3, int l16) {
  const bool odd = l16 & 1, two = l16 & 2;
  const float a = (odd ? s1 : s0) + dpp_f<kDppXor1>(odd ? s0 : s1);
  const float b = (odd ? s3 : s2) + dpp_f<kDppXor1>(odd ? s2 : s3);
  float v = (two ? b : a) + dpp_f<kDppXor2>(two ? a : b);
  v += dpp_f<kDppRor8>(v);
  v += dpp_f<0x124>(v);   // row_ror:4
  return v;
}

// Sums over the lanes of a 16-lane row: up to a lane, before it, and from it on.
__device__ __forceinline__ float lanes_upto(float v) {
  v += dpp_f<kDppShr1>(v);
  v += dpp_f<kDppShr2>(v);
  v += dpp_f<kDppShr4>(v);
  return v + dpp_f<kDppShr8>(v);
}
__device__ __forceinline__ float lanes_before(float v) { return dpp_f<kDppShr1>(lanes_upto(v)); }
__device__ __forceinline__ float lanes_from(float v) {
  v += dpp_f<kDppShl1>(v);
  v += dpp_f<kDppShl2>(v);
  v += dpp_f<kDppShl4>(v);
  return v + dpp_f<kDppShl8>(v);
}

// Tile e of the 16 x 16 tiles on and below the diagonal, row by row (at most
// eight rows).
__device__ __forceinline__ int tile_row(int e) {
  return (e >= 1) + (e >= 3) + (e >= 6) + (e >= 10) + (e >= 15) + (e >= 21) + (e >= 28);
}
__device__ __forceinline__ int tile_col(int e, int row) { return e - row * (row + 1) / 2; }

// 8 consecutive floats of LDS.
__device__ __forceinline__ void load8(const float* p, float (&o)[8]) {
  const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = a[i];
    o[4 + i] = b[i];
  }
}

// Element (n, p) of a state in the workspace, in the order in which the
// backward pass loads it: blocks of 16 n by 32 p, of which lane
// (n % 16) + 16 (p % 32 / 8) holds 8 neighbours p, four by one load.
__device__ __forceinline__ int state_offset(int n, int p) {
  return (((n >> 4) * (kPB / 32) + (p >> 5)) * 2 + ((p >> 2) & 1)) * 256 + ((n & 15) + 16 * ((p & 31) >> 3)) * 4 + (p & 3);
}

}  // namespace scan
}  // namespace muon
