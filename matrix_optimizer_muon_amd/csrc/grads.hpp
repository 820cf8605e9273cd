// Arguments of the training-gradient kernels (grads.hip), shared with the host
// planner and entry points (grads.cpp).  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.hpp"

namespace dmuon {

// An operand of the matrix products is one bf16 plane, or three whose sum is an
// fp32 value (x = hi + mid + lo, 24 bits).  A product of two operands is then the
// sum of plane products; the pairs, smallest first, 4 bits per product.
constexpr int kPlanes = 3;
struct PlanePairs {
  int32_t n;
  uint32_t a, b;               // plane of product p: (a >> 4p) & 15
};
// 1 × 1 planes: one product.  1 × 3 and 3 × 1: three.  3 × 3: the six whose
// factors multiply to at least 2⁻¹⁶ (the others are below fp32's own rounding):
// (1,1) (2,0) (0,2) (1,0) (0,1) (0,0), smallest first.
inline PlanePairs plane_pairs(int planes_a, int planes_b) {
  if (planes_a == 1 && planes_b == 1) return {1, 0, 0};
  if (planes_a == 1) return {3, 0x000, 0x012};
  if (planes_b == 1) return {3, 0x012, 0x000};
  return {6, 0x001021, 0x010201};
}

// rows of a matrix gathered (or not) into zero-padded bf16 planes
struct PackArgs {
  const void* src;             // rows × cols, row stride ld elements
  int64_t ld;
  int32_t f32;                 // source type; fp32 becomes three planes
  int32_t cols;
  int64_t rows;                // destination rows (upper bound when count is set)
  const int32_t* gather;       // source row of destination row i, or null: i
  const int32_t* count;        // device row count, or null: rows
  uint16_t* dst;               // [plane][rows][ldd], columns cols … ldd − 1 zero; or null
  int64_t plane;               // elements between planes
  uint16_t* blocks;            // the same in fragment order, rows padded to 16; or null
  int64_t blocks_plane;
  int32_t ldd;                 // multiple of 64
};

// ---- cross entropy ------------------------------------------------------------
constexpr int64_t kElsewhere = INT32_MIN;    // DMUON_TARGET_ELSEWHERE
constexpr int32_t kTgtNone = -1;             // compact targets that are no vocabulary row
constexpr int32_t kTgtElsewhere = -2;
struct CeScanArgs {
  const void* targets;
  int32_t idx64;
  int32_t backward;
  int64_t ignore;
  int32_t tokens, vocab;
  const float* grad_losses;    // backward
  const float* lse_in;         // backward
  float* losses;               // forward: zeroed where ignored
  float* lse;
  int32_t* rows;               // token of compact row i
  int32_t* pos;                // compact row of token t, or −1
  int32_t* tgt;                // target of compact row i, kTgtElsewhere or kTgtNone
  float* clse;                 // backward: lse of compact row i
  float* cg;                   // backward: gradient weight of compact row i
  int32_t* count;              // number of compact rows
  float* gmax;                 // backward: largest |weight|
};

struct CeStat {
  float m, s;                  // largest logit, Σ exp(z − m)
};

struct CeLogitsArgs {
  const uint16_t* w;           // this piece's rows, [plane][rows][ldw]
  int64_t w_plane, ldw;
  const uint16_t* h;           // compact rows, [plane][tokens][ldh]
  int64_t h_plane, ldh;
  PlanePairs pairs;
  int32_t kt;                  // stages of 32
  int32_t v0, vrows;           // the piece: first vocabulary row, rows
  int32_t tokens;              // compact rows at most
  int32_t tile;                // 256 or 128: the tile's edge
  int32_t tiles_v, tiles_t;
  const int32_t* count;
  const int32_t* tgt;
  // forward
  CeStat* stats;               // [vocabulary tile][tokens]
  float* zt;                   // target's logit
  // backward
  const float* clse;
  const float* cg;
  const float* gmax;
  uint16_t* dz;                // [plane][tokens][ldz]
  int64_t dz_plane;
  int32_t ldz;
};

// losses of few tokens: W in place, hidden states in fragment order
constexpr int kFewTokens = 64; // fp32; bf16 half of them
constexpr int kFewRows = 64;   // vocabulary rows per workgroup and statistics entry
inline int few_tiles(int64_t tokens) { return tokens <= 16 ? 1 : tokens <= 32 ? 2 : 4; }
struct CeFewArgs {
  const void* w;
  int64_t ldw;
  int32_t vec;                 // W's rows are 16-byte aligned
  int32_t width, vocab, tokens;
  int32_t kt;                  // stages of 32 per row of h
  const uint16_t* h;           // [plane][tile of 16 tokens][stage][512]
  int64_t h_plane;
  const int32_t* count;
  const int32_t* tgt;
  CeStat* stats;               // [64 vocabulary rows][tokens]
  float* zt;
};

struct CeRowsArgs {
  const CeStat* stats;
  const float* zt;
  const int32_t* tgt;
  const int32_t* rows;
  const int32_t* count;
  int32_t tokens, tiles_v;
  float* losses;
  float* lse;
};

// ---- gradient products --------------------------------------------------------
// K splits of a product over the tokens that take part, whose number only the
// device knows: the splits were planned for all rows, and the workgroups and the
// partial sums of the tiles that no token reaches go to the others.
struct RowSpread {
  int32_t rows, tiles_r, tile; // rows planned for, their tiles, the tile's edge
  int32_t splits, most;        // splits planned, splits at most
};

// C[row][col] = Σ_k B(k, row)·A(k, col): A's side is contiguous in the output.
struct ProductArgs {
  const uint16_t* a;           // K-major: row k holds A(k, 0 …), [plane][…][lda]
  int64_t a_plane, lda;
  const uint16_t* b;           // K-major like A, or (b_rows) row-major: row r holds B(0 …, r)
  int64_t b_plane, ldb;
  PlanePairs pairs;
  int32_t b_rows;              // 1: b is row-major with K contiguous
  int32_t rows, cols;          // output extent (rows bounded by *count when rows_count)
  int64_t k;                   // K (upper bound when count bounds it)
  const int32_t* count;        // device bound of K (weight gradient) or of the rows (b_rows), or null
  const int32_t* offsets;      // K ranges of `groups` outputs, or null
  int32_t groups;
  int32_t tile;                // 256 or 128: the tile's edge
  int32_t tiles_r, tiles_c, splits;
  RowSpread spread;            // with count and b_rows, instead of tiles_r, splits and part_split
  const float* scale;          // device factor of the result, or null
  void* out;                   // final result: dense rows × cols per group
  int32_t out_f32;
  float* part;                 // [split][group][rows][ldp] fp32 partial sums instead of out
  int64_t part_split;          // elements between splits
  int32_t ldp;
  int32_t add;                 // partial sums add to what is there
};

// out[t][c] = scale·Σ_s part[s][pos[t]][c] (zero where pos[t] < 0)
struct JoinArgs {
  const float* part;
  int64_t part_split;
  int32_t splits, ldp;
  const int32_t* count;        // or null: the splits of `spread` for *count rows, back to back
  RowSpread spread;
  const int32_t* pos;          // or null: t
  const float* scale;          // or null
  int64_t rows;
  int32_t cols;
  void* out;
  int32_t out_f32;
};

// ---- embedding ------------------------------------------------------------------
struct EmbedArgs {
  const void* ids;
  int32_t idx64;
  int32_t f32;                 // table and out
  int64_t tokens, rows;
  int32_t width;
  int32_t unit;                // elements a thread moves at a time: 8 (16-byte rows), 4, 2 or 1
  const void* table;
  int64_t ldt;
  void* out;
  float scale;
};

struct SortArgs {
  const void* ids;             // first pass (keys_in null)
  int32_t idx64;
  int32_t tokens, rows;        // ids outside [0, rows) get the key `rows`
  const uint32_t* keys_in;
  const uint32_t* idx_in;
  uint32_t* keys_out;
  uint32_t* idx_out;
  uint32_t* hist;              // [256][blocks]
  int32_t blocks, shift;
  int32_t key_bits;            // sort by runs: bits of a key
  uint32_t* words;             // the sorted runs, where there are several
};

struct EmbedGradArgs {
  const uint32_t* keys;        // sorted
  const uint32_t* idx;
  int32_t tokens, rows, width;
  int32_t padding;             // id whose gradient row is zero, or −1
  const void* grad;
  int64_t ldg;
  int32_t grad_f32, out_f32, accumulate;
  int32_t vec_in, vec_out;
  int32_t zero_rows;           // table rows per workgroup that clears rows
  float scale;
  void* out;
  int32_t slabs;               // ceil(width / 512)
  int64_t seg_wg;              // workgroups of the sums
  float* part[2];              // sums of whole aligned runs of 32 and 1024 equal keys
};

// ---- 8-bit checkpoints -----------------------------------------------------------
struct CodecArgs {
  const void* x;               // rows × cols, row stride ldx
  int64_t ldx;
  int32_t f32;                 // type of x, or of out
  int32_t cols, blocks;        // blocks = ceil(cols / 32)
  int64_t rows;
  int32_t vec;
  int8_t* q;                   // rows × cols
  uint8_t* exps;               // rows × blocks
  void* out;                   // read back: rows × ldo
  int64_t ldo;
};

constexpr int kSortItems = 4096;         // per workgroup of a sort pass
constexpr int kRun = 32;                 // sorted tokens per first-level sum, and those per second-level one
constexpr int kEmbedRows = 16;           // table rows per workgroup that clears rows, at least (kThreads at most)
constexpr int kEmbedHeads = 8;           // sorted positions per wave that sums ranges
constexpr int kSortRunBits = 13;
constexpr int kSortRun = 1 << kSortRunBits;            // tokens per run of the two-launch sort
constexpr int kSortRunsMax = 65536;                    // tokens it takes

int launch_pack(const PackArgs& a, int phase, void* stream);
int launch_ce_scan(const CeScanArgs& a, void* stream);
int launch_ce_logits(const CeLogitsArgs& a, int backward, int f32, void* stream);
int launch_ce_few_start(const CeScanArgs& a, const PackArgs& p, void* stream);
int launch_ce_few(const CeFewArgs& a, int f32, void* stream);
int launch_ce_rows(const CeRowsArgs& a, void* stream);
int launch_product(const ProductArgs& a, int phase, void* stream);
int launch_join(const JoinArgs& a, int phase, void* stream);
int launch_embed(const EmbedArgs& a, void* stream);
int launch_sort_runs(const SortArgs& a, void* stream);
int launch_sort_pass(const SortArgs& a, void* stream);
int launch_embed_run(const EmbedGradArgs& a, int level, void* stream);
int launch_embed_grad(const EmbedGradArgs& a, void* stream);
int launch_ckpt_quantize(const CodecArgs& a, void* stream);
int launch_ckpt_read(const CodecArgs& a, int phase, void* stream);

}  // namespace dmuon
