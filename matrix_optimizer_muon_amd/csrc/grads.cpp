// C entry points of the training gradients: cross entropy over a large
// vocabulary, embedding lookup and gradient, 8-bit activation checkpoints and the
// weight gradient computed from them.  Validation and planning on the host, then
// launches on the caller's stream; every buffer is the caller's.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <numeric>
#include <string>
#include <vector>

#include "../../include/dmuon_ns.h"
#include "grads.hpp"
#include "host.hpp"

namespace dmuon {
namespace {

static_assert(kElsewhere == DMUON_TARGET_ELSEWHERE, "the kernels' value is the header's");

constexpr int64_t kMaxTokens = (int64_t)1 << 24;    // rows of one cross-entropy or wgrad call
constexpr int64_t kMaxIds = (int64_t)1 << 30;       // ids of one embedding call
constexpr int64_t kMaxWidth = 65536;
constexpr int64_t kMaxRows = (int64_t)1 << 30;      // vocabulary, table rows
constexpr int64_t kMaxLd = (int64_t)1 << 20;        // row strides the kernels take in place
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxExtent = (int64_t)1 << 48;    // bytes of a strided matrix: the largest dense one (2^30 × 65536 fp32)

// A launch takes fewer than 2^32 threads.
bool launchable(int64_t workgroups, int64_t threads) { return workgroups < ((int64_t)1 << 32) / threads; }

// C entry bodies: nothing thrown on the host leaves them.  Where an allocation failed the
// message must not need one: it fits a string's own 15 bytes.
template <typename F>
int guarded(F&& f) {
  clear_error();
  try {
    return f();
  } catch (...) {
    return fail(DMUON_E_HIP, "out of memory");
  }
}

int hip_fail(int e) { return fail(DMUON_E_HIP, std::string("launch failed: ") + hip_error_string(e)); }

// one launch under the debugging switches
template <typename F>
int go(const CallEnv& env, int phase, void* stream, F&& launch) {
  int e = forced(env, phase);
  if (e) return e;
  const int r = launch();
  if (r) return hip_fail(r);
  return settle(env, stream, phase_name(phase));
}

bool float_type(int32_t t) { return t == DMUON_F32 || t == DMUON_BF16; }
int64_t type_bytes(int32_t t) { return t == DMUON_F32 ? 4 : 2; }
bool index_type(int32_t t) { return t == DMUON_I32 || t == DMUON_I64; }

void add_range(std::vector<Range>& rs, const void* p, int64_t bytes, bool ro) {
  if (p && bytes > 0) rs.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, ro});
}
// rows × cols elements of es bytes at a stride of ld (≥ cols, checked before) end within kMaxExtent
bool spans(int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  return rows <= 1 || ld <= (kMaxExtent / es - cols) / (rows - 1);
}
int64_t strided_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  return rows > 0 ? ((rows - 1) * ld + cols) * es : 0;
}

// the workspace's size, and that it meets none of the call's buffers
int check_ws(void* ws, size_t have, size_t need, const std::vector<Range>& rs) {
  int e = check_workspace(ws, have, need);
  if (e) return e;
  const uintptr_t lo = (uintptr_t)ws, hi = lo + need;
  for (const Range& r : rs)
    if (r.lo < hi && lo < r.hi) return fail(DMUON_E_ALIAS, "workspace overlaps a buffer of the call");
  return DMUON_OK;
}

struct Carver {
  char* base;
  size_t off = 0;
  template <typename T>
  T* take(int64_t n) {
    T* p = base ? (T*)(base + off) : nullptr;
    off = align256(off + (size_t)std::max<int64_t>(n, 1) * sizeof(T));
    return p;
  }
};

// Edge of a product's tiles and the K splits that share a tile's sum.
struct Shape {
  int tile, splits;
};

// rows × cols outputs, K of k and `pairs` plane products, `groups` of them.  The
// large core (256², one workgroup per CU) does four times the work of the small
// one (128², three per CU) in the same stage of 32 and loses only where there is
// too little work to fill the CUs: it is taken from 14 of its stages per CU on.
// Measured, checkpoint weight gradients [n, k] over T tokens, small against large,
// each with its best split: 512² over 8192 (4 stages) 35.0 and 38.0 µs, 1536² over
// 2048 (9) 40.0 and 41.0, 1024² over 8192 (16) 50.0 and 48.8, 2048² over 2048 (16)
// 49.2 and 46.5, 4096×3584 over 512 (14) 39.0 and 30.8, 2048×1024 over 32768 (128)
// 217 and 146, 4096² over 32768 1986 and 904.
// The splits take the least of: rounds of workgroups × (stages of each + 6 for its
// fill, drain and stores), plus the partial sums' way through memory and the join.
// Measured, large, 2048² over 8192 tokens: 1, 2, 3, 4 and 8 splits take 152, 115,
// 95, 88 and 109 µs; 2048×1024 over 32768: 4, 6, 8, 12 and 16 take 168, 165, 146,
// 185 and 168.
Shape pick_shape(int64_t rows, int64_t cols, int64_t k, int64_t pairs, int64_t groups) {
  const int64_t stages = std::max<int64_t>(cdiv(k, 32), 1);
  const bool large = cdiv(rows, 256) * cdiv(cols, 256) * groups * stages * pairs >= 14 * 256;
  const int64_t tile = large ? 256 : 128, slots = large ? 256 : 512;
  const int64_t tiles = std::max<int64_t>(cdiv(rows, tile) * cdiv(cols, tile) * groups, 1);
  const double part = large ? 0.09 : 0.033;            // one partial tile, in stages
  int best = 1;
  double least = 0;
  for (int64_t s = 1; s <= 64 && (s == 1 || (stages * pairs >= 8 * s && stages >= 2 * s && tiles * s <= 4 * slots)); ++s) {
    const double cost = (double)cdiv(tiles * s, slots) * (double)(cdiv(stages, s) * pairs + 6) +
                        (s > 1 ? 10 + part * (double)(tiles * s) : 0);
    if (s == 1 || cost < least) {
      least = cost;
      best = (int)s;
    }
  }
  return {(int)tile, best};
}

// Edge of the logits' tiles, which have no splits.  Measured, forward over D
// columns, small against large: 128 large tiles, D 1024 37.4 and 48.5 µs, D 4096 92
// and 116; 256 large tiles, D 256 33.2 and 35.8, D 768 49.0 and 45.4, D 4096 165
// and 131; 2048 large tiles, D 512 172 and 183, D 1024 306 and 273, D 4096 1284 and 883.
int pick_logits_tile(int64_t tokens, int64_t vocab, int64_t k) {
  return cdiv(tokens, 256) * cdiv(vocab, 256) >= 192 && k >= 768 ? 256 : 128;
}

// May the core read this bf16 matrix K-major in place?  16-byte rows, and no tile
// column may reach past the last row's end: the rows touch, or whole tiles.
bool kmajor_in_place(const void* p, int64_t ld, int64_t cols) {
  return ((uintptr_t)p & 15) == 0 && ld % 8 == 0 && ld <= kMaxLd && (ld == cols || cols % kTile == 0);
}

// ---- cross entropy ------------------------------------------------------------
// Bytes of gradient logits (and operand copies of W) that one piece of the
// vocabulary may take.
constexpr int64_t kPieceBytes = (int64_t)256 << 20;

struct CePlan {
  bool f32, direct_w, few;
  int planes;
  int64_t T, D, V, ldd, piece, ldz;
  int tile_z, tiles_v;                   // logits
  Shape sh, sw;                          // hidden-state and weight gradient
  RowSpread spread;                      // of the hidden states' gradient
  // workspace
  int32_t *rows, *pos, *tgt, *count;
  float *clse, *cg, *gmax, *zt, *part_h, *part_w;
  uint16_t *h, *hb, *w, *dz;
  int64_t hb_plane;
  CeStat* stats;
  size_t bytes;
  bool hb_used() const { return few || tile_z == kTile; }       // the logits read fragment order
};

CePlan ce_plan(const dmuon_ce_problem& p, bool backward, char* base) {
  CePlan pl{};
  pl.f32 = p.dtype == DMUON_F32;
  pl.planes = pl.f32 ? kPlanes : 1;
  pl.T = p.tokens;
  pl.D = p.width;
  pl.V = p.vocab;
  pl.ldd = round_up(pl.D, kLdAlign);
  pl.few = !backward && pl.T <= (pl.f32 ? kFewTokens : kFewTokens / 2) && launchable(cdiv(pl.V, kFewRows), kThreads);
  pl.direct_w = pl.few || (!pl.f32 && pl.D % kLdAlign == 0 && kmajor_in_place(p.w, p.ldw, pl.D));
  // the piece: gradient logits of every token (backward) and the copy of W's rows
  const int64_t per_row = (backward ? pl.T * 2 * pl.planes : 0) + (pl.direct_w ? 0 : pl.ldd * 2 * pl.planes);
  int64_t piece = per_row ? std::max<int64_t>(kPieceBytes / per_row, 8 * kTile) : pl.V;
  if (backward) piece = std::min(piece, kMaxLd);       // also the rows' stride of the gradient logits
  // and what one launch of the logits' tiles takes, of either size: whole tiles of 256, 63 at least
  const int64_t most_tiles = ((int64_t)1 << 24) - 1;   // workgroups of 256 threads, a tile of 128 rows each
  piece = std::min(piece, most_tiles / cdiv(pl.T, 128) * 128 / kTile * kTile);
  // equal pieces; where several fill the limit, of as many tile rows as make whole
  // rounds of the weight gradient's tiles over the CUs
  const int64_t n = cdiv(pl.V, std::min(piece, pl.V)), tiles_d = cdiv(pl.D, kTile);
  pl.piece = round_up(cdiv(pl.V, n), kTile);
  const int64_t whole = round_up(pl.piece, 256 / std::gcd(tiles_d, (int64_t)256) * kTile);
  if (n > 1 && backward && whole <= piece) pl.piece = whole;
  pl.ldz = round_up(std::min(pl.piece, pl.V), kLdAlign);
  const int64_t piece_rows = std::min(pl.piece, pl.V);
  const int pairs = pl.f32 ? plane_pairs(pl.planes, pl.planes).n : 1;
  pl.tile_z = pick_logits_tile(pl.T, piece_rows, pl.ldd * pairs);
  pl.tiles_v = (int)cdiv(pl.V, pl.few ? kFewRows : pl.tile_z);
  pl.sh = pick_shape(pl.T, pl.D, piece_rows, pairs, 1);
  const int64_t most = std::min<int64_t>(64, cdiv(piece_rows, 32) * pairs / 8);
  pl.spread = {(int32_t)pl.T, (int32_t)cdiv(pl.T, pl.sh.tile), pl.sh.tile, pl.sh.splits, std::max(pl.sh.splits, (int32_t)most)};
  pl.sw = pick_shape(piece_rows, pl.D, pl.T, pairs, 1);
  Carver c{base};
  pl.rows = c.take<int32_t>(pl.T);
  pl.tgt = c.take<int32_t>(pl.T);
  pl.count = c.take<int32_t>(1);
  // hidden states: the large logits read fragment order, the rest rows
  pl.hb_plane = (pl.few ? few_tiles(pl.T) * 16 : round_up(pl.T, 16)) * pl.ldd;
  if (pl.hb_used()) pl.hb = c.take<uint16_t>(pl.planes * pl.hb_plane);
  if (backward || !pl.hb_used()) pl.h = c.take<uint16_t>(pl.planes * pl.T * pl.ldd);
  if (!pl.direct_w) pl.w = c.take<uint16_t>(pl.planes * piece_rows * pl.ldd);
  if (backward) {
    pl.pos = c.take<int32_t>(pl.T);
    pl.clse = c.take<float>(pl.T);
    pl.cg = c.take<float>(pl.T);
    pl.gmax = c.take<float>(1);
    pl.dz = c.take<uint16_t>(pl.planes * pl.T * pl.ldz);
    pl.part_h = c.take<float>(pl.sh.splits * pl.T * pl.ldd);
    if (pl.sw.splits > 1) pl.part_w = c.take<float>(pl.sw.splits * piece_rows * pl.ldd);
  } else {
    pl.zt = c.take<float>(pl.T);
    pl.stats = c.take<CeStat>((int64_t)pl.tiles_v * pl.T);
  }
  pl.bytes = c.off;
  return pl;
}

int check_ce(const dmuon_ce_problem* p, bool backward, std::vector<Range>* rs) {
  if (!p) return fail(DMUON_E_NULL, "problem is NULL");
  if (!float_type(p->dtype)) return fail(DMUON_E_DTYPE, "dtype must be DMUON_F32 or DMUON_BF16");
  if (!index_type(p->index_dtype)) return fail(DMUON_E_DTYPE, "index_dtype must be DMUON_I32 or DMUON_I64");
  if (p->tokens < 0 || p->tokens > kMaxTokens) return fail(DMUON_E_SHAPE, "tokens must be in [0, 2^24]");
  if (p->width < 1 || p->width > kMaxWidth) return fail(DMUON_E_SHAPE, "width must be in [1, 65536]");
  if (p->vocab < 1 || p->vocab > kMaxRows) return fail(DMUON_E_SHAPE, "vocab must be in [1, 2^30]");
  if (p->ldh < p->width || p->ldw < p->width || p->ldh > kMaxStride || p->ldw > kMaxStride)
    return fail(DMUON_E_SHAPE, "ldh and ldw must be at least width");
  const int64_t es = type_bytes(p->dtype);
  if (!spans(p->tokens, p->width, p->ldh, es) || !spans(p->vocab, p->width, p->ldw, es))
    return fail(DMUON_E_SHAPE, "h and w must end within 2^48 bytes");
  if (cdiv(p->tokens, 128) * cdiv(p->vocab, 128) > INT32_MAX) return fail(DMUON_E_SHAPE, "tokens × vocab is too large");
  // the hidden states' gradient in one launch (of the large tiles, at such a size; the
  // logits and the weight gradient go by pieces that fit)
  if (backward && !launchable(cdiv(p->tokens, 256) * cdiv(p->width, 256), 512))
    return fail(DMUON_E_SHAPE, "tokens × width is too large for one launch");
  if (p->tokens > 0 && (!p->h || !p->targets)) return fail(DMUON_E_NULL, "h and targets must be set");
  if (!p->w) return fail(DMUON_E_NULL, "w must be set");
  if (rs) {
    add_range(*rs, p->h, strided_bytes(p->tokens, p->width, p->ldh, es), true);
    add_range(*rs, p->w, strided_bytes(p->vocab, p->width, p->ldw, es), true);
    add_range(*rs, p->targets, p->tokens * (p->index_dtype == DMUON_I64 ? 8 : 4), true);
  }
  return DMUON_OK;
}

// the compact list of tokens and the operand copy of their hidden states
int ce_start(const dmuon_ce_problem& p, const CePlan& pl, bool backward, const float* lse_in, const float* grad_losses,
             float* losses, float* lse, const CallEnv& env, void* stream) {
  CeScanArgs s{};
  s.targets = p.targets;
  s.idx64 = p.index_dtype == DMUON_I64;
  s.backward = backward;
  s.ignore = p.ignore_index;
  s.tokens = (int32_t)pl.T;
  s.vocab = (int32_t)pl.V;
  s.grad_losses = grad_losses;
  s.lse_in = lse_in;
  s.losses = losses;
  s.lse = lse;
  s.rows = pl.rows;
  s.pos = pl.pos;
  s.tgt = pl.tgt;
  s.clse = pl.clse;
  s.cg = pl.cg;
  s.count = pl.count;
  s.gmax = pl.gmax;
  PackArgs a{};
  a.src = p.h;
  a.ld = p.ldh;
  a.f32 = pl.f32;
  a.cols = (int32_t)pl.D;
  a.rows = pl.T;
  a.gather = pl.rows;
  a.count = pl.count;
  a.dst = pl.h;
  a.plane = pl.T * pl.ldd;
  a.blocks = pl.hb;
  a.blocks_plane = pl.hb_plane;
  a.ldd = (int32_t)pl.ldd;
  if (pl.few) return go(env, PH_CE_PACK, stream, [&] { return launch_ce_few_start(s, a, stream); });
  int e = go(env, PH_CE_PACK, stream, [&] { return launch_ce_scan(s, stream); });
  if (e) return e;
  return go(env, PH_CE_PACK, stream, [&] { return launch_pack(a, PH_CE_PACK, stream); });
}

// one piece of W as the core reads it
int ce_piece(const dmuon_ce_problem& p, const CePlan& pl, int64_t v0, int64_t rows, const uint16_t** w, int64_t* ldw,
             int64_t* plane, const CallEnv& env, void* stream) {
  if (pl.direct_w) {
    *w = (const uint16_t*)p.w + v0 * p.ldw;
    *ldw = p.ldw;
    *plane = 0;
    return DMUON_OK;
  }
  PackArgs a{};
  a.src = (const char*)p.w + v0 * p.ldw * type_bytes(p.dtype);
  a.ld = p.ldw;
  a.f32 = pl.f32;
  a.cols = (int32_t)pl.D;
  a.rows = rows;
  a.dst = pl.w;
  a.plane = rows * pl.ldd;
  a.ldd = (int32_t)pl.ldd;
  *w = pl.w;
  *ldw = pl.ldd;
  *plane = a.plane;
  return go(env, PH_CE_PACK, stream, [&] { return launch_pack(a, PH_CE_PACK, stream); });
}

CeLogitsArgs logits_args(const CePlan& pl, const uint16_t* w, int64_t ldw, int64_t w_plane, int64_t v0, int64_t rows) {
  CeLogitsArgs g{};
  g.w = w;
  g.w_plane = w_plane;
  g.ldw = ldw;
  g.h = pl.hb_used() ? pl.hb : pl.h;
  g.h_plane = pl.hb_used() ? pl.hb_plane : pl.T * pl.ldd;
  g.ldh = pl.ldd;
  g.pairs = plane_pairs(pl.planes, pl.planes);
  g.kt = (int32_t)(pl.ldd / 32);
  g.v0 = (int32_t)v0;
  g.vrows = (int32_t)rows;
  g.tokens = (int32_t)pl.T;
  g.tile = pl.tile_z;
  g.tiles_v = (int32_t)cdiv(rows, pl.tile_z);
  g.tiles_t = (int32_t)cdiv(pl.T, pl.tile_z);
  g.count = pl.count;
  g.tgt = pl.tgt;
  return g;
}

// zeros, as the join of no partial sums
int fill_zero(void* out, int32_t dtype, int64_t rows, int64_t cols, int phase, const CallEnv& env, void* stream) {
  if (rows * cols == 0) return DMUON_OK;
  JoinArgs j{};
  j.rows = rows;
  j.cols = (int32_t)cols;
  j.out = out;
  j.out_f32 = dtype == DMUON_F32;
  return go(env, phase, stream, [&] { return launch_join(j, phase, stream); });
}

// ---- weight gradient from a checkpoint ------------------------------------------
struct WgradPlan {
  bool direct_g;
  int planes;
  Shape shape;
  int64_t ldn, ldk, tiles_r, tiles_c;
  uint16_t *x, *g;
  float* part;
  size_t bytes;
};

WgradPlan wgrad_plan(const dmuon_ckpt8_wgrad_problem& p, char* base) {
  WgradPlan pl{};
  pl.planes = p.grad_dtype == DMUON_F32 ? kPlanes : 1;
  pl.direct_g = p.grad_dtype == DMUON_BF16 && kmajor_in_place(p.grad_out, p.ldg, p.n);
  pl.ldn = round_up(p.n, kLdAlign);
  pl.ldk = round_up(p.k, kLdAlign);
  const int64_t groups = p.offsets ? p.groups : 1, k = p.tokens / std::max<int64_t>(groups, 1);
  pl.shape = pick_shape(p.n, p.k, k, plane_pairs(1, pl.planes).n, groups);
  pl.tiles_r = cdiv(p.n, pl.shape.tile);
  pl.tiles_c = cdiv(p.k, pl.shape.tile);
  Carver c{base};
  pl.x = c.take<uint16_t>(p.tokens * pl.ldk);
  if (!pl.direct_g) pl.g = c.take<uint16_t>(pl.planes * p.tokens * pl.ldn);
  if (pl.shape.splits > 1) pl.part = c.take<float>(pl.shape.splits * groups * p.n * pl.ldk);
  pl.bytes = c.off;
  return pl;
}

int check_wgrad(const dmuon_ckpt8_wgrad_problem* p, std::vector<Range>* rs) {
  if (!p) return fail(DMUON_E_NULL, "problem is NULL");
  if (!float_type(p->grad_dtype) || !float_type(p->out_dtype))
    return fail(DMUON_E_DTYPE, "grad_dtype and out_dtype must be DMUON_F32 or DMUON_BF16");
  if (p->tokens < 0 || p->tokens > kMaxTokens) return fail(DMUON_E_SHAPE, "tokens must be in [0, 2^24]");
  if (p->n < 1 || p->n > kMaxWidth || p->k < 1 || p->k > kMaxWidth) return fail(DMUON_E_SHAPE, "n and k must be in [1, 65536]");
  if (p->ldg < p->n || p->ldg > kMaxStride) return fail(DMUON_E_SHAPE, "ldg must be at least n");
  if (!spans(p->tokens, p->n, p->ldg, type_bytes(p->grad_dtype))) return fail(DMUON_E_SHAPE, "grad_out must end within 2^48 bytes");
  if (p->groups < 0 || p->groups > (1 << 20)) return fail(DMUON_E_SHAPE, "groups must be in [0, 2^20]");
  if (p->reserved != 0) return fail(DMUON_E_SHAPE, "reserved must be 0");
  if (!p->offsets && p->groups > 1) return fail(DMUON_E_NULL, "offsets must be set for more than one group");
  const int64_t groups = p->offsets ? p->groups : 1;
  if (cdiv(p->n, 128) * cdiv(p->k, 128) * std::max<int64_t>(groups, 1) > INT32_MAX / 768)
    return fail(DMUON_E_SHAPE, "too many workgroups in one launch");
  if (p->tokens > 0 && (!p->grad_out || !p->q || !p->exps)) return fail(DMUON_E_NULL, "grad_out, q and exps must be set");
  if (groups > 0 && !p->out) return fail(DMUON_E_NULL, "out must be set");
  if (rs) {
    add_range(*rs, p->grad_out, strided_bytes(p->tokens, p->n, p->ldg, type_bytes(p->grad_dtype)), true);
    add_range(*rs, p->q, p->tokens * p->k, true);
    add_range(*rs, p->exps, p->tokens * cdiv(p->k, 32), true);
    add_range(*rs, p->offsets, (groups + 1) * 4, true);
    add_range(*rs, p->out, groups * p->n * p->k * type_bytes(p->out_dtype), false);
  }
  return DMUON_OK;
}

// ---- embedding ------------------------------------------------------------------
struct EmbedPlan {
  uint32_t *keys[2], *idx[2], *hist, *words;
  float* part[2];
  int blocks, passes, key_bits;
  bool runs;                             // the sort by runs
  size_t bytes;
};

EmbedPlan embed_plan(int64_t tokens, int64_t rows, int64_t width, char* base) {
  EmbedPlan pl{};
  pl.blocks = (int)cdiv(tokens, kSortItems);
  while (rows >> pl.key_bits) ++pl.key_bits;           // keys are 0 … rows
  pl.runs = tokens <= kSortRunsMax && rows + 1 < (int64_t)1 << (32 - kSortRunBits);   // id + 1 fits beside an index
  pl.passes = (int)cdiv(pl.key_bits, 8);
  Carver c{base};
  for (int i = 0; i < (pl.runs ? 1 : 2); ++i) {
    pl.keys[i] = c.take<uint32_t>(tokens);
    pl.idx[i] = c.take<uint32_t>(tokens);
  }
  if (!pl.runs) pl.hist = c.take<uint32_t>((int64_t)256 * pl.blocks);
  else if (tokens > kSortRun) pl.words = c.take<uint32_t>(tokens);
  const int64_t ld = round_up(width, 8);
  int64_t span = kRun;
  for (int l = 0; l < 2; ++l, span *= kRun) pl.part[l] = c.take<float>(tokens / span * ld);
  pl.bytes = c.off;
  return pl;
}

int check_embed_sizes(int64_t tokens, int64_t rows, int64_t width) {
  if (tokens < 0 || tokens > kMaxIds) return fail(DMUON_E_SHAPE, "tokens must be in [0, 2^30]");
  if (rows < 0 || rows > kMaxRows) return fail(DMUON_E_SHAPE, "rows must be in [0, 2^30]");
  if (width < 1 || width > kMaxWidth) return fail(DMUON_E_SHAPE, "width must be in [1, 65536]");
  return DMUON_OK;
}

// table rows per workgroup that clears rows, and workgroups of the sums
int64_t embed_zero_rows(int64_t width, int64_t es) {
  return std::clamp<int64_t>(32768 / (width * es), kEmbedRows, kThreads);
}
int64_t embed_sum_groups(int64_t tokens, int64_t width) { return cdiv(tokens, kEmbedHeads * (kThreads / 64)) * cdiv(width, 512); }

// the gradient's largest launches: the sums with the rows that are cleared (counted for
// an fp32 table), and the run sums, a workgroup per 32 tokens
int check_embed_grad(int64_t tokens, int64_t rows, int64_t width) {
  int e = check_embed_sizes(tokens, rows, width);
  if (e) return e;
  if (!launchable(embed_sum_groups(tokens, width) + cdiv(rows, embed_zero_rows(width, 4)), kThreads))
    return fail(DMUON_E_SHAPE, "tokens × width or rows × width is too large for one launch");
  return DMUON_OK;
}

int check_codec(int64_t rows, int64_t cols, int32_t dtype) {
  if (!float_type(dtype)) return fail(DMUON_E_DTYPE, "dtype must be DMUON_F32 or DMUON_BF16");
  if (rows < 0 || rows > kMaxIds) return fail(DMUON_E_SHAPE, "rows must be in [0, 2^30]");
  if (cols < 0 || cols > kMaxWidth) return fail(DMUON_E_SHAPE, "cols must be in [0, 65536]");
  return DMUON_OK;
}

bool rows16(const void* p, int64_t ld, int64_t cols, int64_t es) {
  return ((uintptr_t)p & 15) == 0 && ld * es % 16 == 0 && cols % 8 == 0;
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_linear_ce_workspace_size(const dmuon_ce_problem* p, int32_t backward, size_t* bytes) {
  return guarded([&]() -> int {
    if (!bytes) return fail(DMUON_E_NULL, "bytes is NULL");
    if (backward != 0 && backward != 1) return fail(DMUON_E_CFG, "backward must be 0 or 1");
    int e = check_ce(p, backward != 0, nullptr);
    if (e) return e;
    *bytes = p->tokens ? ce_plan(*p, backward != 0, nullptr).bytes : 0;
    return DMUON_OK;
  });
}

int dmuon_linear_ce(const dmuon_ce_problem* p, float* losses, float* lse, void* workspace, size_t workspace_bytes,
                    void* stream) {
  return guarded([&]() -> int {
    std::vector<Range> rs;
    int e = check_ce(p, false, &rs);
    if (e) return e;
    if (p->tokens == 0) return DMUON_OK;
    if (!losses || !lse) return fail(DMUON_E_NULL, "losses and lse must be set");
    add_range(rs, losses, p->tokens * 4, false);
    add_range(rs, lse, p->tokens * 4, false);
    if ((e = check_alias(rs))) return e;
    if ((e = check_ws(workspace, workspace_bytes, ce_plan(*p, false, nullptr).bytes, rs))) return e;
    const CePlan pl = ce_plan(*p, false, (char*)workspace);
    const CallEnv env = call_env();
    if ((e = forced(env, -2))) return e;
    if ((e = ce_start(*p, pl, false, nullptr, nullptr, losses, lse, env, stream))) return e;
    if (pl.few) {
      CeFewArgs f{};
      f.w = p->w;
      f.ldw = p->ldw;
      f.vec = ((uintptr_t)p->w & 15) == 0 && p->ldw * type_bytes(p->dtype) % 16 == 0;
      f.width = (int32_t)pl.D;
      f.vocab = (int32_t)pl.V;
      f.tokens = (int32_t)pl.T;
      f.kt = (int32_t)(pl.ldd / 32);
      f.h = pl.hb;
      f.h_plane = pl.hb_plane;
      f.count = pl.count;
      f.tgt = pl.tgt;
      f.stats = pl.stats;
      f.zt = pl.zt;
      if ((e = go(env, PH_CE_LOGITS, stream, [&] { return launch_ce_few(f, pl.f32, stream); }))) return e;
    }
    for (int64_t v0 = 0; v0 < pl.V && !pl.few; v0 += pl.piece) {
      const int64_t rows = std::min(pl.piece, pl.V - v0);
      const uint16_t* w;
      int64_t ldw, plane;
      if ((e = ce_piece(*p, pl, v0, rows, &w, &ldw, &plane, env, stream))) return e;
      CeLogitsArgs g = logits_args(pl, w, ldw, plane, v0, rows);
      g.stats = pl.stats;
      g.zt = pl.zt;
      if ((e = go(env, PH_CE_LOGITS, stream, [&] { return launch_ce_logits(g, 0, pl.f32, stream); }))) return e;
    }
    CeRowsArgs r{};
    r.stats = pl.stats;
    r.zt = pl.zt;
    r.tgt = pl.tgt;
    r.rows = pl.rows;
    r.count = pl.count;
    r.tokens = (int32_t)pl.T;
    r.tiles_v = pl.tiles_v;
    r.losses = losses;
    r.lse = lse;
    return go(env, PH_CE_ROWS, stream, [&] { return launch_ce_rows(r, stream); });
  });
}

int dmuon_linear_ce_backward(const dmuon_ce_problem* p, const float* lse, const float* grad_losses, void* grad_h,
                             void* grad_w, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    std::vector<Range> rs;
    int e = check_ce(p, true, &rs);
    if (e) return e;
    if (!grad_h && !grad_w) return DMUON_OK;
    if (p->tokens > 0 && (!lse || !grad_losses)) return fail(DMUON_E_NULL, "lse and grad_losses must be set");
    const int64_t es = type_bytes(p->dtype);
    add_range(rs, lse, p->tokens * 4, true);
    add_range(rs, grad_losses, p->tokens * 4, true);
    add_range(rs, grad_h, p->tokens * p->width * es, false);
    add_range(rs, grad_w, p->vocab * p->width * es, false);
    if ((e = check_alias(rs))) return e;
    const CallEnv env = call_env();
    if (p->tokens == 0) {
      if ((e = forced(env, -2))) return e;
      return grad_w ? fill_zero(grad_w, p->dtype, p->vocab, p->width, PH_CE_GRADS, env, stream) : DMUON_OK;
    }
    if ((e = check_ws(workspace, workspace_bytes, ce_plan(*p, true, nullptr).bytes, rs))) return e;
    const CePlan pl = ce_plan(*p, true, (char*)workspace);
    if ((e = forced(env, -2))) return e;
    if ((e = ce_start(*p, pl, true, lse, grad_losses, nullptr, nullptr, env, stream))) return e;
    for (int64_t v0 = 0; v0 < pl.V; v0 += pl.piece) {
      const int64_t rows = std::min(pl.piece, pl.V - v0);
      const uint16_t* w;
      int64_t ldw, plane;
      if ((e = ce_piece(*p, pl, v0, rows, &w, &ldw, &plane, env, stream))) return e;
      CeLogitsArgs g = logits_args(pl, w, ldw, plane, v0, rows);
      g.clse = pl.clse;
      g.cg = pl.cg;
      g.gmax = pl.gmax;
      g.dz = pl.dz;
      g.dz_plane = pl.T * pl.ldz;
      g.ldz = (int32_t)pl.ldz;
      if ((e = go(env, PH_CE_LOGITS, stream, [&] { return launch_ce_logits(g, 1, pl.f32, stream); }))) return e;
      if (grad_w) {
        ProductArgs q{};
        q.a = pl.h;
        q.a_plane = pl.T * pl.ldd;
        q.lda = pl.ldd;
        q.b = pl.dz;
        q.b_plane = g.dz_plane;
        q.ldb = pl.ldz;
        q.pairs = plane_pairs(pl.planes, pl.planes);
        q.rows = (int32_t)rows;
        q.cols = (int32_t)pl.D;
        q.k = pl.T;
        q.count = pl.count;
        q.groups = 1;
        q.tile = pl.sw.tile;
        q.tiles_r = (int32_t)cdiv(rows, q.tile);
        q.tiles_c = (int32_t)cdiv(pl.D, q.tile);
        q.splits = pl.sw.splits;
        q.scale = pl.gmax;
        q.out = (char*)grad_w + v0 * pl.D * es;
        q.out_f32 = pl.f32;
        if (q.splits > 1) {
          q.part = pl.part_w;
          q.ldp = (int32_t)pl.ldd;
          q.part_split = rows * pl.ldd;
        }
        if ((e = go(env, PH_CE_GRADS, stream, [&] { return launch_product(q, PH_CE_GRADS, stream); }))) return e;
        if (q.splits > 1) {
          JoinArgs j{};
          j.part = q.part;
          j.part_split = q.part_split;
          j.splits = q.splits;
          j.ldp = q.ldp;
          j.scale = pl.gmax;
          j.rows = rows;
          j.cols = (int32_t)pl.D;
          j.out = q.out;
          j.out_f32 = pl.f32;
          if ((e = go(env, PH_CE_GRADS, stream, [&] { return launch_join(j, PH_CE_GRADS, stream); }))) return e;
        }
      }
      if (grad_h) {
        ProductArgs q{};
        q.a = w;
        q.a_plane = plane;
        q.lda = ldw;
        q.b = pl.dz;
        q.b_plane = g.dz_plane;
        q.ldb = pl.ldz;
        q.pairs = plane_pairs(pl.planes, pl.planes);
        q.b_rows = 1;
        q.rows = (int32_t)pl.T;
        q.cols = (int32_t)pl.D;
        q.k = rows;
        q.count = pl.count;
        q.groups = 1;
        q.tile = pl.sh.tile;
        q.tiles_r = (int32_t)cdiv(pl.T, q.tile);
        q.tiles_c = (int32_t)cdiv(pl.D, q.tile);
        q.splits = pl.sh.splits;
        q.spread = pl.spread;
        q.part = pl.part_h;
        q.ldp = (int32_t)pl.ldd;
        q.add = v0 > 0;
        if ((e = go(env, PH_CE_GRADS, stream, [&] { return launch_product(q, PH_CE_GRADS, stream); }))) return e;
      }
    }
    if (!grad_h) return DMUON_OK;
    JoinArgs j{};
    j.part = pl.part_h;
    j.count = pl.count;
    j.spread = pl.spread;
    j.ldp = (int32_t)pl.ldd;
    j.pos = pl.pos;
    j.scale = pl.gmax;
    j.rows = pl.T;
    j.cols = (int32_t)pl.D;
    j.out = grad_h;
    j.out_f32 = pl.f32;
    return go(env, PH_CE_GRADS, stream, [&] { return launch_join(j, PH_CE_GRADS, stream); });
  });
}

int dmuon_embedding(const void* ids, int32_t index_dtype, int64_t tokens, const void* table, int64_t ldt, int64_t rows,
                    int64_t width, int32_t dtype, float scale, void* out, void* stream) {
  return guarded([&]() -> int {
    if (!index_type(index_dtype)) return fail(DMUON_E_DTYPE, "index_dtype must be DMUON_I32 or DMUON_I64");
    if (!float_type(dtype)) return fail(DMUON_E_DTYPE, "dtype must be DMUON_F32 or DMUON_BF16");
    int e = check_embed_sizes(tokens, rows, width);
    if (e) return e;
    if (ldt < width || ldt > kMaxStride) return fail(DMUON_E_SHAPE, "ldt must be at least width");
    if (!spans(rows, width, ldt, type_bytes(dtype))) return fail(DMUON_E_SHAPE, "table must end within 2^48 bytes");
    if (!std::isfinite(scale)) return fail(DMUON_E_CFG, "scale must be finite");
    if (tokens == 0) return DMUON_OK;
    if (!ids || !out || (rows > 0 && !table)) return fail(DMUON_E_NULL, "ids, table and out must be set");
    const int64_t es = type_bytes(dtype);
    std::vector<Range> rs;
    add_range(rs, ids, tokens * (index_dtype == DMUON_I64 ? 8 : 4), true);
    add_range(rs, table, strided_bytes(rows, width, ldt, es), true);
    add_range(rs, out, tokens * width * es, false);
    if ((e = check_alias(rs))) return e;
    const CallEnv env = call_env();
    if ((e = forced(env, -2))) return e;
    EmbedArgs a{};
    a.ids = ids;
    a.idx64 = index_dtype == DMUON_I64;
    a.f32 = dtype == DMUON_F32;
    a.tokens = tokens;
    a.rows = rows;
    a.width = (int32_t)width;
    // elements of a row that one thread moves: 8, or what the alignment allows
    const uint64_t align = (uint64_t)(uintptr_t)table | (uint64_t)(uintptr_t)out | (uint64_t)(ldt * es) | (uint64_t)(width * es);
    a.unit = rows16(table, ldt, width, es) && rows16(out, width, width, es) ? 8
             : align % (2 * es) ? 1 : align % (4 * es) ? 2 : 4;
    a.table = table;
    a.ldt = ldt;
    a.out = out;
    a.scale = scale;
    return go(env, PH_EMBED, stream, [&] { return launch_embed(a, stream); });
  });
}

int dmuon_embedding_backward_workspace_size(int64_t tokens, int64_t rows, int64_t width, size_t* bytes) {
  return guarded([&]() -> int {
    if (!bytes) return fail(DMUON_E_NULL, "bytes is NULL");
    int e = check_embed_grad(tokens, rows, width);
    if (e) return e;
    *bytes = tokens && rows ? embed_plan(tokens, rows, width, nullptr).bytes : 0;
    return DMUON_OK;
  });
}

int dmuon_embedding_backward(const void* ids, int32_t index_dtype, int64_t tokens, const void* grad_out, int64_t ldg,
                             int32_t grad_dtype, int64_t rows, int64_t width, float scale, int64_t padding_id,
                             void* grad_table, int32_t out_dtype, int32_t accumulate, void* workspace,
                             size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    if (!index_type(index_dtype)) return fail(DMUON_E_DTYPE, "index_dtype must be DMUON_I32 or DMUON_I64");
    if (!float_type(grad_dtype) || !float_type(out_dtype))
      return fail(DMUON_E_DTYPE, "grad_dtype and out_dtype must be DMUON_F32 or DMUON_BF16");
    int e = check_embed_grad(tokens, rows, width);
    if (e) return e;
    if (ldg < width || ldg > kMaxStride) return fail(DMUON_E_SHAPE, "ldg must be at least width");
    if (!spans(tokens, width, ldg, type_bytes(grad_dtype))) return fail(DMUON_E_SHAPE, "grad_out must end within 2^48 bytes");
    if (!std::isfinite(scale)) return fail(DMUON_E_CFG, "scale must be finite");
    if (accumulate != 0 && accumulate != 1) return fail(DMUON_E_CFG, "accumulate must be 0 or 1");
    if (rows == 0) return DMUON_OK;
    if (!grad_table || (tokens > 0 && (!ids || !grad_out))) return fail(DMUON_E_NULL, "ids, grad_out and grad_table must be set");
    const CallEnv env = call_env();
    if (tokens == 0) {
      if ((e = forced(env, -2))) return e;
      return accumulate ? DMUON_OK : fill_zero(grad_table, out_dtype, rows, width, PH_EMBED_GRAD, env, stream);
    }
    std::vector<Range> rs;
    add_range(rs, ids, tokens * (index_dtype == DMUON_I64 ? 8 : 4), true);
    add_range(rs, grad_out, strided_bytes(tokens, width, ldg, type_bytes(grad_dtype)), true);
    add_range(rs, grad_table, rows * width * type_bytes(out_dtype), false);
    if ((e = check_alias(rs))) return e;
    if ((e = check_ws(workspace, workspace_bytes, embed_plan(tokens, rows, width, nullptr).bytes, rs))) return e;
    const EmbedPlan pl = embed_plan(tokens, rows, width, (char*)workspace);
    if ((e = forced(env, -2))) return e;
    SortArgs s{};
    s.ids = ids;
    s.idx64 = index_dtype == DMUON_I64;
    s.tokens = (int32_t)tokens;
    s.rows = (int32_t)rows;
    s.hist = pl.hist;
    s.blocks = pl.blocks;
    EmbedGradArgs a{};
    if (pl.runs) {
      s.key_bits = pl.key_bits;
      s.words = pl.words;
      a.keys = s.keys_out = pl.keys[0];
      a.idx = s.idx_out = pl.idx[0];
      if ((e = go(env, PH_EMBED_GRAD, stream, [&] { return launch_sort_runs(s, stream); }))) return e;
    } else {
      for (int k = 0; k < pl.passes; ++k) {
        s.keys_in = k ? pl.keys[(k + 1) & 1] : nullptr;
        s.idx_in = k ? pl.idx[(k + 1) & 1] : nullptr;
        a.keys = s.keys_out = pl.keys[k & 1];
        a.idx = s.idx_out = pl.idx[k & 1];
        s.shift = 8 * k;
        if ((e = go(env, PH_EMBED_GRAD, stream, [&] { return launch_sort_pass(s, stream); }))) return e;
      }
    }
    a.tokens = (int32_t)tokens;
    a.rows = (int32_t)rows;
    a.width = (int32_t)width;
    a.padding = padding_id >= 0 && padding_id < rows ? (int32_t)padding_id : -1;
    a.grad = grad_out;
    a.ldg = ldg;
    a.grad_f32 = grad_dtype == DMUON_F32;
    a.out_f32 = out_dtype == DMUON_F32;
    a.accumulate = accumulate;
    a.zero_rows = (int32_t)embed_zero_rows(width, type_bytes(out_dtype));
    a.vec_in = rows16(grad_out, ldg, width, type_bytes(grad_dtype));
    a.vec_out = rows16(grad_table, width, width, type_bytes(out_dtype));
    a.scale = scale;
    a.out = grad_table;
    a.slabs = (int32_t)cdiv(width, 512);
    a.seg_wg = embed_sum_groups(tokens, width);
    for (int l = 0; l < 2; ++l) a.part[l] = pl.part[l];
    int64_t span = kRun;
    for (int l = 0; l < 2 && span <= tokens; ++l, span *= kRun)
      if ((e = go(env, PH_EMBED_GRAD, stream, [&] { return launch_embed_run(a, l, stream); }))) return e;
    return go(env, PH_EMBED_GRAD, stream, [&] { return launch_embed_grad(a, stream); });
  });
}

int dmuon_ckpt8_quantize(const void* x, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, int8_t* q, uint8_t* exps,
                         void* stream) {
  return guarded([&]() -> int {
    int e = check_codec(rows, cols, dtype);
    if (e) return e;
    if (ldx < cols || ldx > kMaxStride) return fail(DMUON_E_SHAPE, "ldx must be at least cols");
    if (!spans(rows, cols, ldx, type_bytes(dtype))) return fail(DMUON_E_SHAPE, "x must end within 2^48 bytes");
    if (rows * cols == 0) return DMUON_OK;
    if (!x || !q || !exps) return fail(DMUON_E_NULL, "x, q and exps must be set");
    const int64_t es = type_bytes(dtype), blocks = cdiv(cols, 32);
    std::vector<Range> rs;
    add_range(rs, x, strided_bytes(rows, cols, ldx, es), true);
    add_range(rs, q, rows * cols, false);
    add_range(rs, exps, rows * blocks, false);
    if ((e = check_alias(rs))) return e;
    const CallEnv env = call_env();
    if ((e = forced(env, -2))) return e;
    CodecArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.f32 = dtype == DMUON_F32;
    a.cols = (int32_t)cols;
    a.blocks = (int32_t)blocks;
    a.rows = rows;
    a.vec = ((uintptr_t)x & 15) == 0 && ldx * es % 16 == 0;
    a.q = q;
    a.exps = exps;
    return go(env, PH_CKPT_CODEC, stream, [&] { return launch_ckpt_quantize(a, stream); });
  });
}

int dmuon_ckpt8_dequantize(const int8_t* q, const uint8_t* exps, int64_t rows, int64_t cols, void* out, int32_t dtype,
                           void* stream) {
  return guarded([&]() -> int {
    int e = check_codec(rows, cols, dtype);
    if (e) return e;
    if (rows * cols == 0) return DMUON_OK;
    if (!q || !exps || !out) return fail(DMUON_E_NULL, "q, exps and out must be set");
    const int64_t es = type_bytes(dtype), blocks = cdiv(cols, 32);
    std::vector<Range> rs;
    add_range(rs, q, rows * cols, true);
    add_range(rs, exps, rows * blocks, true);
    add_range(rs, out, rows * cols * es, false);
    if ((e = check_alias(rs))) return e;
    const CallEnv env = call_env();
    if ((e = forced(env, -2))) return e;
    CodecArgs a{};
    a.f32 = dtype == DMUON_F32;
    a.cols = (int32_t)cols;
    a.blocks = (int32_t)blocks;
    a.rows = rows;
    a.vec = ((uintptr_t)out & 15) == 0 && cols * es % 16 == 0;
    a.q = (int8_t*)q;
    a.exps = (uint8_t*)exps;
    a.out = out;
    a.ldo = cols;
    return go(env, PH_CKPT_CODEC, stream, [&] { return launch_ckpt_read(a, PH_CKPT_CODEC, stream); });
  });
}

int dmuon_ckpt8_wgrad_workspace_size(const dmuon_ckpt8_wgrad_problem* p, size_t* bytes) {
  return guarded([&]() -> int {
    if (!bytes) return fail(DMUON_E_NULL, "bytes is NULL");
    int e = check_wgrad(p, nullptr);
    if (e) return e;
    *bytes = p->tokens && !(p->offsets && p->groups == 0) ? wgrad_plan(*p, nullptr).bytes : 0;
    return DMUON_OK;
  });
}

int dmuon_ckpt8_wgrad(const dmuon_ckpt8_wgrad_problem* p, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    std::vector<Range> rs;
    int e = check_wgrad(p, &rs);
    if (e) return e;
    const int64_t groups = p->offsets ? p->groups : 1;
    if (groups == 0) return DMUON_OK;
    if ((e = check_alias(rs))) return e;
    const CallEnv env = call_env();
    if (p->tokens == 0) {
      if ((e = forced(env, -2))) return e;
      return fill_zero(p->out, p->out_dtype, groups * p->n, p->k, PH_CKPT_WGRAD, env, stream);
    }
    if ((e = check_ws(workspace, workspace_bytes, wgrad_plan(*p, nullptr).bytes, rs))) return e;
    const WgradPlan pl = wgrad_plan(*p, (char*)workspace);
    if ((e = forced(env, -2))) return e;
    CodecArgs r{};
    r.cols = (int32_t)p->k;
    r.blocks = (int32_t)cdiv(p->k, 32);
    r.rows = p->tokens;
    r.vec = 1;
    r.q = (int8_t*)p->q;
    r.exps = (uint8_t*)p->exps;
    r.out = pl.x;
    r.ldo = pl.ldk;
    if ((e = go(env, PH_CKPT_WGRAD, stream, [&] { return launch_ckpt_read(r, PH_CKPT_WGRAD, stream); }))) return e;
    if (!pl.direct_g) {
      PackArgs a{};
      a.src = p->grad_out;
      a.ld = p->ldg;
      a.f32 = p->grad_dtype == DMUON_F32;
      a.cols = (int32_t)p->n;
      a.rows = p->tokens;
      a.dst = pl.g;
      a.plane = p->tokens * pl.ldn;
      a.ldd = (int32_t)pl.ldn;
      if ((e = go(env, PH_CKPT_WGRAD, stream, [&] { return launch_pack(a, PH_CKPT_WGRAD, stream); }))) return e;
    }
    ProductArgs q{};
    q.a = pl.x;
    q.lda = pl.ldk;
    q.b = pl.direct_g ? (const uint16_t*)p->grad_out : pl.g;
    q.ldb = pl.direct_g ? p->ldg : pl.ldn;
    q.b_plane = p->tokens * pl.ldn;
    q.pairs = plane_pairs(1, pl.planes);
    q.rows = (int32_t)p->n;
    q.cols = (int32_t)p->k;
    q.k = p->tokens;
    q.offsets = p->offsets;
    q.groups = (int32_t)groups;
    q.tile = pl.shape.tile;
    q.tiles_r = (int32_t)pl.tiles_r;
    q.tiles_c = (int32_t)pl.tiles_c;
    q.splits = pl.shape.splits;
    q.out = p->out;
    q.out_f32 = p->out_dtype == DMUON_F32;
    if (q.splits > 1) {
      q.part = pl.part;
      q.ldp = (int32_t)pl.ldk;
      q.part_split = groups * p->n * pl.ldk;
    }
    if ((e = go(env, PH_CKPT_WGRAD, stream, [&] { return launch_product(q, PH_CKPT_WGRAD, stream); }))) return e;
    if (q.splits == 1) return DMUON_OK;
    JoinArgs j{};
    j.part = q.part;
    j.part_split = q.part_split;
    j.splits = q.splits;
    j.ldp = q.ldp;
    j.rows = groups * p->n;
    j.cols = (int32_t)p->k;
    j.out = p->out;
    j.out_f32 = q.out_f32;
    return go(env, PH_CKPT_WGRAD, stream, [&] { return launch_join(j, PH_CKPT_WGRAD, stream); });
  });
}

}  // extern "C"
