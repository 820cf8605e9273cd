// C entry points of the log probabilities from logits in memory, with entropies and
// alternatives, and of their gradient.
#include <cmath>
#include <vector>

#include "entry.hpp"
#include "grads.hpp"
#include "logprobs.hpp"

namespace dmuon {
namespace {

constexpr int64_t kMaxVocab = (int64_t)1 << 22;     // words of a row of logits
constexpr int64_t kCaches = (int64_t)256 << 20;     // bytes: what the last cache before memory holds
constexpr int64_t kMaxKeys = 6144;                  // candidates of a row's pieces together, in the joining workgroup's LDS
static_assert(kMaxVocab <= kMaxKeys / kTopMost * (kPieceMost - 16), "the largest vocabulary in pieces that can be joined");

struct RowsPlan {
  bool wave;
  int64_t piece, pieces;
  RowStat* stats;
  uint64_t* cand;
  size_t bytes;
};

// A row is one wave's where it is short, else one workgroup's, or several pieces' where it
// is too long for a workgroup or the rows are too few to fill the card.
RowsPlan rows_plan(const dmuon_logprobs_problem& p, char* base) {
  RowsPlan pl{};
  pl.wave = p.top ? p.vocab <= kWaveTop || (p.vocab <= kWaveTopMost && p.tokens >= kWaveTopRows)
                  : p.vocab <= wave_row(p.dtype == DMUON_F32, p.tokens);
  pl.piece = p.vocab;
  pl.pieces = 1;
  if (pl.wave) return pl;
  int64_t n = p.tokens >= kRowsEnough ? 1 : std::min<int64_t>({cdiv(2048, p.tokens), cdiv(p.vocab, kPieceLeast), kPiecesMost, p.top ? kMaxKeys / p.top : kPiecesMost});
  n = std::max<int64_t>(n, p.vocab <= kPieceMost ? 1 : cdiv(p.vocab, kPieceMost - 16));
  pl.piece = round_up(cdiv(p.vocab, n), 8);
  pl.pieces = cdiv(p.vocab, pl.piece);
  if (pl.pieces > 1 && p.vocab - (pl.pieces - 1) * pl.piece < 16) {    // the last one's rest goes to the others: two units at least
    pl.piece += 16;
    pl.pieces = cdiv(p.vocab, pl.piece);
  }
  // Pieces with alternatives by a wave each, or by a workgroup each where they do not fill
  // the card: 1 × 128000 with 20 alternatives 13.7 and 12.5 µs, 32 × 50257 14.2 and 13.4,
  // 64 × 128000 17.7 and 20.0, with 64 of them 23.8 and 28.
  pl.wave = p.top && pl.piece <= kWaveTop && p.tokens * pl.pieces > 1024;
  if (pl.pieces == 1) return pl;
  Carver c{base};
  pl.stats = c.take<RowStat>(p.tokens * pl.pieces);
  if (p.top) pl.cand = c.take<uint64_t>(p.tokens * pl.pieces * p.top);
  pl.bytes = c.off;
  return pl;
}

int check_rows(const dmuon_logprobs_problem* p, bool backward) {
  if (!p) return fail(DMUON_E_NULL, "problem is NULL");
  if (!float_type(p->dtype)) return fail(DMUON_E_DTYPE, "dtype must be DMUON_F32 or DMUON_BF16");
  if (!index_type(p->index_dtype)) return fail(DMUON_E_DTYPE, "index_dtype must be DMUON_I32 or DMUON_I64");
  if (p->tokens < 0 || p->tokens > kMaxTokens) return fail(DMUON_E_SHAPE, "tokens must be in [0, 2^24]");
  if (p->vocab < 1 || p->vocab > kMaxVocab) return fail(DMUON_E_SHAPE, "vocab must be in [1, 2^22]");
  if (p->ld < p->vocab || p->ld > kMaxStride) return fail(DMUON_E_SHAPE, "ld must be at least vocab");
  if (!spans(p->tokens, p->vocab, p->ld, type_bytes(p->dtype))) return fail(DMUON_E_SHAPE, "logits must end within 2^48 bytes");
  if (!logit_scale(p->scale)) return fail(DMUON_E_CFG, "scale must be in [2^-20, 2^20]");
  if (!backward && (p->top < 0 || p->top > kTopMost || p->top > p->vocab))
    return fail(DMUON_E_CFG, "top must be in [0, 128] and at most vocab");
  if (p->tokens > 0 && !p->logits) return fail(DMUON_E_NULL, "logits must be set");
  if (p->tokens > 0) {
    const RowsPlan pl = backward ? RowsPlan{} : rows_plan(*p, nullptr);
    const bool waves = backward ? p->vocab <= kGradWave : pl.wave;
    const int64_t work = p->tokens * (backward ? cdiv(p->vocab, kThreads * kGradUnits * 8) : pl.pieces);
    if (!launchable(work, waves ? 64 : kThreads)) return fail(DMUON_E_SHAPE, "tokens × vocab is too large for one launch");
  }
  return DMUON_OK;
}

void rows_ranges(const dmuon_logprobs_problem& p, bool logits, std::vector<Range>& rs) {
  rs.reserve(8);
  if (logits) add_range(rs, p.logits, strided_bytes(p.tokens, p.vocab, p.ld, type_bytes(p.dtype)), true);
  add_range(rs, p.targets, p.tokens * (p.index_dtype == DMUON_I64 ? 8 : 4), true);
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_logprobs_workspace_size(const dmuon_logprobs_problem* p, size_t* bytes) {
  return guarded([&]() -> int {
    if (!bytes) return fail(DMUON_E_NULL, "bytes is NULL");
    int e = check_rows(p, false);
    if (e) return e;
    *bytes = p->tokens ? rows_plan(*p, nullptr).bytes : 0;
    return DMUON_OK;
  });
}

int dmuon_logprobs(const dmuon_logprobs_problem* p, float* logprobs, float* entropy, float* lse, int64_t* top_ids,
                   float* top_logprobs, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    int e = check_rows(p, false);
    if (e) return e;
    if (p->tokens == 0) return DMUON_OK;
    if (!entropy || !lse) return fail(DMUON_E_NULL, "entropy and lse must be set");
    if (!logprobs != !p->targets) return fail(DMUON_E_NULL, "logprobs and targets must be set together");
    if (p->top && (!top_ids || !top_logprobs)) return fail(DMUON_E_NULL, "top_ids and top_logprobs must be set");
    std::vector<Range> rs;
    rows_ranges(*p, true, rs);
    add_range(rs, logprobs, p->tokens * 4, false);
    add_range(rs, entropy, p->tokens * 4, false);
    add_range(rs, lse, p->tokens * 4, false);
    add_range(rs, top_ids, p->tokens * p->top * 8, false);
    add_range(rs, top_logprobs, p->tokens * p->top * 4, false);
    if ((e = check_alias(rs))) return e;
    const size_t need = rows_plan(*p, nullptr).bytes;
    if (need && (e = check_ws(workspace, workspace_bytes, need, rs))) return e;
    const RowsPlan pl = rows_plan(*p, (char*)workspace);
    const CallEnv env = call_env();
    if ((e = forced(env, -2))) return e;
    LogprobsArgs a{};
    a.logits = p->logits;
    a.ld = p->ld;
    a.rows = p->tokens;
    a.vocab = (int32_t)p->vocab;
    a.top = p->top;
    a.piece = (int32_t)pl.piece;
    a.pieces = (int32_t)pl.pieces;
    a.wave_rows = pl.wave;
    a.once = p->tokens * p->vocab * (int64_t)type_bytes(p->dtype) > kCaches && (p->top == 0 || (p->dtype == DMUON_BF16 && p->vocab > 1024 * p->top));
    a.scale = p->scale;
    a.targets = p->targets;
    a.idx64 = p->index_dtype == DMUON_I64;
    a.ignore = p->ignore_index;
    a.logprobs = logprobs;
    a.entropy = entropy;
    a.lse = lse;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.stats = pl.stats;
    a.cand = pl.cand;
    const int f32 = p->dtype == DMUON_F32;
    if ((e = go(env, PH_LOGPROBS, stream, [&] { return launch_logprobs(a, f32, stream); }))) return e;
    if (a.pieces == 1) return DMUON_OK;
    return go(env, PH_LOGPROBS, stream, [&] { return launch_logprobs_join(a, f32, stream); });
  });
}

int dmuon_logprobs_backward(const dmuon_logprobs_problem* p, const float* lse, const float* entropy, const float* grad_logprobs,
                            const float* grad_entropy, void* grad_logits, int64_t ld_grad, void* stream) {
  return guarded([&]() -> int {
    int e = check_rows(p, true);
    if (e) return e;
    if (ld_grad < p->vocab || ld_grad > kMaxStride) return fail(DMUON_E_SHAPE, "ld_grad must be at least vocab");
    const int64_t es = type_bytes(p->dtype);
    if (!spans(p->tokens, p->vocab, ld_grad, es)) return fail(DMUON_E_SHAPE, "grad_logits must end within 2^48 bytes");
    if (p->tokens == 0) return DMUON_OK;
    if (!lse || !grad_logits) return fail(DMUON_E_NULL, "lse and grad_logits must be set");
    if (!grad_logprobs && !grad_entropy) return fail(DMUON_E_NULL, "grad_logprobs or grad_entropy must be set");
    if (grad_logprobs && !p->targets) return fail(DMUON_E_NULL, "grad_logprobs needs targets");
    if (grad_entropy && !entropy) return fail(DMUON_E_NULL, "grad_entropy needs entropy");
    const bool in_place = grad_logits == p->logits && ld_grad == p->ld;
    std::vector<Range> rs;
    rows_ranges(*p, !in_place, rs);
    add_range(rs, lse, p->tokens * 4, true);
    if (grad_entropy) add_range(rs, entropy, p->tokens * 4, true);
    add_range(rs, grad_logprobs, p->tokens * 4, true);
    add_range(rs, grad_entropy, p->tokens * 4, true);
    add_range(rs, grad_logits, strided_bytes(p->tokens, p->vocab, ld_grad, es), false);
    if ((e = check_alias(rs))) return e;
    const CallEnv env = call_env();
    if ((e = forced(env, -2))) return e;
    LogprobsGradArgs a{};
    a.logits = p->logits;
    a.ld = p->ld;
    a.rows = p->tokens;
    a.vocab = (int32_t)p->vocab;
    a.pieces = p->vocab <= kGradWave ? 1 : (int32_t)cdiv(p->vocab, kThreads * kGradUnits * 8);
    const int64_t bytes = (int64_t)type_bytes(p->dtype);
    a.units = (int32_t)round_up(cdiv(cdiv(p->vocab * bytes, 16), a.pieces), 8);
    a.aligned = p->vocab * bytes >= 16 && (uintptr_t)p->logits % 16 == 0 && p->ld * bytes % 16 == 0;
    a.scale = p->scale;
    a.targets = p->targets;
    a.idx64 = p->index_dtype == DMUON_I64;
    a.ignore = p->ignore_index;
    a.lse = lse;
    a.entropy = entropy;
    a.grad_logprobs = grad_logprobs;
    a.grad_entropy = grad_entropy;
    a.out = grad_logits;
    a.ldo = ld_grad;
    return go(env, PH_LOGPROBS_GRAD, stream, [&] { return launch_logprobs_grad(a, p->dtype == DMUON_F32, stream); });
  });
}

}  // extern "C"
