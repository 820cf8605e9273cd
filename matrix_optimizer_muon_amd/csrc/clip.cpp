// C entry points of the global norm over many gradients and of clipping by it: validation,
// the table of tensors in the caller's workspace, launches.
#include <cmath>
#include <cstring>
#include <vector>

#include "clip.hpp"
#include "entry.hpp"

namespace dmuon {
namespace {

constexpr int64_t kMaxElements = (int64_t)1 << 41;       // of all tensors: chunks and launches stay in 32 bits

struct ClipPlan {
  std::vector<char> table;               // entries, then first chunks
  size_t off_chunks = 0, off_part = 0, bytes = 0;
  int32_t n = 0, groups = 0, chunks = 0;
  uint32_t tag = 0;
  ClipTable at(char* ws) const {
    return {(const ClipProblem*)ws, (const int32_t*)(ws + off_chunks), (double*)(ws + off_part), n, groups, chunks, tag};
  }
};

// FNV-1a over 8-byte words, folded
uint32_t hash_words(const std::vector<char>& t) {
  uint64_t h = 14695981039346656037ull;
  for (size_t i = 0; i + 8 <= t.size(); i += 8) {
    uint64_t w;
    std::memcpy(&w, t.data() + i, 8);
    h = (h ^ w) * 1099511628211ull;
    h ^= h >> 29;
  }
  return (uint32_t)(h ^ h >> 32);
}

// The tensors that are not empty; `clip`: each must have somewhere to write.
int make_plan(const dmuon_grad_tensor* t, int32_t n, bool clip, ClipPlan& pl) {
  if (n < 0) return fail(DMUON_E_SHAPE, "n_tensors < 0");
  if (n > 0 && !t) return fail(DMUON_E_NULL, "tensors is NULL");
  int64_t elements = 0, chunks = 0;
  int32_t used = 0;
  for (int32_t i = 0; i < n; ++i) {
    const dmuon_grad_tensor& x = t[i];
    const auto bad = [&](int code, const char* what) { return fail(code, "tensor " + std::to_string(i) + ": " + what); };
    if (x.numel < 0 || x.numel > kMaxElements) return bad(DMUON_E_SHAPE, "numel must be in [0, 2^41]");
    if (!float_type(x.dtype) || (x.out && !float_type(x.out_dtype))) return bad(DMUON_E_DTYPE, "types must be DMUON_F32 or DMUON_BF16");
    if (x.numel == 0) continue;
    if (!x.grad) return bad(DMUON_E_NULL, "grad must be set");
    if (clip && !x.out) return bad(DMUON_E_NULL, "out must be set");
    if (x.out == x.grad && x.out_dtype != x.dtype) return bad(DMUON_E_DTYPE, "in place the types must agree");
    elements += x.numel;
    if (elements > kMaxElements) return fail(DMUON_E_SHAPE, "more than 2^41 elements");
    chunks += cdiv(x.numel, kClipChunk);
    ++used;
  }
  if (chunks > (int64_t)1 << 30) return fail(DMUON_E_SHAPE, "too many tensors and elements");
  pl.n = used;
  pl.chunks = (int32_t)chunks;
  pl.groups = (int32_t)std::min<int64_t>(chunks, kClipGroups);
  if (!used) return DMUON_OK;
  pl.off_chunks = align256((size_t)used * sizeof(ClipProblem));
  const size_t table = align256(pl.off_chunks + ((size_t)used + 1) * sizeof(int32_t));
  pl.off_part = table;
  pl.bytes = align256(pl.off_part + (size_t)pl.groups * sizeof(double));
  pl.table.assign(table, 0);
  ClipProblem* probs = (ClipProblem*)pl.table.data();
  int32_t* chunk0 = (int32_t*)(pl.table.data() + pl.off_chunks);
  int32_t at = 0, k = 0;
  for (int32_t i = 0; i < n; ++i) {
    const dmuon_grad_tensor& x = t[i];
    if (x.numel == 0) continue;
    probs[k] = {x.numel, x.grad, x.out, x.dtype == DMUON_F32, x.out ? x.out_dtype == DMUON_F32 : 0, 0, 0};
    chunk0[k++] = at;
    at += (int32_t)cdiv(x.numel, kClipChunk);
  }
  chunk0[k] = at;
  pl.tag = hash_words(pl.table);
  for (k = 0; k < used; ++k) probs[k].tag = pl.tag;
  return DMUON_OK;
}

std::vector<Range> ranges(const dmuon_grad_tensor* t, int32_t n, const float* norm, bool norm_read) {
  std::vector<Range> rs;
  for (int32_t i = 0; i < n; ++i) {
    if (t[i].out != t[i].grad) add_range(rs, t[i].grad, t[i].numel * type_bytes(t[i].dtype), true);
    add_range(rs, t[i].out, t[i].out ? t[i].numel * type_bytes(t[i].out_dtype) : 0, false);
  }
  add_range(rs, norm, 4, norm_read);
  return rs;
}

// `norm` meets none of the tensors (their own overlaps are checked by prepare)
int check_norm(const float* norm, bool read, const std::vector<Range>& rs) {
  const uintptr_t lo = (uintptr_t)norm;
  for (size_t i = 0; i + 1 < rs.size(); ++i)                   // the last one is norm itself
    if ((!read || !rs[i].ro) && rs[i].lo < lo + 4 && lo < rs[i].hi) return fail(DMUON_E_ALIAS, "norm overlaps a tensor");
  return DMUON_OK;
}

int prepare(const dmuon_grad_tensor* t, int32_t n, void* ws, size_t ws_bytes, void* stream) {
  ClipPlan pl;
  int e = make_plan(t, n, false, pl);
  if (e) return e;
  if (!pl.n) return DMUON_OK;
  std::vector<Range> rs = ranges(t, n, nullptr, false);
  if ((e = check_alias(rs))) return e;
  if ((e = check_ws(ws, ws_bytes, pl.bytes, rs))) return e;
  const CallEnv env = call_env();
  if ((e = forced(env, -2))) return e;
  return write_table(ws, pl.table, stream, env);
}

int run(const dmuon_grad_tensor* t, int32_t n, bool clip, float max_norm, float eps, bool measure, float* norm, void* ws,
        size_t ws_bytes, void* stream) {
  if (clip && (!(max_norm >= 0.f) || !std::isfinite(max_norm))) return fail(DMUON_E_CFG, "max_norm must be finite and >= 0");
  if (clip && (!(eps >= 0.f) || !std::isfinite(eps))) return fail(DMUON_E_CFG, "eps must be finite and >= 0");
  ClipPlan pl;
  int e = make_plan(t, n, clip, pl);
  if (e) return e;
  if (!norm) return fail(DMUON_E_NULL, "norm must be set");
  if (!pl.n && !measure) return DMUON_OK;
  const std::vector<Range> rs = ranges(t, n, norm, clip && !measure);
  if ((e = check_norm(norm, clip && !measure, rs))) return e;
  if (pl.n && (e = check_ws(ws, ws_bytes, pl.bytes, rs))) return e;
  const CallEnv env = call_env();
  if ((e = forced(env, -2))) return e;
  const ClipTable tab = pl.at((char*)ws);
  if (measure && pl.n && (e = go(env, PH_GRAD_NORM, stream, [&] { return launch_grad_norm(tab, stream); }))) return e;
  if (!clip || !pl.n) return go(env, PH_GRAD_NORM, stream, [&] { return launch_grad_norm_join(tab, norm, stream); });
  const ClipScalars s = {max_norm, eps, measure, norm};
  return go(env, PH_GRAD_CLIP, stream, [&] { return launch_grad_clip(tab, s, stream); });
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_grad_workspace_size(const dmuon_grad_tensor* tensors, int32_t n_tensors, size_t* bytes) {
  return guarded([&]() -> int {
    if (!bytes) return fail(DMUON_E_NULL, "bytes is NULL");
    ClipPlan pl;
    int e = make_plan(tensors, n_tensors, false, pl);
    if (e) return e;
    *bytes = pl.bytes;
    return DMUON_OK;
  });
}

int dmuon_grad_prepare(const dmuon_grad_tensor* tensors, int32_t n_tensors, void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int { return prepare(tensors, n_tensors, workspace, workspace_bytes, stream); });
}

int dmuon_grad_norm_run(const dmuon_grad_tensor* tensors, int32_t n_tensors, float* norm, void* workspace, size_t workspace_bytes,
                        void* stream) {
  return guarded([&]() -> int { return run(tensors, n_tensors, false, 0.f, 0.f, true, norm, workspace, workspace_bytes, stream); });
}

int dmuon_grad_clip_run(const dmuon_grad_tensor* tensors, int32_t n_tensors, float max_norm, float eps, int32_t measure, float* norm,
                        void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    if (measure != 0 && measure != 1) return fail(DMUON_E_CFG, "measure must be 0 or 1");
    return run(tensors, n_tensors, true, max_norm, eps, measure != 0, norm, workspace, workspace_bytes, stream);
  });
}

}  // extern "C"
