// Host code shared by the C entry points of the training operators (grads.cpp,
// logprobs.cpp, clip.cpp): limits, argument checks, workspace layout, launches.
#pragma once

#include <algorithm>
#include <string>
#include <vector>

#include "../../include/dmuon_ns.h"
#include "host.hpp"
#include "internal.hpp"

namespace dmuon {

constexpr int64_t kMaxTokens = (int64_t)1 << 24;    // rows of one cross-entropy or wgrad call
constexpr int64_t kMaxIds = (int64_t)1 << 30;       // ids of one embedding call
constexpr int64_t kMaxWidth = 65536;
constexpr int64_t kMaxRows = (int64_t)1 << 30;      // vocabulary, table rows
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxExtent = (int64_t)1 << 48;    // bytes of a strided matrix: the largest dense one (2^30 × 65536 fp32)

// A launch takes fewer than 2^32 threads.
inline bool launchable(int64_t workgroups, int64_t threads) { return workgroups < ((int64_t)1 << 32) / threads; }

// C entry bodies: nothing thrown on the host leaves them.  Where an allocation failed the
// message must not need one: it fits a string's own 15 bytes.
template <typename F>
inline int guarded(F&& f) {
  clear_error();
  try {
    return f();
  } catch (...) {
    return fail(DMUON_E_HIP, "out of memory");
  }
}

inline int hip_fail(int e) { return fail(DMUON_E_HIP, std::string("launch failed: ") + hip_error_string(e)); }

// one launch under the debugging switches
template <typename F>
inline int go(const CallEnv& env, int phase, void* stream, F&& launch) {
  int e = forced(env, phase);
  if (e) return e;
  const int r = launch();
  if (r) return hip_fail(r);
  return settle(env, stream, phase_name(phase));
}

inline bool float_type(int32_t t) { return t == DMUON_F32 || t == DMUON_BF16; }
inline int64_t type_bytes(int32_t t) { return t == DMUON_F32 ? 4 : 2; }
inline bool index_type(int32_t t) { return t == DMUON_I32 || t == DMUON_I64; }

// scale of the logits that log probabilities are taken of
inline bool logit_scale(float s) { return s >= 0x1p-20f && s <= 0x1p20f; }

inline void add_range(std::vector<Range>& rs, const void* p, int64_t bytes, bool ro) {
  if (p && bytes > 0) rs.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, ro});
}
// rows × cols elements of es bytes at a stride of ld (≥ cols, checked before) end within kMaxExtent
inline bool spans(int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  return rows <= 1 || ld <= (kMaxExtent / es - cols) / (rows - 1);
}
inline int64_t strided_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  return rows > 0 ? ((rows - 1) * ld + cols) * es : 0;
}

// the workspace's size, and that it meets none of the call's buffers
inline int check_ws(void* ws, size_t have, size_t need, const std::vector<Range>& rs) {
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

}  // namespace dmuon
