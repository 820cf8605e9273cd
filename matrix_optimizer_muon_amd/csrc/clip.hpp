// Arguments of the gradient-norm and clipping kernels (clip.hip), shared with their entry
// points (clip.cpp).  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.hpp"

namespace dmuon {

constexpr int kClipChunk = kThreads * 32;    // elements per chunk: 32 per thread, in units of 16 bytes
constexpr int kClipGroups = 2048;            // workgroups at most: 8 for every CU

// One tensor as the kernels see it.
struct ClipProblem {
  int64_t numel;
  const void* grad;
  void* out;                   // null: the norm only
  int32_t f32, out_f32;
  uint32_t tag;                // plan tag (see ClipTable::tag)
  int32_t pad;                 // explicit: the table is hashed
};
static_assert(sizeof(ClipProblem) == 40, "ClipProblem must have no implicit padding");

struct ClipTable {
  const ClipProblem* probs;    // device
  const int32_t* chunk0;       // device, [n + 1]: first chunk of each tensor, then their number
  double* part;                // device, [groups]: sums of squares
  int32_t n, groups, chunks;
  uint32_t tag;                // hash of the host-built table: a workgroup whose entries
                               // carry another tag (the workspace does not hold this plan's
                               // table) exits at once
};

struct ClipScalars {
  float max_norm, eps;
  int32_t measured;            // 1: the norm of `part`, written to norm; 0: norm is read
  float* norm;
};

int launch_grad_norm(const ClipTable& tab, void* stream);
int launch_grad_norm_join(const ClipTable& tab, float* norm, void* stream);
int launch_grad_clip(const ClipTable& tab, const ClipScalars& s, void* stream);

}  // namespace dmuon
