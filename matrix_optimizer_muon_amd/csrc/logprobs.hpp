// Arguments of the log-probability kernels (logprobs.hip), shared with their entry
// points (logprobs.cpp).  Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include "internal.hpp"

namespace dmuon {

constexpr int kTopMost = 128;            // alternatives per row
constexpr int kGroupUnits = 8;           // units of 8 elements that a thread takes together
constexpr int kGroups = 8;               // such groups per thread at most
constexpr int kPieceMost = kThreads * kGroupUnits * 8 * kGroups;     // 131072 columns per workgroup
constexpr int kPieceLeast = kThreads * 8;                            // 2048
constexpr int kRowsEnough = 1024;        // rows from which on none is cut into pieces to fill the card
constexpr int kPiecesMost = 64;          // pieces of one row (a wave joins them)
// Rows that take one wave each: without alternatives up to 12288 words (fp32 4096, or 8192
// where the rows are so few that workgroups would share them), with them up to 4096, or
// 12288 where there are rows enough.  fp32, by a wave and by workgroups: 50 × 5000 5.4 and
// 6.8 µs, 300 × 8192 7.6 and 9.5, 1000 × 8192 9.0 and 14.2; from 1024 rows on 1024 × 4200 7.5
// and 7.1, 2048 × 8192 14.4 and 14.2, 4096 × 6500 25.2 and 24.1.
inline int64_t wave_row(bool f32, int64_t rows) { return !f32 ? 12288 : rows < kRowsEnough ? 8192 : 4096; }
constexpr int kWaveTop = 64 * 8 * 8;                 // 4096: the units' maxima of a row in 8 registers
constexpr int kWaveTopMost = 3 * kWaveTop;           // 12288: in 24
// With 20 alternatives by a wave and by workgroups, bf16 (fp32): 256 × 12288 15.2 and 13.9 µs
// (17.3 and 16.8), 512 × 12288 16.6 and 17.1 (18.0 and 19.1), 800 × 8192 13.7 and 19.4 (15.7 and
// 21.8), 4096 × 8192 25.2 and 28.5 (34.9 and 36.7).  From 1024 rows on a workgroup has a row to
// itself, and is ahead while all rows are in flight: 1024 × 8192 14.8 and 12.0 (16.4 and 14.9).
constexpr int kWaveTopRows = 512;
constexpr int kGradUnits = 4;            // times 8 elements per thread of the gradient
constexpr int kGradWave = 64 * kGradUnits * 8;       // 2048: rows up to this take one wave each

// Σ 2^t and Σ t·2^t of a row's piece, m its largest logit and t its exponents (see logprobs.hip)
struct RowStat {
  float m, s, u;
};

struct LogprobsArgs {
  const void* logits;          // rows × vocab, row stride ld
  int64_t ld;
  int64_t rows;
  int32_t vocab;
  int32_t top;                 // alternatives, 0: none
  int32_t piece, pieces;       // columns per workgroup, workgroups per row
  int32_t wave_rows;           // 1: a wave per row
  int32_t once;                // 1: read nontemporally
  float scale;
  const void* targets;         // or null: every row takes part, none has a target
  int32_t idx64;
  int64_t ignore;
  float* logprobs;             // null without targets
  float* entropy;
  float* lse;
  int64_t* top_ids;            // [rows][top]
  float* top_logprobs;
  // where pieces > 1
  RowStat* stats;              // [rows][pieces]
  uint64_t* cand;              // [rows][pieces][top], best first, 0 where there are fewer
};

struct LogprobsGradArgs {
  const void* logits;
  int64_t ld;
  int64_t rows;
  int32_t vocab;
  int32_t pieces;              // workgroups (or waves) per row
  int32_t units;               // units of 16 bytes of each
  int32_t aligned;             // the logits' rows start on 16 bytes and hold a unit
  float scale;
  const void* targets;         // or null
  int32_t idx64;
  int64_t ignore;
  const float* lse;
  const float* entropy;        // with grad_entropy
  const float* grad_logprobs;  // or null
  const float* grad_entropy;   // or null
  void* out;                   // rows × vocab, row stride ldo
  int64_t ldo;
};

int launch_logprobs(const LogprobsArgs& a, int f32, void* stream);
int launch_logprobs_join(const LogprobsArgs& a, int f32, void* stream);
int launch_logprobs_grad(const LogprobsGradArgs& a, int f32, void* stream);

}  // namespace dmuon
