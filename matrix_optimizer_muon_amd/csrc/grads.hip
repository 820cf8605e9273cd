// HIP kernels of the training gradients for gfx950 (MI355X): softmax cross entropy
// over a large vocabulary, embedding lookup and its gradient, activation
// checkpoints in 8 bits and the weight gradient computed from them.
//
// The matrix products run on two contraction cores of this file, built from the step's
// parts (core.hpp): 256 × 256 tiles where there is work to fill every CU, 128 × 128
// tiles elsewhere.  fp32 operands enter them as three bf16 planes whose sum is the fp32
// value.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <mutex>

#include "core.hpp"
#include "grads.hpp"

namespace dmuon {

// ---------------------------------------------------------------------------
// small helpers
// ---------------------------------------------------------------------------
// 8 consecutive elements as fp32: 16-byte loads where `vec`, else element by
// element with zeros from column `left` on
__device__ __forceinline__ void unpack8(const u32x4_t& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = __uint_as_float(w[k] << 16);
    v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(gptr<const uint16_t> p, bool vec, int left, float (&v)[8]) {
  if (vec) {
    const u32x4_t u = *(gptr<const u32x4_t>)p;
    unpack8(u, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? bf16_to_f32(p[e]) : 0.f;
  }
}
__device__ __forceinline__ void load8(gptr<const float> p, bool vec, int left, float (&v)[8]) {
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_t a = ((gptr<const f32x4_t>)p)[h];
      v[4 * h] = a.x; v[4 * h + 1] = a.y; v[4 * h + 2] = a.z; v[4 * h + 3] = a.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < left ? p[e] : 0.f;
  }
}
__device__ __forceinline__ u32x4_t pack8(const float (&v)[8]) {
  return u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}
// NT: nontemporal, for results that this library does not read again (the lookup of
// 32768 tokens 85.6 → 83.6 µs, a checkpoint stored and read back 92 → 86)
template <bool NT = false>
__device__ __forceinline__ void store8(gptr<uint16_t> p, bool vec, int left, const float (&v)[8]) {
  if (vec) {
    if (NT) __builtin_nontemporal_store(pack8(v), (gptr<u32x4_t>)p);
    else *(gptr<u32x4_t>)p = pack8(v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = f32_to_bf16(v[e]);
  }
}
template <bool NT = false>
__device__ __forceinline__ void store8(gptr<float> p, bool vec, int left, const float (&v)[8]) {
  if (vec) {
    const f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    if (NT) {
      __builtin_nontemporal_store(a, (gptr<f32x4_t>)p);
      __builtin_nontemporal_store(b, (gptr<f32x4_t>)p + 1);
    } else {
      ((gptr<f32x4_t>)p)[0] = a;
      ((gptr<f32x4_t>)p)[1] = b;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) p[e] = v[e];
  }
}

// An int32 or int64 index, as its dwords and without a branch, so that several
// loads of a thread are in flight together.
__device__ __forceinline__ int64_t load_index(const void* p, int idx64, int64_t i) {
  const gptr<const int32_t> q = glob((const int32_t*)p) + (i << idx64);
  const int32_t lo = q[0], hi = q[idx64];
  return (int64_t)(((uint64_t)(uint32_t)(idx64 ? hi : lo >> 31) << 32) | (uint32_t)lo);
}

// x = hi + mid + lo, each a bf16 value: hi is x rounded to bf16 (cut off where
// rounding would overflow), mid the rest rounded, lo the rest of that: 24 bits.
// An infinity or NaN sits in lo alone: lo meets only the other side's hi (plane_pairs),
// which is 0 for a 0 only, so that an infinity times another finite number stays one
// (in hi it would meet the mid and lo of that number, which may be 0: NaN).  Two
// infinities meet each other's hi = 0 and give NaN.
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
  const bool special = (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u;
  float hi = bf16_to_f32(f32_to_bf16(x));
  if ((__float_as_uint(hi) & 0x7f800000u) == 0x7f800000u && !special) hi = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  const float r = x - hi;
  const float mid = bf16_to_f32(f32_to_bf16(r));
  p[0] = special ? 0.f : hi;
  p[1] = special ? 0.f : mid;
  p[2] = special ? x : bf16_to_f32(f32_to_bf16(r - mid));
}

// ---------------------------------------------------------------------------
// operand copies: rows of a matrix (gathered by an index list or in order) as
// zero-padded bf16 planes, row-major, in fragment order, or both from one read.
// Bound by memory.  A wave takes 8 rows × 64 columns: whole lines on the way in and
// in the row-major copy, and runs of 128 bytes in the fragment order (a chunk's 8
// rows lie together).  8192×4096 bf16, both copies: 32 µs; threads along a row and a
// launch per copy took 20 + 62, most of it for 16-byte pieces of lines.
// ---------------------------------------------------------------------------
// columns c … c + 7 of destination row r, from source row sr
__device__ __forceinline__ void pack_piece(const PackArgs& a, int64_t r, int64_t sr, int c, bool vec) {
  const int left = a.cols - c;
  const int64_t at = r * a.ldd + c;
  const int64_t blk = ((r >> 4) * (a.ldd >> 5) + (c >> 5)) * 512 + (((c >> 3) & 3) * 16 + (r & 15)) * 8;
  float v[8];
  if (a.f32) {
    load8(glob((const float*)a.src) + sr * a.ld + c, vec && left >= 8, left, v);
    float p[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s[3];
      split3(v[e], s);
      p[0][e] = s[0]; p[1][e] = s[1]; p[2][e] = s[2];
    }
#pragma unroll
    for (int q = 0; q < kPlanes; ++q) {
      const u32x4_t w = pack8(p[q]);
      if (a.dst) *(gptr<u32x4_t>)(glob(a.dst) + q * a.plane + at) = w;
      if (a.blocks) *(gptr<u32x4_t>)(glob(a.blocks) + q * a.blocks_plane + blk) = w;
    }
  } else {
    load8(glob((const uint16_t*)a.src) + sr * a.ld + c, vec && left >= 8, left, v);
    const u32x4_t w = pack8(v);                     // bf16 → fp32 → bf16 is exact
    if (a.dst) *(gptr<u32x4_t>)(glob(a.dst) + at) = w;
    if (a.blocks) *(gptr<u32x4_t>)(glob(a.blocks) + blk) = w;
  }
}
__global__ __launch_bounds__(kThreads) void k_pack(PackArgs a) {
  const int64_t rows = a.count ? (int64_t)*a.count : a.rows;
  const int lane = threadIdx.x & 63;
  const uint32_t per = (uint32_t)a.ldd >> 6;         // units of 64 columns per row
  const uint32_t n = (uint32_t)((rows + 7) >> 3) * per;     // ≤ 2^21 × 2^10
  const bool vec = (a.ld & 7) == 0 && ((uintptr_t)a.src & 15) == 0;
  const uint32_t step = gridDim.x * (kThreads / 64);
  for (uint64_t u = (uint64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); u < n; u += step) {
    const uint32_t g = (uint32_t)u / per;
    const int64_t r = (int64_t)g * 8 + (lane >> 3);
    if (r < rows) pack_piece(a, r, a.gather ? (int64_t)a.gather[r] : r, (int)((uint32_t)u - g * per) * 64 + (lane & 7) * 8, vec);
  }
}

// ---------------------------------------------------------------------------
// cross entropy: the compact list of tokens that take part, in order.  One
// workgroup walks the tokens 8192 at a time, the loads of a step issued together:
// places come from ballots and one scan over (row of 1024 tokens, wave).
// Forward: tokens whose target is not ignore_index (the others get loss and lse
// 0).  Backward: those whose target also lies in the vocabulary, or in another shard of
// it (kElsewhere: a row of probabilities without a target), and whose weight is not zero.  The largest finite |weight| (1 if there is none) goes out too: dZ uses
// weights relative to it and the products' epilogues multiply it back, so that a
// uniform weight leaves p − δ unscaled when it is rounded to bf16 and tiny weights do
// not underflow.
// Latency bound: forward 5.6 µs for 4096 tokens, backward 8.7 for 8192 (a walk over one
// range per thread: 39).
// ---------------------------------------------------------------------------
constexpr int kScanThreads = 1024;
constexpr int kScanRows = 8;
__device__ __forceinline__ bool in_vocab(int64_t y, int32_t vocab) { return y >= 0 && y < vocab; }
// what the list keeps of a target: a vocabulary row, kTgtElsewhere or kTgtNone
__device__ __forceinline__ int32_t list_target(int64_t y, int32_t vocab) {
  return in_vocab(y, vocab) ? (int32_t)y : y == kElsewhere ? kTgtElsewhere : kTgtNone;
}
__global__ __launch_bounds__(kScanThreads) void k_ce_scan(CeScanArgs a) {
  constexpr int waves = kScanThreads / 64, parts = kScanRows * waves;      // 128 partial counts
  __shared__ int place[parts];
  __shared__ int total;
  __shared__ float wave_max[waves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float gm = 0.f;
  int base = 0;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kScanRows * kScanThreads) {
    int64_t y[kScanRows];
    float g[kScanRows], l[kScanRows];
#pragma unroll
    for (int k = 0; k < kScanRows; ++k) {
      const int64_t t = t0 + k * kScanThreads + tid;
      const int64_t u = t < a.tokens ? t : a.tokens - 1;
      y[k] = load_index(a.targets, a.idx64, u);
      g[k] = l[k] = 0.f;
      if (a.backward) {
        g[k] = glob(a.grad_losses)[u];
        l[k] = glob(a.lse_in)[u];
      }
      if (t >= a.tokens) y[k] = a.ignore;
    }
    uint64_t in[kScanRows];
#pragma unroll
    for (int k = 0; k < kScanRows; ++k) {
      const bool part = y[k] != a.ignore && (!a.backward || ((in_vocab(y[k], a.vocab) || y[k] == kElsewhere) && !(g[k] == 0.f)));
      in[k] = __ballot(part);
      if (part && fabsf(g[k]) < INFINITY) gm = fmaxf(gm, fabsf(g[k]));
      if (lane == 0) place[k * waves + wave] = __popcll(in[k]);
    }
    __syncthreads();
    if (wave == 0) {                        // exclusive scan of the 128 counts, two per lane
      const int c0 = place[2 * lane], c1 = place[2 * lane + 1];
      int incl = c0 + c1;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(incl, o, 64);
        if (lane >= o) incl += up;
      }
      place[2 * lane] = base + incl - c0 - c1;
      place[2 * lane + 1] = base + incl - c1;
      if (lane == 63) total = base + incl;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kScanRows; ++k) {
      const int64_t t = t0 + k * kScanThreads + tid;
      if (t >= a.tokens) continue;
      const bool part = (in[k] >> lane) & 1;
      const int i = place[k * waves + wave] + __popcll(in[k] & ((1ull << lane) - 1));
      if (a.backward) a.pos[t] = part ? i : -1;
      if (part) {
        a.rows[i] = (int32_t)t;
        a.tgt[i] = list_target(y[k], a.vocab);
        if (a.backward) {
          a.clse[i] = l[k];
          a.cg[i] = g[k];
        }
      } else if (!a.backward) {
        a.losses[t] = 0.f;
        a.lse[t] = 0.f;
      }
    }
    base = total;
    __syncthreads();
  }
  if (tid == 0) *a.count = base;
  if (!a.backward) return;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor(gm, o, 64));
  if (lane == 0) wave_max[wave] = gm;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < waves; ++w) gm = fmaxf(gm, wave_max[w]);
    *a.gmax = gm > 0.f ? gm : 1.f;
  }
}

// ---------------------------------------------------------------------------
// the two cores of the products
// ---------------------------------------------------------------------------
// Swizzle of the 64-byte rows of a row-major stage: 16-byte chunk c of row r sits at
// chunk c ^ row_swz(r).  A 16-byte LDS read is served 16 lanes at a time, lanes 0–3,
// 12–15 and 20–27 together (then 4–11, 16–19 and 28–31, and the same 32 lanes on): in
// the fragments read here (lane l: row l & 15, chunk l >> 4) those are row quads 0 and 3
// of one chunk and quads 1 and 2 of the next, which this order puts into four different
// chunks, so all 64 banks serve a step.  (Quad order 0 1 2 3 counts a conflict per read.)
__device__ __forceinline__ int row_swz(int r) { return (-(r >> 2)) & 3; }

// Small core: 128 × 128 per workgroup of 4 waves, 64 × 64 per wave, for products
// whose tiles are few or whose K is short.  K is staged through LDS like the step's
// core does (64-byte rows for row-major operands, 32 k-rows of 256 bytes for K-major
// ones, the same swizzles), three stages of 16 KiB, so that three workgroups share a
// CU: their waves are not in step, one's copies, prologue and epilogue run beside the
// others' products.  One barrier per stage: a wave waits for its own share of stage
// kt before it, so behind it the whole stage has landed and every wave is done with
// stage kt − 1, whose slot stage kt + 2 takes.
constexpr int kSmallStage = 2 * 128 * kRowBytes;        // 16 KiB
constexpr int kSmallStages = 3;

template <bool TA, bool TB>
__device__ __forceinline__ void gemm_small(const Operands& op, char* smem, f32x16_t (&acc)[2][2]) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave >> 1, wc = wave & 1;
  const __amdgpu_buffer_rsrc_t ra = range_rsrc(op.a, (int64_t)(op.rows_a < 128 ? op.rows_a : 128) * op.lda_b);
  const __amdgpu_buffer_rsrc_t rb = range_rsrc(op.b, (int64_t)(op.rows_b < 128 ? op.rows_b : 128) * op.ldb_b);
  // copies: wave w fills rows [32w, 32w + 32) of each operand, 16 rows (row-major) or
  // 4 k-rows (K-major) per instruction; lane l lands at byte 16·l of its 1 KiB
  int offa[2], offb[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = (wave * 2 + q) * 16 + (lane >> 2);
    const int c = (lane & 3) ^ row_swz(row);
    const int kr = 4 * (wave * 2 + q) + (lane >> 4), un = lane & 15;
    const int lun = (((un >> 1) ^ kmaj_swz(kr)) << 1) | (un & 1);
    offa[q] = TA ? kr * op.lda_b + op.cola_b + lun * 16 : row * op.lda_b + c * 16;
    offb[q] = TB ? kr * op.ldb_b + op.colb_b + lun * 16 : row * op.ldb_b + c * 16;
  }
  // fragments: 4 of 16 rows and 4 of 16 columns, all 32 k of a stage
  int fa_off[4], fb_off[4], ta_off[4][2], tb_off[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ar = wr * 64 + 16 * i + (lane & 15), br = wc * 64 + 16 * i + (lane & 15), c = lane >> 4;
    fa_off[i] = ar * kRowBytes + ((c ^ row_swz(ar)) * 16);
    fb_off[i] = 128 * kRowBytes + br * kRowBytes + ((c ^ row_swz(br)) * 16);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int kr = 8 * (lane >> 4) + 4 * t + ((lane & 15) >> 2), sub = 4 * (lane & 3);
      const int na = wr * 64 + 16 * i + sub, nb = wc * 64 + 16 * i + sub;
      ta_off[i][t] = kr * 256 + (((na >> 4) ^ kmaj_swz(kr)) << 5) + ((2 * na) & 31);
      tb_off[i][t] = 128 * kRowBytes + kr * 256 + (((nb >> 4) ^ kmaj_swz(kr)) << 5) + ((2 * nb) & 31);
    }
  }
  auto kmaj_rsrc = [&](const char* p, int ld_b, int rows, int kt) {
    const int left = rows - 32 * kt;
    return range_rsrc(p + (int64_t)kt * 32 * ld_b, (int64_t)(left < 0 ? 0 : (left < 32 ? left : 32)) * ld_b);
  };
  auto issue = [&](int kt, int slot) {
    char* base = smem + slot * kSmallStage;
    const __amdgpu_buffer_rsrc_t sa = TA ? kmaj_rsrc(op.a, op.lda_b, op.rows_a, kt) : ra;
    const __amdgpu_buffer_rsrc_t sb = TB ? kmaj_rsrc(op.b, op.ldb_b, op.rows_b, kt) : rb;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      char* da = base + (wave * 2 + q) * 1024;
      char* db = da + 128 * kRowBytes;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sa, (__attribute__((address_space(3))) void*)da, 16,
                                               offa[q] + (TA ? 0 : kt * kRowBytes), 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sb, (__attribute__((address_space(3))) void*)db, 16,
                                               offb[q] + (TB ? 0 : kt * kRowBytes), 0, 0, 0);
    }
  };
  const int KT = op.ktiles;
  if (KT > 0) issue(0, 0);
  if (KT > 1) issue(1, 1);
  int slot = 0;
#pragma unroll 1
  for (int kt = 0; kt < KT; ++kt) {
    if (kt + 1 < KT) DMUON_WAIT_VM(4);                   // own share of stage kt (4 copies per stage)
    else DMUON_WAIT_VM(0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (kt + 2 < KT) issue(kt + 2, slot == 0 ? 2 : slot - 1);
    const char* base = smem + slot * kSmallStage;
    auto tr16 = [&](int off0, int off1) {
      const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)(base + off0));
      const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)(base + off1));
      u32x4_t r;
      r.x = (uint32_t)(uint16_t)lo.x | ((uint32_t)(uint16_t)lo.y << 16);
      r.y = (uint32_t)(uint16_t)lo.z | ((uint32_t)(uint16_t)lo.w << 16);
      r.z = (uint32_t)(uint16_t)hi.x | ((uint32_t)(uint16_t)hi.y << 16);
      r.w = (uint32_t)(uint16_t)hi.z | ((uint32_t)(uint16_t)hi.w << 16);
      return r;
    };
    u32x4_t fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fa[i] = TA ? tr16(ta_off[i][0], ta_off[i][1]) : *(const u32x4_t*)(base + fa_off[i]);
      fb[i] = TB ? tr16(tb_off[i][0], tb_off[i][1]) : *(const u32x4_t*)(base + fb_off[i]);
    }
    static_for<4>([&](auto Sq) {
      constexpr int qs = decltype(Sq)::value;
      static_for<4>([&](auto Tq) {
        constexpr int qt = decltype(Tq)::value;
        mfma_quarter<2 * (qs & 1) + (qt & 1)>(acc[qs >> 1][qt >> 1], fa[qs], fb[qt]);
      });
    });
    __builtin_amdgcn_sched_barrier(0);                   // the fragments are in registers before the next barrier
    slot = slot == 2 ? 0 : slot + 1;
  }
  __syncthreads();                                       // LDS is free for the caller
}

// ---------------------------------------------------------------------------
// Large core: 256 × 256 per workgroup of 8 waves, 128 × 64 per wave, 32-deep stages
// through LDS, one barrier per stage.
//
// A wave multiplies the fragments of stage kt, which it read during stage kt − 1, and
// reads those of stage kt + 1 in between: after the four MFMAs of a row fragment its
// registers take the next stage's (the four column fragments have a second set).  So no
// MFMA waits for LDS, and the barrier only orders the copies: before barrier kt every
// wave has waited for its own share of stage kt + 1; behind it the stage is whole, and
// stage kt − 1's slot is free (its fragments were multiplied before the barrier) for
// the copies issued next.
//
// An operand is staged in one of three forms, each moved in whole 128-byte lines (the
// 64-byte pieces of a 32-deep row-major stage cost 2.6 times as much per byte):
//   kKMajor  k-rows of 512 bytes, four slots of 16 KiB, read with transposing loads;
//   kRows    row-major, two stages at a time as 128-byte rows: three slots of 32 KiB;
//   kBlocks  fragment order, blocks of 16 rows × 32 k ([row block][k block][lane][16
//            bytes], lane l holding row l & 15 and k 8(l >> 4) … + 7): four slots of
//            16 KiB, contiguous at both ends.
// Stages past the last are issued with an empty range (no traffic), so that the counts
// of copies in flight are the same throughout.
// What bounds it is the way from L2 into LDS: at 8192 tokens × 16000 rows × 4096 the
// weight gradient takes 797 µs (the step's core, two barriers per stage and two wave
// groups in turn, 907), without its copies less than 580, without its LDS reads 624, and
// with 4 waves of 128 × 128, which read LDS a third less, 4% more.  The matrix cores are
// busy for 61% of it, at 2.06 GHz.
// ---------------------------------------------------------------------------
enum StageForm : int { kKMajor = 0, kRows = 1, kBlocks = 2 };
typedef __attribute__((address_space(3))) char lds_char;
constexpr int kSlot = kTile * kRowBytes;                // 16 KiB: one operand's stage
constexpr int form_lds(int form) { return form == kRows ? 6 * kSlot : 4 * kSlot; }

struct Side {
  const char* p;                // kKMajor: k-row 0; kRows: first row of the tile; kBlocks: the tile's first block
  int64_t pitch;                // bytes between k-rows, rows, or row blocks
  int64_t extent;               // kKMajor: k-rows; kRows: rows from the tile's first; kBlocks: bytes from p
  int col_b;                    // kKMajor: byte of the tile's first column in a k-row
};

// the copies of one operand and its fragments in LDS; N fragments of 16 rows per wave
template <int FORM, int N>
struct Stager {
  Side s;
  lds_char* lds;                                         // the operand's ring
  int off[FORM == kRows ? 4 : 2];
  int frag[FORM == kKMajor ? N : 2];                     // see read()
  __amdgpu_buffer_rsrc_t whole;                          // kRows
  int wave, lane;

  __device__ __forceinline__ Stager(const Side& side, char* ring, int first) : s(side), lds((lds_char*)ring) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (FORM == kKMajor) {
      const int ld = (int)s.pitch;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int kr = 2 * (wave * 2 + q) + (lane >> 5), un = lane & 31;
        const int lun = (((un >> 1) ^ kmaj_swz(kr)) << 1) | (un & 1);
        off[q] = kr * ld + s.col_b + lun * 16;
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {                      // k-rows kr and kr + 4 share the swizzle
        const int kr = 8 * (lane >> 4) + ((lane & 15) >> 2);
        const int n = first + 16 * i + 4 * (lane & 3);
        frag[i] = kr * 512 + (((n >> 4) ^ kmaj_swz(kr)) << 5) + ((2 * n) & 31);
      }
    } else if constexpr (FORM == kRows) {
      // 8 rows of 128 bytes per instruction; 16-byte chunk c of row r at chunk
      // c ^ ((r >> 1) & 7): the 16 lanes a 16-byte read serves together (see row_swz)
      // then fall on 16 different chunks of the two row parities
      const int ld = (int)s.pitch;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = (wave * 4 + q) * 8 + (lane >> 3);
        off[q] = row * ld + (((lane & 7) ^ ((row >> 1) & 7)) << 4);
      }
      const int rows = (int)(s.extent < kTile ? s.extent : kTile);
      whole = range_rsrc(s.p, (int64_t)rows * s.pitch);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = first + (lane & 15);
        frag[h] = row * 128 + (((4 * h + (lane >> 4)) ^ ((row >> 1) & 7)) << 4);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) off[q] = lane * 16;
      frag[0] = (first >> 4) * 1024 + lane * 16;
      frag[1] = 0;
    }
  }
  // LDS byte of stage kt's slot
  __device__ __forceinline__ lds_char* slot(int kt) const {
    if constexpr (FORM == kRows) return lds + (kt >> 1) % 3 * (2 * kSlot);
    return lds + (kt & 3) * kSlot;
  }
  // two copies into a slot: a stage of kKMajor and kBlocks, one half of the rows of a
  // pair of stages (the pair of the even stage kt) of kRows
  __device__ __forceinline__ void issue(lds_char* base, int kt, bool live, int half = 0) const {
    typedef __attribute__((address_space(3))) void lds_void;
    if constexpr (FORM == kRows) {
      __amdgpu_buffer_rsrc_t r = whole;
      if (!live) r = range_rsrc(nullptr, 0);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(base + (wave * 4 + 2 * half + q) * 1024), 16,
                                                 (half ? off[2 + q] : off[q]) + kt * 64, 0, 0, 0);
    } else if constexpr (FORM == kKMajor) {
      int left = (int)s.extent - 32 * kt;
      left = !live || left < 0 ? 0 : (left < 32 ? left : 32);
      const __amdgpu_buffer_rsrc_t r = range_rsrc(s.p + (int64_t)kt * 32 * s.pitch, (int64_t)left * s.pitch);
#pragma unroll
      for (int q = 0; q < 2; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(base + (wave * 2 + q) * 1024), 16, off[q], 0, 0, 0);
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int64_t at = (wave * 2 + q) * s.pitch + (int64_t)kt * 1024;
        const bool in = live && at + 1024 <= s.extent;
        const __amdgpu_buffer_rsrc_t r = range_rsrc(in ? s.p + at : nullptr, 1024);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(base + (wave * 2 + q) * 1024), 16, off[q], 0, 0, 0);
      }
    }
  }
  // fragment I of a stage; half: which 64 bytes of a kRows row
  template <int I>
  __device__ __forceinline__ u32x4_t read(const lds_char* base, int half) const {
    typedef const __attribute__((address_space(3))) u32x4_t lds_u32x4;
    typedef __attribute__((address_space(3))) v4i16_t lds_v4i16;
    if constexpr (FORM == kKMajor) {
      const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(base + frag[I]));
      const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(base + frag[I] + 4 * 512));
      u32x4_t r;
      r.x = (uint32_t)(uint16_t)lo.x | ((uint32_t)(uint16_t)lo.y << 16);
      r.y = (uint32_t)(uint16_t)lo.z | ((uint32_t)(uint16_t)lo.w << 16);
      r.z = (uint32_t)(uint16_t)hi.x | ((uint32_t)(uint16_t)hi.y << 16);
      r.w = (uint32_t)(uint16_t)hi.z | ((uint32_t)(uint16_t)hi.w << 16);
      return r;
    } else if constexpr (FORM == kRows) {
      return *(lds_u32x4*)(base + frag[half] + I * (16 * 128));
    } else {
      return *(lds_u32x4*)(base + frag[0] + I * 1024);
    }
  }
};

// One stage: copies into wa, wb and wr (a row-major operand's pair), the MFMAs on
// fa / cur, and the next stage's fragments from na and nb.  The slots read and the slots
// written are different ones; `restrict` tells the compiler, which would otherwise wait
// for every copy in flight before a transposing read.
template <int FA, int FB, bool EVEN>
__device__ __forceinline__ void large_stage(const Stager<FA, 8>& a, const Stager<FB, 4>& b, const lds_char* __restrict__ na,
                                            const lds_char* __restrict__ nb, lds_char* __restrict__ wa,
                                            lds_char* __restrict__ wb, int kt, int KT, u32x4_t (&fa)[8], u32x4_t (&cur)[4],
                                            u32x4_t (&nxt)[4], f32x16_t (&acc)[4][2]) {
  // the copies after barrier kt: one stage (kt + 3) of the four-slot operands, half of a
  // pair (first the one of kt + 4, at odd kt the rest of it) of the row-major one
  constexpr int pair = EVEN ? 4 : 3, half = EVEN ? 0 : 1;
  if constexpr (FA == kRows) a.issue(wa, kt + pair, kt + pair < KT, half);
  else a.issue(wa, kt + 3, kt + 3 < KT);
  if constexpr (FB == kRows) b.issue(wb, kt + pair, kt + pair < KT, half);
  else b.issue(wb, kt + 3, kt + 3 < KT);
  __builtin_amdgcn_sched_barrier(0);
  static_for<8>([&](auto Sq) {
    constexpr int qs = decltype(Sq)::value;
    static_for<4>([&](auto Tq) {
      constexpr int qt = decltype(Tq)::value;
      mfma_quarter<2 * (qs & 1) + (qt & 1)>(acc[qs >> 1][qt >> 1], fa[qs], cur[qt]);
    });
    fa[qs] = a.template read<qs>(na, EVEN ? 1 : 0);
    if constexpr ((qs & 1) == 0) nxt[qs / 2] = b.template read<qs / 2>(nb, EVEN ? 1 : 0);
    __builtin_amdgcn_sched_barrier(0);
  });
}

// acc (quarter layout) += Σ over KT stages; FA and FB not both kRows (LDS)
template <int FA, int FB>
__device__ __forceinline__ void gemm_large(const Side& sa, const Side& sb, int KT, char* smem, f32x16_t (&acc)[4][2]) {
  static_assert(!(FA == kRows && FB == kRows), "two row-major operands do not fit the LDS");
  if (KT <= 0) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Stager<FA, 8> a(sa, smem, (wave >> 2) * 128);
  const Stager<FB, 4> b(sb, smem + form_lds(FA), (wave & 3) * 64);
  // prologue: stages 0 to 2 (of a row-major operand the pairs 0, 1 and 2, 3), the order of
  // the loop: 12 copies (stage 0 whole after the first 4 to 6, 8 or 6 behind it)
  if constexpr (FA == kRows) { a.issue(a.slot(0), 0, true, 0); a.issue(a.slot(0), 0, true, 1); }
  if constexpr (FB == kRows) { b.issue(b.slot(0), 0, true, 0); b.issue(b.slot(0), 0, true, 1); }
  for (int st = 0; st < 3; ++st) {
    if constexpr (FA != kRows) a.issue(a.slot(st), st, st < KT);
    if constexpr (FB != kRows) b.issue(b.slot(st), st, st < KT);
    if (st == 1) {
      if constexpr (FA == kRows) a.issue(a.slot(2), 2, 2 < KT, 0);
      if constexpr (FB == kRows) b.issue(b.slot(2), 2, 2 < KT, 0);
    }
    if (st == 2) {
      if constexpr (FA == kRows) a.issue(a.slot(2), 2, 2 < KT, 1);
      if constexpr (FB == kRows) b.issue(b.slot(2), 2, 2 < KT, 1);
    }
  }
  DMUON_WAIT_VM(8);                                      // own share of stage 0: 8 of the copies above come after it
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  u32x4_t fa[8], f0[4], f1[4];
  static_for<8>([&](auto I) { fa[decltype(I)::value] = a.template read<decltype(I)::value>(a.slot(0), 0); });
  static_for<4>([&](auto I) { f0[decltype(I)::value] = b.template read<decltype(I)::value>(b.slot(0), 0); });
  auto stage = [&](auto Even, int kt) {
    DMUON_WAIT_VM(4);                                    // all but the last stage's copies: stage kt + 1 has landed
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    large_stage<FA, FB, decltype(Even)::value>(a, b, a.slot(kt + 1), b.slot(kt + 1), a.slot(FA == kRows ? kt + 4 : kt + 3),
                                               b.slot(FB == kRows ? kt + 4 : kt + 3), kt, KT, fa,
                                               decltype(Even)::value ? f0 : f1, decltype(Even)::value ? f1 : f0, acc);
  };
  int kt = 0;
#pragma unroll 1
  for (; kt + 1 < KT; kt += 2) {
    stage(std::true_type{}, kt);
    stage(std::false_type{}, kt + 1);
  }
  if (kt < KT) stage(std::true_type{}, kt);
  DMUON_WAIT_VM(0);                                      // the empty copies past the last stage write LDS too
  __syncthreads();
}

template <int I>
__device__ __forceinline__ void zero_acc(f32x16_t (&acc)[I][2]) {
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
}

// acc = Σ over the plane pairs of the operands, given at plane 0 (planes in elements)
template <bool TA, bool TB>
__device__ __forceinline__ void small_planes(const Operands& op, int64_t a_plane, int64_t b_plane, const PlanePairs& pp,
                                             char* smem, f32x16_t (&acc)[2][2]) {
  zero_acc(acc);
#pragma unroll 1
  for (int p = 0; p < pp.n; ++p) {
    Operands o = op;
    o.a += (int64_t)((pp.a >> (4 * p)) & 15) * a_plane * 2;
    o.b += (int64_t)((pp.b >> (4 * p)) & 15) * b_plane * 2;
    gemm_small<TA, TB>(o, smem, acc);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) quarters_to_32x32(acc[i][j]);
}
template <int FA, int FB>
__device__ __forceinline__ void large_planes(const Side& sa, const Side& sb, int KT, int64_t a_plane, int64_t b_plane,
                                             const PlanePairs& pp, char* smem, f32x16_t (&acc)[4][2]) {
  zero_acc(acc);
#pragma unroll 1
  for (int p = 0; p < pp.n; ++p) {
    Side x = sa, y = sb;
    x.p += (int64_t)((pp.a >> (4 * p)) & 15) * a_plane * 2;
    y.p += (int64_t)((pp.b >> (4 * p)) & 15) * b_plane * 2;
    gemm_large<FA, FB>(x, y, KT, smem, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) quarters_to_32x32(acc[i][j]);
}

// Tile shapes.  A workgroup computes rows (A's side) × columns (B's side) of a
// product; a wave holds 32·I rows and 64 columns as I × 2 blocks of 32 × 32.
//   Large: 256 × 256 on 8 waves (gemm_large), one workgroup per CU;
//   Small: 128 × 128 on 4 waves (gemm_small), three workgroups per CU.
struct Large {
  static constexpr int I = 4, WC = 4;                    // row blocks per wave, waves along the columns
  static constexpr int M = 256, N = 256, Threads = 512, Lds = form_lds(kRows) + form_lds(kBlocks);   // 160 KiB
};
struct Small {
  static constexpr int I = 2, WC = 2;
  static constexpr int M = 128, N = 128, Threads = 256, Lds = kSmallStages * kSmallStage;
};

// A tile whose lanes hold output rows (the tile's columns) and whose registers hold
// consecutive output columns (the tile's rows) goes out through LDS as whole rows of
// 16-byte pieces.  f(i, j, r) is the value of register r of block (i, j).
// Rows ≥ rows and columns ≥ cols are dropped; `vec` says that whole pieces may be
// stored as such.  The stores are nontemporal: with plain ones the experts' weight
// gradients (738 MB of fp32) took 329 µs instead of 273, the cross-entropy gradients
// of 2400 tokens 2.60 ms instead of 2.35.
template <typename S, typename F>
__device__ __forceinline__ void store_tile(uint16_t* out, int64_t ld, int rows, int cols, bool vec, char* smem, F f) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = wave / S::WC, wc = wave % S::WC, h = lane >> 5, r32 = lane & 31;
  // 16-byte pieces XOR-swizzled by the row, so that the 32 rows one 8-byte write
  // instruction touches fall in all banks
  constexpr int P = S::M / 8;                            // pieces per row
#pragma unroll
  for (int i = 0; i < S::I; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int rq = 0; rq < 4; ++rq) {
        const int row = wc * 64 + j * 32 + r32;
        const int piece = (wr * S::I + i) * 4 + rq;
        const uint2 v = make_uint2(pack_bf16x2(f(i, j, 4 * rq), f(i, j, 4 * rq + 1)),
                                   pack_bf16x2(f(i, j, 4 * rq + 2), f(i, j, 4 * rq + 3)));
        *(uint2*)(smem + row * (P * 16) + ((piece ^ (row & (P - 1) & 31)) << 4) + h * 8) = v;
      }
  __syncthreads();
#pragma unroll 4
  for (int q = 0; q < S::N * P / S::Threads; ++q) {
    const int id = tid + S::Threads * q;
    const int row = id / P, piece = id % P;
    const u32x4_t v = *(const u32x4_t*)(smem + row * (P * 16) + ((piece ^ (row & (P - 1) & 31)) << 4));
    const int left = cols - piece * 8;
    if (row >= rows || left <= 0) continue;
    gptr<uint16_t> d = glob(out) + (int64_t)row * ld + piece * 8;
    if (vec && left >= 8) {
      __builtin_nontemporal_store(v, (gptr<u32x4_t>)d);
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) d[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
  __syncthreads();
}
// fp32: half of the rows at a time.  PART: a partial sum, which is read again soon
// (plain stores) and may `add` to what is there.
template <typename S, bool PART = false, typename F>
__device__ __forceinline__ void store_tile(float* out, int64_t ld, int rows, int cols, bool vec, char* smem, F f,
                                           bool add = false) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = wave / S::WC, wc = wave % S::WC, h = lane >> 5, r32 = lane & 31;
  constexpr int P = S::M / 4, R = S::N / 2;              // pieces per row, rows at a time
#pragma unroll 1
  for (int hf = 0; hf < 2; ++hf) {
    if (wc / (S::WC / 2) == hf) {
#pragma unroll
      for (int i = 0; i < S::I; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int rq = 0; rq < 4; ++rq) {
            const int row = wc % (S::WC / 2) * 64 + j * 32 + r32;
            const int piece = (wr * S::I + i) * 8 + rq * 2 + h;
            *(float4*)(smem + row * (P * 16) + ((piece ^ (row & 31)) << 4)) =
                make_float4(f(i, j, 4 * rq), f(i, j, 4 * rq + 1), f(i, j, 4 * rq + 2), f(i, j, 4 * rq + 3));
          }
    }
    __syncthreads();
#pragma unroll 4
    for (int q = 0; q < R * P / S::Threads; ++q) {
      const int id = tid + S::Threads * q;
      const int lr = id / P, piece = id % P, row = hf * R + lr;
      f32x4_t v = *(const f32x4_t*)(smem + lr * (P * 16) + ((piece ^ (lr & 31)) << 4));
      const int left = cols - piece * 4;
      if (row >= rows || left <= 0) continue;
      gptr<float> d = glob(out) + (int64_t)row * ld + piece * 4;
      if (PART) {                                        // whole pieces: ld is a multiple of 64
        if (add) v += *(gptr<f32x4_t>)d;
        *(gptr<f32x4_t>)d = v;
      } else if (vec && left >= 4) {
        __builtin_nontemporal_store(v, (gptr<f32x4_t>)d);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (e < left) d[e] = v[e];
      }
    }
    __syncthreads();
  }
}

// The map of xcd_logical_block<64> over the first G workgroups of a launch, G known on
// the device only; the others have nothing to do.
__device__ __forceinline__ int live_block(int G) {
  constexpr int run = 64, win = 8 * run;
  const int b = blockIdx.x, w = b / win, xcd = b & 7, slot = (b >> 3) - w * run;
  if ((w + 1) * win <= G) return w * win + xcd * run + slot;
  const int left = G - w * win, per = left >> 3, rem = left & 7;
  return w * win + (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + slot;
}

// ---------------------------------------------------------------------------
// logits tiles, 256 vocabulary rows × 256 tokens: z(v, t) = Σ_d W(v, d)·H(t, d).
// W is the core's A operand, so a lane's registers hold vocabulary entries of one
// token: the softmax statistics of a tile are register reductions, one exchange
// between the two lane halves and one between the two wave groups, through LDS.
// The logits themselves are never stored.
//   forward:  per tile and token the largest logit and Σ exp(z − largest), and the
//             target's logit;
//   backward: dZ(t, v) = g_t·(exp(z − lse_t) − [v = target]), rounded to bf16 (one
//             rounding, at most 2⁻⁸ of each entry: the matrix cores take bf16, and a
//             second plane would double both products; fp32 operands: three planes).
//             The gradients are then 0.0018 to 0.0023 of their norm away from the
//             64-bit ones, their own rounding to bf16 alone 0.0017; in fp32 4·10⁻⁷.
// The exponentials are 2^((z − largest)·log₂e) and 2^((z − lse)·log₂e), the difference
// first: it is exact where the two are close, so that the largest logit's own term is 1
// and a certain token's probability too, whatever their size (one fused multiply-add,
// z·log₂e − lse·log₂e, is off by lse·2⁻²⁴ in the exponent).  The target's entry is looked
// for only in parts of a tile that hold one (6% of them at 128000 words).  Bound by the product (see the large core): 4096 tokens × 4096, vocabulary
// 32000, forward: the whole call 870 µs = 1.23 PFLOP/s (the kernel under the profiler, at
// other clocks, 875 to 1210); 8192 × 4096 and 16384 rows, backward: 850 to 890 µs on
// average = 1.23 to 1.29.  Of a tile's 109 µs about 10 are prologue and epilogue, which nothing overlaps.
// ---------------------------------------------------------------------------
template <typename S, bool BACKWARD, bool F32>
__global__ __launch_bounds__(S::Threads) void k_ce_logits(CeLogitsArgs g) {
  extern __shared__ __align__(16) char smem[];
  // the order is laid over the tiles that tokens reach, so that every XCD gets its
  // share of them (2400 of 4001 tokens, vocabulary 50257: 692 µs over all tiles, 485 so)
  const int count = *g.count;
  const int tiles_t = (count + S::N - 1) / S::N, live = tiles_t * g.tiles_v;
  if ((int)blockIdx.x >= live) return;
  int tt, tv;
  band_tile(live_block(live), tiles_t, g.tiles_v, tt, tv);
  const int row0 = tv * S::M, col0 = tt * S::N;   // vocabulary (in the piece), tokens
  f32x16_t acc[S::I][2];
  const char* wp = (const char*)(g.w + (int64_t)row0 * g.ldw);
  if constexpr (S::I == 4) {
    const int64_t at = (int64_t)(col0 / 16) * (g.ldh / 32) * 1024;       // H is in fragment order
    const Side sa = {wp, g.ldw * 2, g.vrows - row0, 0};
    const Side sb = {(const char*)g.h + at, (g.ldh / 32) * 1024, g.h_plane * 2 - at, 0};
    large_planes<kRows, kBlocks>(sa, sb, g.kt, g.w_plane, g.h_plane, g.pairs, smem, acc);
  } else {
    Operands op;
    op.a = wp;
    op.b = (const char*)(g.h + (int64_t)col0 * g.ldh);
    op.lda_b = (int)(g.ldw * 2);
    op.ldb_b = (int)(g.ldh * 2);
    op.rows_a = g.vrows - row0;
    op.rows_b = count - col0;
    op.cola_b = op.colb_b = 0;
    op.ktiles = g.kt;
    small_planes<false, false>(op, g.w_plane, g.h_plane, g.pairs, smem, acc);
  }

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wr = wave / S::WC, wc = wave % S::WC, h = lane >> 5, r32 = lane & 31;
  const int vleft = g.vrows - row0 - wr * (32 * S::I) - h * 4;       // valid while register row < vleft
  const bool ragged = g.vrows - row0 < S::M;
  // register row of the target of column j's token, or −1
  int want[2];
  float L[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
  int tok[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    tok[j] = col0 + wc * 64 + j * 32 + r32;
    want[j] = -1;
    if (tok[j] < count) {
      const int y = g.tgt[tok[j]] - g.v0 - row0;
      if (y >= 0 && y < S::M && g.tgt[tok[j]] >= 0 && y / (32 * S::I) == wr && ((y >> 2) & 1) == h) want[j] = y % (32 * S::I) - 4 * h;
      if constexpr (BACKWARD) {
        L[j] = g.clse[tok[j]];
        w[j] = g.cg[tok[j]] / *g.gmax;
      }
    }
  }
  auto reg_row = [](int i, int r) { return i * 32 + (r >> 2) * 8 + (r & 3); };

  constexpr float kLog2e = 1.44269504088896341f;
  if constexpr (!BACKWARD) {
    CeStat* st = (CeStat*)smem;                              // [wave row][token of the tile]
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (ragged) {
#pragma unroll
        for (int i = 0; i < S::I; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (reg_row(i, r) >= vleft) acc[i][j][r] = -INFINITY;
      }
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < S::I; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) m = fmaxf(m, acc[i][j][r]);
      m = fmaxf(m, __shfl_xor(m, 32, 64));
      const float m0 = m == -INFINITY ? 0.f : m;             // then s is 0, or NaN if a logit is
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < S::I; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) s += __builtin_amdgcn_exp2f((acc[i][j][r] - m0) * kLog2e);
      s += __shfl_xor(s, 32, 64);
      if (h == 0) st[wr * S::N + wc * 64 + j * 32 + r32] = CeStat{m, s};
      if (__any(want[j] >= 0)) {                             // few tiles hold a token's target
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < S::I; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (reg_row(i, r) == want[j]) z = acc[i][j][r];
        if (want[j] >= 0) g.zt[tok[j]] = z;
      }
    }
    __syncthreads();
    if (tid < S::N && col0 + tid < count) {
      const CeStat a = st[tid], b = st[S::N + tid];
      const float m = fmaxf(a.m, b.m);
      const float sa = a.m == -INFINITY ? a.s : a.s * __expf(a.m - m);
      const float sb = b.m == -INFINITY ? b.s : b.s * __expf(b.m - m);
      g.stats[(int64_t)(g.v0 / S::M + tv) * g.tokens + col0 + tid] = CeStat{m, sa + sb};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int i = 0; i < S::I; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_amdgcn_exp2f((acc[i][j][r] - L[j]) * kLog2e);
      if (__any(want[j] >= 0)) {
#pragma unroll
        for (int i = 0; i < S::I; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (reg_row(i, r) == want[j]) acc[i][j][r] -= 1.f;
      }
#pragma unroll
      for (int i = 0; i < S::I; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] *= w[j];
      if (ragged) {
#pragma unroll
        for (int i = 0; i < S::I; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (reg_row(i, r) >= vleft) acc[i][j][r] = 0.f;
      }
    }
    uint16_t* out = g.dz + (int64_t)col0 * g.ldz + row0;
    const int rows = count - col0, cols = g.ldz - row0;
    if constexpr (F32) {
      // three planes: each stores what bf16 holds of the rest (exact differences)
#pragma unroll 1
      for (int q = 0; q < kPlanes; ++q) {
        store_tile<S>(out + q * g.dz_plane, g.ldz, rows, cols, true, smem, [&](int i, int j, int r) { return acc[i][j][r]; });
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < S::I; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] -= bf16_to_f32(f32_to_bf16(acc[i][j][r]));
      }
    } else {
      store_tile<S>(out, g.ldz, rows, cols, true, smem, [&](int i, int j, int r) { return acc[i][j][r]; });
    }
  }
}

// ---------------------------------------------------------------------------
// losses of at most 32 tokens (fp32: 64).  The bytes of W bound them, so W streams once from
// memory into registers: a wave takes 16 vocabulary rows over all of D, the
// fragments of U stages of 32 in flight while those before are multiplied, and the
// hidden states come from the caches (64 KiB at 16 tokens × 2048).  W is read as it
// is, of either type and any stride; fp32 values are split into planes in registers,
// their leading product summed apart from the five corrections.
// W's loads are nontemporal: with the caches full of another kernel's results, bf16,
// 16 tokens × 2048 and a vocabulary of 32000, the call takes 42 µs, with plain loads 61.
// The tiles of 128 against this, bf16, behind another kernel's results: 16 tokens × 4096,
// vocabulary 8000 75 and 41 µs, 32000 129 and 71, 128000 281 and 242; 32 tokens 76 and 47,
// 130 and 82, 292 and 284.  Called back to back, 32 tokens: 63 and 43, 75 and 78, 224 and
// 282: there the tiles win from a W of about 256 MB on (at 16 tokens from 1 GB, 221 and
// 238), which is not taken: a loss follows the model that made its hidden states.  64
// tokens behind a full cache 113 and 110, 262 and 363 (not taken).  fp32 × 2048, 32000:
// 16 tokens 405 and 75 µs, 64 tokens 421 and 135 (the tiles need W as planes first).
// ---------------------------------------------------------------------------
// The scan and the packing of so few tokens, in one launch: every wave finds the
// tokens' places by itself with one ballot.
__global__ __launch_bounds__(kThreads) void k_ce_few_start(CeScanArgs a, PackArgs p) {
  __shared__ int place[kThreads / 64][kFewTokens];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool here = lane < a.tokens;
  const int64_t y = load_index(a.targets, a.idx64, here ? lane : 0);
  const bool part = here && y != a.ignore;
  const uint64_t in = __ballot(part);
  const int count = __popcll(in), i = __popcll(in & ((1ull << lane) - 1));
  if (part) place[wave][i] = lane;
  if (blockIdx.x == 0 && wave == 0) {
    if (part) {
      a.rows[i] = lane;
      a.tgt[i] = list_target(y, a.vocab);
    } else if (here) {
      a.losses[lane] = 0.f;
      a.lse[lane] = 0.f;
    }
    if (lane == 0) *a.count = count;
  }
  __syncthreads();
  const int per = p.ldd >> 6;
  const int u = blockIdx.x * (kThreads / 64) + wave, g = u / per;
  const int c = (u - g * per) * 64 + (lane & 7) * 8, r = g * 8 + (lane >> 3);
  if (r >= count) return;
  pack_piece(p, r, place[wave][r], c, (p.ld & 7) == 0 && ((uintptr_t)p.src & 15) == 0);
}

template <typename T>
struct FewRaw;                           // 8 elements of a row of W as they were loaded
template <>
struct FewRaw<uint16_t> {
  u32x4_t u;
  __device__ __forceinline__ void load(gptr<const uint16_t> p) { u = __builtin_nontemporal_load((gptr<const u32x4_t>)p); }
  __device__ __forceinline__ void set(const float (&v)[8]) { u = pack8(v); }
  __device__ __forceinline__ void planes(u32x4_t (&f)[1]) const { f[0] = u; }
};
template <>
struct FewRaw<float> {
  f32x4_t a, b;
  __device__ __forceinline__ void load(gptr<const float> p) {
    a = __builtin_nontemporal_load((gptr<const f32x4_t>)p);
    b = __builtin_nontemporal_load((gptr<const f32x4_t>)p + 1);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = f32x4_t{v[0], v[1], v[2], v[3]};
    b = f32x4_t{v[4], v[5], v[6], v[7]};
  }
  __device__ __forceinline__ void planes(u32x4_t (&f)[kPlanes]) const {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float p[kPlanes][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float s[3];
      split3(v[e], s);
      p[0][e] = s[0]; p[1][e] = s[1]; p[2][e] = s[2];
    }
#pragma unroll
    for (int q = 0; q < kPlanes; ++q) f[q] = pack8(p[q]);
  }
};

__device__ __forceinline__ void mfma16(const u32x4_t& a, const u32x4_t& b, f32x4_t& c) {
  bf16x8_t va, vb;
  __builtin_memcpy(&va, &a, 16);
  __builtin_memcpy(&vb, &b, 16);
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, vb, c, 0, 0, 0);
}

// T: W's type, NT: tiles of 16 tokens, U: stages in flight
template <typename T, int NT, int U>
__global__ __launch_bounds__(kThreads) void k_ce_few(CeFewArgs g) {
  constexpr int P = sizeof(T) == 4 ? kPlanes : 1, waves = kThreads / 64;
  __shared__ CeStat part[waves][NT * 16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4, n = lane & 15;
  const int v0 = (blockIdx.x * waves + wave) * 16;
  const int row = v0 + n < g.vocab ? v0 + n : g.vocab - 1;               // a row of W, also past its end
  const gptr<const T> w = glob((const T*)g.w) + (int64_t)row * g.ldw;
  const gptr<const u32x4_t> h = (gptr<const u32x4_t>)glob(g.h) + n;       // fragment order: chunk c of stage k of tile j at 64·(j·kt + k) + 16·c
  const int64_t plane = g.h_plane / 8;
  const int full = g.vec ? g.width / 32 : 0;
  f32x4_t acc[NT][P == 1 ? 1 : 2];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int x = 0; x < (P == 1 ? 1 : 2); ++x) acc[j][x] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // Chunk c (8 columns) of W's row and of the tokens, for lane group q.  A sum may
  // take its K in any order: in the loop over whole stages a lane group takes the
  // chunks 2q and 2q + 1 of a pair of bf16 stages, 32 bytes together, so that a pair of loads
  // asks for whole lines (one stage after the other: 44 µs against 42.8 at 16 tokens).
  auto chunk = [&](int k, int odd) { return P == 1 ? 4 * k + 2 * q + odd : 4 * (k + odd) + q; };
  auto hidden = [&](int c, u32x4_t (&b)[NT][P]) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int x = 0; x < P; ++x) b[j][x] = h[x * plane + (int64_t)j * g.kt * 64 + c * 16];
  };
  auto multiply = [&](const FewRaw<T>& raw, const u32x4_t (&b)[NT][P]) {
    u32x4_t f[P];
    raw.planes(f);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if constexpr (P == 1) {
        mfma16(f[0], b[j][0], acc[j][0]);
      } else {
        mfma16(f[1], b[j][1], acc[j][1]);
        mfma16(f[2], b[j][0], acc[j][1]);
        mfma16(f[0], b[j][2], acc[j][1]);
        mfma16(f[1], b[j][0], acc[j][1]);
        mfma16(f[0], b[j][1], acc[j][1]);
        mfma16(f[0], b[j][0], acc[j][0]);
      }
    }
  };
  FewRaw<T> cur[U], next[U];
  u32x4_t hc[U][NT][P], hn[U][NT][P];
  int k = 0;
  if (full >= U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = chunk(u & ~1, u & 1);
      cur[u].load(w + c * 8);
      hidden(c, hc[u]);
    }
    for (; k + 2 * U <= full; k += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = chunk(k + U + (u & ~1), u & 1);
        next[u].load(w + c * 8);
        hidden(c, hn[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) multiply(cur[u], hc[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        cur[u] = next[u];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int x = 0; x < P; ++x) hc[u][j][x] = hn[u][j][x];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(cur[u], hc[u]);
    k += U;
  }
  const int last = (g.width + 31) / 32;
  for (; k < last; ++k) {                 // the rest, and rows that are not 16-byte aligned
    float x[8];
    load8(w + k * 32 + q * 8, k < full, g.width - k * 32 - q * 8, x);
    FewRaw<T> raw;
    raw.set(x);
    u32x4_t b[NT][P];
    hidden(4 * k + q, b);
    multiply(raw, b);
  }

  const int count = *g.count;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    f32x4_t z = acc[j][0];
    if constexpr (P > 1) z += acc[j][P > 1 ? 1 : 0];
    const float zr[4] = {z.x, z.y, z.z, z.w};
    const int t = j * 16 + n;
    const int want = t < count ? g.tgt[t] - v0 - 4 * q : -1;
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (v0 + 4 * q + r < g.vocab) m = fmaxf(m, zr[r]);
    m = fmaxf(m, __shfl_xor(m, 16, 64));
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    const float m0 = m == -INFINITY ? 0.f : m;               // then s is 0, or NaN if a logit is
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (v0 + 4 * q + r < g.vocab) {
        s += __expf(zr[r] - m0);
        if (r == want) g.zt[t] = zr[r];
      }
    s += __shfl_xor(s, 16, 64);
    s += __shfl_xor(s, 32, 64);
    if (q == 0) part[wave][t] = CeStat{m, s};
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < NT * 16 && t < count) {
    float m = part[0][t].m, s = 0.f;
#pragma unroll
    for (int x = 1; x < waves; ++x) m = fmaxf(m, part[x][t].m);
#pragma unroll
    for (int x = 0; x < waves; ++x) s += part[x][t].m == -INFINITY ? part[x][t].s : part[x][t].s * __expf(part[x][t].m - m);
    g.stats[(int64_t)blockIdx.x * g.tokens + t] = CeStat{m, s};
  }
}

// ---------------------------------------------------------------------------
// the tiles' statistics of each token joined: lse = M + log Σ s·exp(m − M),
// loss = (M − z_target) + log Σ …: neither term is negative, and the logarithm keeps its
// digits beside a large M (a target in another shard: the lse; one outside the
// vocabulary: NaN).  TOK tokens per
// workgroup: 16, or 4 where the tokens are few and their entries many (16 tokens: 500
// entries 5.6 and 3.2 µs, 2000 entries 17.8 and 5.9).
// ---------------------------------------------------------------------------
// (m, s) joined with another pair; a NaN in s stays
__device__ __forceinline__ void join_stat(CeStat& a, CeStat b) {
  const float m = fmaxf(a.m, b.m);
  a.s = (a.m == -INFINITY ? a.s : a.s * __expf(a.m - m)) + (b.m == -INFINITY ? b.s : b.s * __expf(b.m - m));
  a.m = m;
}
template <int TOK>
__global__ __launch_bounds__(kThreads) void k_ce_rows(CeRowsArgs a) {
  constexpr int per = kThreads / TOK, waves = kThreads / 64;
  __shared__ CeStat part[waves][TOK];
  const int count = *a.count;
  const int i0 = blockIdx.x * TOK;
  if (i0 >= count) return;
  const int ti = threadIdx.x % TOK, k = threadIdx.x / TOK;
  const int i = i0 + ti;
  CeStat all = {-INFINITY, 0.f};
  if (i < count) {
    for (int v = k; v < a.tiles_v; v += 4 * per) {
      CeStat x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        x[u] = v + per * u < a.tiles_v ? a.stats[(int64_t)(v + per * u) * a.tokens + i] : CeStat{-INFINITY, 0.f};
      const float m = fmaxf(fmaxf(fmaxf(x[0].m, x[1].m), fmaxf(x[2].m, x[3].m)), all.m);
      float s = all.m == -INFINITY ? all.s : all.s * __expf(all.m - m);
#pragma unroll
      for (int u = 0; u < 4; ++u) s += x[u].m == -INFINITY ? x[u].s : x[u].s * __expf(x[u].m - m);
      all = CeStat{m, s};
    }
  }
#pragma unroll
  for (int o = TOK; o < 64; o <<= 1) join_stat(all, CeStat{__shfl_xor(all.m, o, 64), __shfl_xor(all.s, o, 64)});
  if ((threadIdx.x & 63) < TOK) part[threadIdx.x >> 6][ti] = all;
  __syncthreads();
  if (threadIdx.x < TOK && i < count) {
    for (int q = 1; q < waves; ++q) join_stat(all, part[q][ti]);
    const float ls = logf(all.s);                            // ≥ 0: the largest logit's own term is 1
    const int t = a.rows[i];
    const int y = a.tgt[i];
    a.lse[t] = all.m + ls;
    a.losses[t] = y >= 0 ? (all.m - a.zt[i]) + ls : y == kTgtElsewhere ? all.m + ls : __uint_as_float(0x7fc00000u);
  }
}

// ---------------------------------------------------------------------------
// gradient products: C[row][col] = Σ_k B(k, row)·A(k, col), A K-major, B K-major
// (weight gradients: k = tokens) or row-major (hidden-state gradient: k =
// vocabulary).  The lanes hold rows and the registers consecutive columns.  The K
// range may be split over `splits` workgroups per tile, which then leave fp32
// partial sums for k_join; the hidden-state gradient adds up its vocabulary
// pieces that way too.  Its rows are the tokens that take part: with 2400 of 4001
// and planned splits of 2, 160 of 256 workgroups had work, and the gradient took 644
// µs over the vocabulary of 50257 against 435 with the splits spread over them.
// Bound by the core: 8192 tokens × 4096 and 16384 vocabulary rows, weight gradient
// 815 to 850 µs = 1.32 PFLOP/s, hidden states 840 to 870 = 1.29; 8192 × 4096 × 11008 from
// a checkpoint 630 to 670, at best 600, 688 tiles in three rounds of 256 CUs.  Short K is
// bound by the stores: 64 experts of 1408 × 2048 over 250 tokens each, 738 MB of fp32,
// 240 to 270 µs, at best 219 (averages of runs under the profiler, at its clocks).
// ---------------------------------------------------------------------------
__device__ __forceinline__ int row_splits(int rows, const RowSpread& p) {
  if (rows <= 0) return 1;
  const int by_grid = p.splits * p.tiles_r / ((rows + p.tile - 1) / p.tile);   // workgroups launched
  const int by_memory = (int)((int64_t)p.splits * p.rows / rows);              // partial sums' room
  const int s = by_grid < by_memory ? by_grid : by_memory;
  return s < p.most ? s : p.most;
}
template <typename S, bool TB>
__global__ __launch_bounds__(S::Threads) void k_product(ProductArgs g) {
  extern __shared__ __align__(16) char smem[];
  int rows = g.rows, tiles_r = g.tiles_r, splits = g.splits;
  int64_t k0 = 0, k1 = g.k, part_split = g.part_split;
  if (g.count) {
    const int n = *g.count;
    if (TB) {
      k1 = n < k1 ? n : k1;
    } else {
      rows = n < rows ? n : rows;
      tiles_r = (rows + S::N - 1) / S::N;
      splits = row_splits(rows, g.spread);
      part_split = (int64_t)rows * g.ldp;
    }
  }
  const int tiles = tiles_r * g.tiles_c, live = tiles * g.groups * splits;
  if ((int)blockIdx.x >= live) return;
  int u = live_block(live);
  const int split = u / (tiles * g.groups);
  u -= split * tiles * g.groups;
  const int group = u / tiles;
  u -= group * tiles;
  int tr, tc;
  if (g.tiles_c <= tiles_r) band_tile(u, g.tiles_c, tiles_r, tc, tr);
  else band_tile(u, tiles_r, g.tiles_c, tr, tc);
  const int row0 = tr * S::N, col0 = tc * S::M;
  if (g.offsets) {                       // clamped, so that no offset leaves the operands
    const int64_t a = g.offsets[group], b = g.offsets[group + 1];
    k0 = a < 0 ? 0 : (a < g.k ? a : g.k);
    k1 = b < k0 ? k0 : (b < g.k ? b : g.k);
  }
  if (splits > 1) {                      // whole pairs of stages per split
    const int64_t st = (k1 - k0 + 63) / 64, per = (st + splits - 1) / splits;
    const int64_t lo = k0 + per * split * 64, hi = lo + per * 64;
    k1 = hi < k1 ? hi : k1;
    k0 = lo < k1 ? lo : k1;
  }
  f32x16_t acc[S::I][2];
  const int kt = (int)((k1 - k0 + 31) / 32);
  const char* ap = (const char*)(g.a + k0 * g.lda);
  const char* bp = (const char*)(TB ? g.b + k0 * g.ldb : g.b + (int64_t)row0 * g.ldb + k0);
  if constexpr (S::I == 4) {
    const Side sa = {ap, g.lda * 2, k1 - k0, col0 * 2};
    const Side sb = {bp, g.ldb * 2, TB ? k1 - k0 : (int64_t)(rows - row0), row0 * 2};
    large_planes<kKMajor, TB ? kKMajor : kRows>(sa, sb, kt, g.a_plane, g.b_plane, g.pairs, smem, acc);
  } else {
    Operands op;
    op.a = ap;
    op.b = bp;
    op.lda_b = (int)(g.lda * 2);
    op.ldb_b = (int)(g.ldb * 2);
    op.rows_a = (int)(k1 - k0);
    op.rows_b = TB ? (int)(k1 - k0) : rows - row0;
    op.cola_b = col0 * 2;
    op.colb_b = TB ? row0 * 2 : 0;
    op.ktiles = kt;
    small_planes<true, TB>(op, g.a_plane, g.b_plane, g.pairs, smem, acc);
  }

  if (g.part) {
    store_tile<S, true>(g.part + split * part_split + ((int64_t)group * g.rows + row0) * g.ldp + col0, g.ldp, rows - row0, g.ldp - col0,
                        true, smem, [&](int i, int j, int r) { return acc[i][j][r]; }, g.add);
    return;
  }
  const float s = g.scale ? *g.scale : 1.f;
  const int64_t at = ((int64_t)group * g.rows + row0) * g.cols + col0;
  const int rl = rows - row0, cl = g.cols - col0;
  if (g.out_f32)
    store_tile<S>((float*)g.out + at, g.cols, rl, cl, (g.cols & 3) == 0 && ((uintptr_t)g.out & 15) == 0, smem,
               [&](int i, int j, int r) { return acc[i][j][r] * s; });
  else
    store_tile<S>((uint16_t*)g.out + at, g.cols, rl, cl, (g.cols & 7) == 0 && ((uintptr_t)g.out & 15) == 0, smem,
               [&](int i, int j, int r) { return acc[i][j][r] * s; });
}

// partial sums joined in a fixed order, scaled and rounded to the output's type
__global__ __launch_bounds__(kThreads) void k_join(JoinArgs a) {
  const int per = (a.cols + 7) >> 3;
  const int64_t n = a.rows * per, step = (int64_t)gridDim.x * kThreads;
  const float s = a.scale ? *a.scale : 1.f;
  const bool vec = (a.cols & 7) == 0 && ((uintptr_t)a.out & 15) == 0;
  int splits = a.splits;
  int64_t part_split = a.part_split;
  if (a.count) {
    const int taken = *a.count;
    splits = row_splits(taken, a.spread);
    part_split = (int64_t)taken * a.ldp;
  }
  for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < n; id += step) {
    const int64_t t = id / per;
    const int c = (int)(id - t * per) * 8;
    const int left = a.cols - c;
    const int64_t r = a.pos ? (int64_t)a.pos[t] : t;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r >= 0) {
      for (int q = 0; q < splits; ++q) {
        float x[8];
        load8(glob((const float*)a.part) + q * part_split + r * a.ldp + c, true, 8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += x[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= s;
    }
    if (a.out_f32) store8<true>(glob((float*)a.out) + t * a.cols + c, vec, left, v);
    else store8<true>(glob((uint16_t*)a.out) + t * a.cols + c, vec, left, v);
  }
}

// ---------------------------------------------------------------------------
// embedding lookup: out[t] = scale·table[id_t], zeros for an id outside the table.
// One piece of 8 elements per thread and step, a wave covers whole cache lines.  Bound by
// memory: 32768 tokens × 4096 bf16 84 µs, 6.4 TB/s of rows read (some from caches) and
// written; 32 tokens 3 µs, a launch.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void k_embed(EmbedArgs a) {
  const int per = a.width >> 3;
  const int64_t n = a.tokens * per, step = (int64_t)gridDim.x * kThreads;
  for (int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x; q < n; q += step) {
    const int64_t t = q / per;
    const int c = (int)(q - t * per) * 8;
    const int64_t id = load_index(a.ids, a.idx64, t);
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (id >= 0 && id < a.rows) {
      load8(glob((const T*)a.table) + id * a.ldt + c, true, 8, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= a.scale;
    }
    store8<true>(glob((T*)a.out) + t * a.width + c, true, 8, v);
  }
}

// Rows without 16-byte pieces of 8 elements: N elements per thread, the largest unit
// that the rows' alignment allows, so that a wave still covers whole lines (25472 tokens
// × 684 fp32: 23 µs, bf16 16; eight elements one by one per thread 62 and 39).
template <typename T, int N>
__global__ __launch_bounds__(kThreads) void k_embed_units(EmbedArgs a) {
  typedef T unit __attribute__((ext_vector_type(N)));
  const int per = a.width / N;
  const int64_t n = a.tokens * per, step = (int64_t)gridDim.x * kThreads;
  for (int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x; q < n; q += step) {
    const int64_t t = q / per;
    const int c = (int)(q - t * per) * N;
    const int64_t id = load_index(a.ids, a.idx64, t);
    unit u = {};
    if (id >= 0 && id < a.rows) {
      u = *(gptr<const unit>)(glob((const T*)a.table) + id * a.ldt + c);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if constexpr (sizeof(T) == 4) u[e] *= a.scale;
        else u[e] = f32_to_bf16(bf16_to_f32(u[e]) * a.scale);
      }
    }
    __builtin_nontemporal_store(u, (gptr<unit>)(glob((T*)a.out) + t * a.width + c));
  }
}

// ---------------------------------------------------------------------------
// stable radix sort of (id, token) pairs, 8 bits of the id per pass.  Ids outside
// the table get the key `rows` and sort last.
//
// Up to 65536 tokens (and ids below 2^19) take two launches: k_sort_block sorts runs
// of 8192 tokens, one workgroup each, and k_sort_merge places every pair by its rank
// in the other runs (one launch when one run is all).  In a run the words (id, index
// in the run) stay in registers; a pass ranks 64 of them at a time among equal
// digits by ballots, exchanges them through LDS and reads them back.  Every wave owns
// a contiguous part, so equal ids keep the order of their tokens whatever the timing.
// More tokens take three launches per pass.  Measured: 8192 tokens 14 µs (six
// launches of the general path: 40 and their gaps).
// ---------------------------------------------------------------------------
constexpr int kSortWaves = kThreads / 64;
constexpr int kSortRounds = kSortItems / kThreads;
constexpr int kBlockWaves = kScanThreads / 64;

// Lanes whose 8-bit digit equals this lane's, among those `on`.  Per bit: the lanes
// that have it (a ballot), complemented where this lane has not.
__device__ __forceinline__ uint64_t match_digit(uint32_t d, uint64_t on) {
  uint32_t lo = (uint32_t)on, hi = (uint32_t)(on >> 32);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const uint64_t m = __ballot((d >> b) & 1);
    const uint32_t mine = (uint32_t)((int32_t)(d << (31 - b)) >> 31);     // all ones where this lane has the bit
    lo &= ~((uint32_t)m ^ mine);
    hi &= ~((uint32_t)(m >> 32) ^ mine);
  }
  return ((uint64_t)hi << 32) | lo;
}
// LDS reads and writes of one wave stay in order, and are not moved across this
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_sched_barrier(0);     // nor is the ballots' arithmetic, which would hold registers for every round
}

template <int ITEMS>
__global__ __launch_bounds__(kScanThreads) void k_sort_block(SortArgs a) {
  __shared__ uint32_t words[kScanThreads * ITEMS];
  __shared__ uint32_t cnt[kBlockWaves][256];
  __shared__ uint32_t wave_sum[kBlockWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int first = wave * 64 * ITEMS + lane;              // item r of this lane: first + 64 r
  const int64_t run0 = (int64_t)blockIdx.x * kSortRun;
  const int n = (int)(a.tokens - run0 < kSortRun ? a.tokens - run0 : kSortRun);
  uint32_t w[ITEMS];
  uint32_t at[ITEMS];                                      // rank in the wave's part
#pragma unroll
  for (int r = 0; r < ITEMS; ++r) {
    const int i = first + 64 * r;
    const int64_t id = load_index(a.ids, a.idx64, run0 + (i < n ? i : n - 1));
    const uint32_t key = id >= 0 && id < a.rows ? (uint32_t)id : (uint32_t)a.rows;
    w[r] = i < n ? (key << kSortRunBits) | (uint32_t)i : 0xffffffffu;     // past the end: last, and stays last
  }
  for (int shift = 0; shift < a.key_bits; shift += 8) {
    const int bits = a.key_bits - shift < 8 ? a.key_bits - shift : 8;
    const uint32_t mask = (1u << bits) - 1;
#pragma unroll
    for (int k = 0; k < 4; ++k) cnt[wave][lane + 64 * k] = 0;
    wave_order();
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) {
      const uint32_t d = (w[r] >> (kSortRunBits + shift)) & mask;
      const uint64_t same = match_digit(d, ~0ull);
      const uint32_t rank = (uint32_t)__popcll(same & ((1ull << lane) - 1));
      const uint32_t before = cnt[wave][d];
      at[r] = before + rank;
      wave_order();                                        // every lane has read before the first of each digit adds
      if (rank == 0) cnt[wave][d] = before + (uint32_t)__popcll(same);
      wave_order();
    }
    __syncthreads();
    // exclusive scan over (digit, wave): thread t holds waves 4(t & 3) … + 3 of digit t >> 2
    const int d0 = tid >> 2, v0 = 4 * (tid & 3);
    uint32_t c[4], s = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c[k] = cnt[v0 + k][d0];
      s += c[k];
    }
    uint32_t incl = s;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t up = __shfl_up(incl, o, 64);
      if (lane >= o) incl += up;
    }
    if (lane == 63) wave_sum[wave] = incl;
    __syncthreads();
    uint32_t base = incl - s;
    for (int v = 0; v < wave; ++v) base += wave_sum[v];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      cnt[v0 + k][d0] = base;
      base += c[k];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) words[cnt[wave][(w[r] >> (kSortRunBits + shift)) & mask] + at[r]] = w[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ITEMS; ++r) w[r] = words[first + 64 * r];
  }
  const bool all = a.tokens <= kSortRun;                   // the run is everything: write pairs, else words
#pragma unroll
  for (int r = 0; r < ITEMS; ++r) {
    const int i = first + 64 * r;
    if (i >= n) continue;
    if (all) {
      a.keys_out[i] = w[r] >> kSortRunBits;
      a.idx_out[i] = w[r] & (kSortRun - 1);
    } else {
      a.words[run0 + i] = w[r];
    }
  }
}

// Rank of every word among all runs: its place in its own, plus the words of the
// earlier runs with an id not above its own and of the later ones with an id below
// it.  The searches of a thread advance together, one probe of every run per step.
// Latency bound: 13 µs for 32768 tokens.
__global__ __launch_bounds__(kThreads) void k_sort_merge(SortArgs a) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= a.tokens) return;
  const int run = (int)(i / kSortRun), runs = (a.tokens + kSortRun - 1) / kSortRun;
  const uint32_t w = a.words[i], key = w >> kSortRunBits;
  constexpr int kMaxRuns = kSortRunsMax / kSortRun;
  int lo[kMaxRuns], hi[kMaxRuns];
#pragma unroll
  for (int q = 0; q < kMaxRuns; ++q) {
    lo[q] = 0;
    hi[q] = 0;
    if (q < runs && q != run) hi[q] = a.tokens - q * kSortRun < kSortRun ? a.tokens - q * kSortRun : kSortRun;
  }
  // first word of run q at or above `bound`: the id itself, or the next one for an
  // earlier run (the planner keeps rows + 1 below 2^19, so the bound fits)
  for (int step = 0; step <= kSortRunBits; ++step) {
#pragma unroll
    for (int q = 0; q < kMaxRuns; ++q) {
      if (lo[q] >= hi[q]) continue;
      const int mid = (lo[q] + hi[q]) >> 1;
      const uint32_t bound = (key + (q < run ? 1u : 0u)) << kSortRunBits;
      if (glob(a.words)[(int64_t)q * kSortRun + mid] < bound) lo[q] = mid + 1;
      else hi[q] = mid;
    }
  }
  int at = (int)(i - (int64_t)run * kSortRun);
#pragma unroll
  for (int q = 0; q < kMaxRuns; ++q) at += lo[q];
  a.keys_out[at] = key;
  a.idx_out[at] = (uint32_t)(run * kSortRun) + (w & (kSortRun - 1));
}

// The same for any number of tokens: per pass the digit counts of every workgroup,
// one scan over [digit][workgroup], and the stable placement.
__device__ __forceinline__ void sort_pair(const SortArgs& a, int64_t i, uint32_t& key, uint32_t& idx) {
  if (a.keys_in) {
    key = a.keys_in[i];
    idx = a.idx_in[i];
  } else {
    const int64_t id = load_index(a.ids, a.idx64, i);
    key = id >= 0 && id < a.rows ? (uint32_t)id : (uint32_t)a.rows;
    idx = (uint32_t)i;
  }
}

__global__ __launch_bounds__(kThreads) void k_sort_count(SortArgs a) {
  __shared__ uint32_t cnt[256];
  cnt[threadIdx.x] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kSortItems;
#pragma unroll 4
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = base + r * kThreads + threadIdx.x;
    if (i < a.tokens) {
      uint32_t key, idx;
      sort_pair(a, i, key, idx);
      atomicAdd(&cnt[(key >> a.shift) & 255], 1u);
    }
  }
  __syncthreads();
  a.hist[(int64_t)threadIdx.x * a.blocks + blockIdx.x] = cnt[threadIdx.x];
}

// exclusive scan of hist[256·blocks] in place, one workgroup
__global__ __launch_bounds__(kScanThreads) void k_sort_scan(SortArgs a) {
  __shared__ uint32_t wave_sum[kBlockWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = 256 * a.blocks, chunk = (n + kScanThreads - 1) / kScanThreads;
  const int i0 = tid * chunk, i1 = i0 + chunk < n ? i0 + chunk : n;
  uint32_t s = 0;
  for (int i = i0; i < i1; ++i) s += a.hist[i];
  uint32_t incl = s;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t up = __shfl_up(incl, o, 64);
    if (lane >= o) incl += up;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  uint32_t at = incl - s;
  for (int w = 0; w < wave; ++w) at += wave_sum[w];
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = a.hist[i];
    a.hist[i] = at;
    at += x;
  }
}

__global__ __launch_bounds__(kThreads) void k_sort_place(SortArgs a) {
  __shared__ uint32_t at[kSortWaves][256];           // next slot of each wave and digit
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) at[w][tid] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kSortItems + wave * (kSortItems / kSortWaves);
  uint32_t key[kSortRounds], idx[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = base + r * 64 + lane;
    key[r] = idx[r] = 0;
    if (i < a.tokens) {
      sort_pair(a, i, key[r], idx[r]);
      atomicAdd(&at[wave][(key[r] >> a.shift) & 255], 1u);
    }
  }
  __syncthreads();
  uint32_t first = a.hist[(int64_t)tid * a.blocks + blockIdx.x];
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    const uint32_t c = at[w][tid];
    at[w][tid] = first;
    first += c;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = base + r * 64 + lane;
    const bool on = i < a.tokens;
    const uint32_t d = (key[r] >> a.shift) & 255;
    const uint64_t same = match_digit(d, __ballot(on));
    const int rank = __popcll(same & ((1ull << lane) - 1));
    uint32_t slot = 0;
    if (on) slot = at[wave][d];
    wave_order();
    if (on && rank == 0) at[wave][d] = slot + (uint32_t)__popcll(same);
    wave_order();
    if (on) {
      a.keys_out[slot + rank] = key[r];
      a.idx_out[slot + rank] = idx[r];
    }
  }
}

// ---------------------------------------------------------------------------
// the table's gradient from the sorted tokens.
// A row's gradient is the sum over a contiguous range of sorted tokens.  Ranges
// are cut at fixed multiples of 32 and 1024: a whole aligned run of equal ids is
// summed once by k_embed_run (level 0 from the tokens, level 1 from 32 sums of
// level 0), and k_embed_grad adds at most 62 tokens and 62 first-level sums to a
// row besides its second-level ones, so a frequent token is spread over many
// workgroups and the order of every sum is fixed.
// ---------------------------------------------------------------------------
template <typename G> struct Raw8;                   // 8 elements as loaded
template <> struct Raw8<uint16_t> {
  u32x4_t u;
  __device__ __forceinline__ void load(gptr<const uint16_t> p) { u = *(gptr<const u32x4_t>)p; }
  __device__ __forceinline__ void add(float (&v)[8]) const {
    float x[8];
    unpack8(u, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += x[k];
  }
};
template <> struct Raw8<float> {
  f32x4_t u[2];
  __device__ __forceinline__ void load(gptr<const float> p) {
    u[0] = ((gptr<const f32x4_t>)p)[0];
    u[1] = ((gptr<const f32x4_t>)p)[1];
  }
  __device__ __forceinline__ void add(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] += u[0][k];
      v[4 + k] += u[1][k];
    }
  }
};

// v += Σ of rows s … e − 1 (of row(i)), in order, 8 loads in flight
template <typename G, typename R>
__device__ __forceinline__ void add_rows(int s, int e, bool vec, int left, float (&v)[8], R row) {
  constexpr int kAhead = 8;
  if (vec) {
    for (int i = s; i < e; i += kAhead) {
      Raw8<G> x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i + u < e) x[u].load(row(i + u));
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i + u < e) x[u].add(v);
    }
  } else {
#pragma unroll 1
    for (int i = s; i < e; ++i) {
      float x[8];
      load8(row(i), false, left, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] += x[k];
    }
  }
}
template <typename G>
__device__ __forceinline__ void add_tokens(const EmbedGradArgs& a, int s, int e, int c, float (&v)[8]) {
  add_rows<G>(s, e, a.vec_in, a.width - c, v, [&](int i) { return glob((const G*)a.grad) + (int64_t)a.idx[i] * a.ldg + c; });
}
__device__ __forceinline__ void add_sums(const float* part, int ld, int s, int e, int c, float (&v)[8]) {
  add_rows<float>(s, e, true, 8, v, [&](int i) { return glob(part) + (int64_t)i * ld + c; });
}

// One whole run of equal ids per workgroup and 512 columns; each wave sums a
// quarter of it, the quarters are added in order.  6 and 3 µs (levels 0 and 1) for 8192
// tokens × 2048 of natural frequencies, 28 and 5 for 32768 × 4096.
template <typename G, int LEVEL>
__global__ __launch_bounds__(kThreads) void k_embed_run(EmbedGradArgs a) {
  constexpr int span = LEVEL == 0 ? kRun : kRun * kRun;
  __shared__ float sum[kThreads / 64][512];
  const int64_t s = (int64_t)blockIdx.x * span;
  if (s + span > a.tokens) return;
  const uint32_t key = a.keys[s];
  if (key != a.keys[s + span - 1] || key >= (uint32_t)a.rows || (int64_t)key == (int64_t)a.padding) return;
  const int ld = (a.width + 7) & ~7;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.y * 512 + lane * 8;
  constexpr int quarter = kRun / (kThreads / 64);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < ld) {
    const int i = (LEVEL == 0 ? (int)s : (int)blockIdx.x * kRun) + wave * quarter;
    if constexpr (LEVEL == 0) add_tokens<G>(a, i, i + quarter, c, v);
    else add_sums(a.part[0], ld, i, i + quarter, c, v);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[wave][lane * 8 + k] = v[k];
  __syncthreads();
  for (int k = threadIdx.x; k < 512; k += kThreads) {
    const int col = blockIdx.y * 512 + k;
    if (col < ld) glob(a.part[LEVEL])[(int64_t)blockIdx.x * ld + col] = (sum[0][k] + sum[1][k]) + (sum[2][k] + sum[3][k]);
  }
}

// [s, e) of sorted positions added to v: whole aligned runs through their sums
template <typename G>
__device__ __forceinline__ void add_range(const EmbedGradArgs& a, int s, int e, int c, float (&v)[8]) {
  const int ld = (a.width + 7) & ~7;
  const int s0 = (s + kRun - 1) / kRun, e0 = e / kRun;          // whole first-level runs [s0, e0)
  if (s0 >= e0) {
    add_tokens<G>(a, s, e, c, v);
    return;
  }
  add_tokens<G>(a, s, s0 * kRun, c, v);
  const int s1 = (s0 + kRun - 1) / kRun, e1 = e0 / kRun;
  if (s1 >= e1) {
    add_sums(a.part[0], ld, s0, e0, c, v);
  } else {
    add_sums(a.part[0], ld, s0, s1 * kRun, c, v);
    add_sums(a.part[1], ld, s1, e1, c, v);
    add_sums(a.part[0], ld, e1 * kRun, e0, c, v);
  }
  add_tokens<G>(a, e0 * kRun, e, c, v);
}

// first sorted position with an id ≥ want, by one wave: 64 probes per step
__device__ __forceinline__ int wave_lower_bound(const uint32_t* keys, int n, int64_t want) {
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = n;                                // the answer is in [lo, hi]
  while (hi - lo > 0) {
    const int step = (hi - lo + 63) / 64;
    const int at = lo + lane * step;                 // probe: keys[at] < want?
    const bool below = at < hi && (int64_t)keys[at] < want;
    const int k = __popcll(__ballot(below));         // the probes below come first
    if (k == 0) return lo;
    const int nlo = lo + (k - 1) * step + 1;
    const int nhi = k < 64 ? (lo + k * step < hi ? lo + k * step : hi) : hi;
    lo = nlo;
    hi = nhi;
  }
  return lo;
}

// One launch, two kinds of workgroups: the sums, which wait on latency, first, then
// the zeros, which wait on bandwidth.  Zeros leave with nontemporal stores: with plain
// ones the sums' loads waited behind them (8192 tokens into 32000 × 2048 bf16: 55 µs,
// nontemporal 33 = 5 TB/s, either alone 20 to 24; interleaved 59, zeros first 57).
//   sums:  one wave per 8 sorted positions and 512 columns.  It owns the ranges that
//          begin there: the rows of their tokens among the 8 are loaded at once, added
//          in order, and a range that ends is written (or added) to its row.  A range
//          that goes on past the 8 is finished (32 tokens and more: summed) by
//          add_range.
//   zeros: 16 to 256 table rows per workgroup, 32 KiB where they are short (92945 × 64
//          bf16, 14976 tokens: 15 µs, 16 rows each 30); those without tokens are cleared (none of them
//          when accumulating).
template <typename G, typename O>
__device__ __forceinline__ void embed_sums(const EmbedGradArgs& a, int64_t wg) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slab = (int)(wg % a.slabs);
  const int64_t at = (wg / a.slabs * (kThreads / 64) + wave) * kEmbedHeads;
  if (at >= a.tokens) return;
  const int s0 = (int)at, p = s0 + lane;
  // 64 keys and token indices from s0; a head is a key that differs from the one before
  const bool in = p < a.tokens;
  const int pc = in ? p : a.tokens - 1;
  const uint32_t key = a.keys[pc], idx = a.idx[pc], prev = a.keys[pc > 0 ? pc - 1 : 0];
  const uint64_t heads = __ballot(p == 0 || !in || key != prev);       // a position past the end ends a range
  const int c = slab * 512 + lane * 8;
  const bool mine = c < a.width;
  const int have = a.tokens - s0 < kEmbedHeads ? a.tokens - s0 : kEmbedHeads;
  const uint32_t h8 = (uint32_t)heads & ((1u << have) - 1);
  if (!h8) return;
  const int first = __ffs(h8) - 1, last = 31 - __clz(h8);
  // the last range's end: among the 64 keys, else by search
  const uint64_t after = heads & ~((2ull << last) - 1);
  const int e = after ? s0 + __ffsll((unsigned long long)after) - 1
                      : s0 + 64 + wave_lower_bound(a.keys + s0 + 64, a.tokens - s0 - 64, (int64_t)__builtin_amdgcn_readlane((int)key, last) + 1);
  const bool longer = e - s0 > kEmbedHeads;          // it goes on past the 8
  const bool summed = longer && (e - (s0 + last) >= kRun || !a.vec_in);
  const int stop = summed ? last : (longer ? kEmbedHeads : e - s0);    // positions [first, stop) are loaded here
  Raw8<G> x[kEmbedHeads];
  const bool direct = mine && a.vec_in;
#pragma unroll
  for (int u = 0; u < kEmbedHeads; ++u)
    if (direct && u >= first && u < stop)
      x[u].load(glob((const G*)a.grad) + (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)idx, u) * a.ldg + c);
  auto finish = [&](int l, float (&v)[8]) {          // write the row of the range that begins at position l
    const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)key, l);
    if (!mine || k >= (uint32_t)a.rows || (int64_t)k == (int64_t)a.padding) return;
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= a.scale;
    gptr<O> out = glob((O*)a.out) + (int64_t)k * a.width + c;
    if (a.accumulate) {
      float o[8];
      load8((gptr<const O>)out, a.vec_out, a.width - c, o);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += o[q];
    }
    store8(out, a.vec_out, a.width - c, v);
  };
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  int head = first;
#pragma unroll
  for (int u = 0; u < kEmbedHeads; ++u) {
    if (u < first || u >= stop) continue;
    if (u > first && ((h8 >> u) & 1)) {
      finish(head, v);
      head = u;
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = 0.f;
    }
    if (a.vec_in) {
      x[u].add(v);
    } else if (mine) {
      float y[8];
      load8(glob((const G*)a.grad) + (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)idx, u) * a.ldg + c, false, a.width - c, y);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] += y[q];
    }
  }
  if (summed) {
    if (stop > first) finish(head, v);
    head = last;
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = 0.f;
    if (mine) add_range<G>(a, s0 + last, e, c, v);
  } else if (longer && mine) {
    add_tokens<G>(a, s0 + kEmbedHeads, e, c, v);
  }
  finish(head, v);
}

template <typename O>
__device__ __forceinline__ void embed_zeros(const EmbedGradArgs& a, int64_t wg, int* start) {
  const int n = a.zero_rows;
  const int64_t v0 = wg * n;
  const int wave = threadIdx.x >> 6;
  if (wave < 2) {
    const int at = wave_lower_bound(a.keys, a.tokens, wave ? v0 + n : v0);
    if ((threadIdx.x & 63) == 0) start[wave ? n : 0] = at;
  }
  __syncthreads();
  const int lo0 = start[0], hi0 = start[n];
  __syncthreads();
  // start[r] becomes nonzero where row v0 + r has tokens: by marking the keys of a
  // short range, by a search per row for a long one
  if ((int)threadIdx.x < n) {
    int has = 0;
    if (hi0 - lo0 > kThreads) {
      const int64_t want = v0 + threadIdx.x;
      int lo = lo0, hi = hi0;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)a.keys[mid] < want) lo = mid + 1; else hi = mid;
      }
      has = lo < hi0 && (int64_t)a.keys[lo] == want;
    }
    start[threadIdx.x] = has;
  }
  __syncthreads();
  if (hi0 - lo0 <= kThreads && (int)threadIdx.x < hi0 - lo0) start[(int64_t)a.keys[lo0 + threadIdx.x] - v0] = 1;
  __syncthreads();
  constexpr int E = 16 / (int)sizeof(O);             // elements per 16-byte store
  const int per = a.vec_out ? a.width / E : a.width;     // stores per row
  const int rows = a.rows - v0 < n ? (int)(a.rows - v0) : n;
  for (int q = threadIdx.x; q < rows * per; q += kThreads) {
    const int r = q / per, c = q - r * per;
    if (start[r] && v0 + r != a.padding) continue;
    gptr<O> out = glob((O*)a.out) + (v0 + r) * a.width;
    if (a.vec_out) __builtin_nontemporal_store(u32x4_t{0u, 0u, 0u, 0u}, (gptr<u32x4_t>)(out + c * E));
    else out[c] = O(0);
  }
}

template <typename G, typename O>
__global__ __launch_bounds__(kThreads) void k_embed_grad(EmbedGradArgs a) {
  __shared__ int start[kThreads + 1];
  const int64_t wg = blockIdx.x;
  if (wg < a.seg_wg) embed_sums<G, O>(a, wg);
  else embed_zeros<O>(a, wg - a.seg_wg, start);
}

// ---------------------------------------------------------------------------
// 8-bit checkpoints.  32 columns of a row share the exponent byte b, q is a signed
// byte and the value q·2^(b − 133).  b is the biased fp32 exponent of the block's
// largest magnitude (one more where that would round to 128, unless b = 254, where
// q saturates at 127), so that q = rint(x·2^(133 − b)) has |q| ≤ 127 and every
// value is kept to within 2^(b − 134), half a step, or a step where q saturates (at
// most 1/127.5 of the block's largest).  A block whose largest magnitude is below 2^−126
// becomes zeros (b = 0); a block that holds an infinity or NaN reads back as NaN
// (b = 255).  q·2^(b − 133) is exact in bf16.
// Four threads share a block, 8 columns each.  Bound by memory: 8192 × 11008 bf16 stored
// in 50 µs (5.4 TB/s), read back in 40 (6.8 TB/s, what was just stored from the caches).
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void k_ckpt_quantize(CodecArgs a) {
  const int64_t n = a.rows * a.blocks * 4, step = (int64_t)gridDim.x * kThreads;
  const bool vec_q = (a.cols & 7) == 0 && ((uintptr_t)a.q & 7) == 0;
  // whole waves step together: the exchanges below are among four neighbours
  for (int64_t id0 = (int64_t)blockIdx.x * kThreads; id0 < n; id0 += step) {
    const int64_t id = id0 + threadIdx.x;
    const bool on = id < n;
    const int64_t blk = id >> 2;
    const int64_t r = on ? blk / a.blocks : 0;
    const int b = (int)(blk - r * a.blocks);
    const int c = b * 32 + (int)(id & 3) * 8;
    const int left = a.cols - c;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on && left > 0) load8(glob((const T*)a.x) + r * a.ldx + c, a.vec && left >= 8, left, v);
    uint32_t m = 0;                                            // largest magnitude's bits (NaN above inf)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t u = __float_as_uint(v[e]) & 0x7fffffffu;
      m = u > m ? u : m;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const uint32_t u = (uint32_t)__shfl_xor((int)m, o, 64);
      m = u > m ? u : m;
    }
    int eb = (int)(m >> 23);                                   // 0: zeros, 255: not finite
    if (eb > 0 && eb < 254 && (m & 0x7fffffu) >= 0x7f0000u) ++eb;   // 127.5/64 = 1.9921875 and up
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float q = eb > 0 && eb < 255 ? rintf(__builtin_amdgcn_ldexpf(v[e], 133 - eb)) : 0.f;
      q = fminf(fmaxf(q, -127.f), 127.f);
      w[e >> 2] |= ((uint32_t)(int)q & 255u) << (8 * (e & 3));
    }
    if (!on) continue;
    gptr<int8_t> d = glob(a.q) + r * a.cols + c;
    if (vec_q && left >= 8) {
      typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
      *(gptr<u32x2>)d = u32x2{w[0], w[1]};         // nontemporal: as fast, but reading 90 MB back takes 55 µs instead of 42
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) d[e] = (int8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
    if ((id & 3) == 0) glob(a.exps)[blk] = (uint8_t)eb;
  }
}

template <typename T, bool NT>
__global__ __launch_bounds__(kThreads) void k_ckpt_read(CodecArgs a) {
  const int per = (a.cols + 7) >> 3;
  const int64_t n = a.rows * per, step = (int64_t)gridDim.x * kThreads;
  const bool vec_q = (a.cols & 7) == 0 && ((uintptr_t)a.q & 7) == 0;
  for (int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x; id < n; id += step) {
    const int64_t r = id / per;
    const int c = (int)(id - r * per) * 8;
    const int left = a.cols - c;
    const int eb = glob((const uint8_t*)a.exps)[r * a.blocks + (c >> 5)];
    gptr<const int8_t> q = glob((const int8_t*)a.q) + r * a.cols + c;
    uint32_t w[2] = {0u, 0u};
    if (vec_q) {
      typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 u = __builtin_nontemporal_load((gptr<const u32x2>)q);   // read once: experts' gradients 263 → 237 µs
      w[0] = u.x;
      w[1] = u.y;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) w[e >> 2] |= ((uint32_t)q[e] & 255u) << (8 * (e & 3));
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = __builtin_amdgcn_ldexpf((float)(int8_t)(w[e >> 2] >> (8 * (e & 3))), eb - 133);
      v[e] = eb == 255 ? __uint_as_float(0x7fc00000u) : x;
    }
    store8<NT>(glob((T*)a.out) + r * a.ldo + c, a.vec && left >= 8, left, v);
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
// Workgroups of a grid-stride kernel: enough to fill 256 CUs several times over
static unsigned stride_grid(int64_t items) {
  const int64_t wg = cdiv(items, kThreads);
  return (unsigned)(wg < 1 ? 1 : (wg < 16384 ? wg : 16384));
}

// Dynamic LDS limit of a kernel, raised once per device (first calls may come from
// several threads); `ready` holds one bit per device.
static int raise_lds(const void* kernel, int bytes, std::atomic<uint64_t>& ready) {
  static std::mutex mu;
  int dev = 0;
  int e = (int)hipGetDevice(&dev);
  if (e) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t)1 << dev : 0;
  if (bit && (ready.load(std::memory_order_acquire) & bit)) return 0;
  std::lock_guard<std::mutex> lk(mu);
  e = (int)hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == 0 && bit) ready.fetch_or(bit, std::memory_order_release);
  return e;
}

#define DMUON_LAUNCH(phase, stream, kernel, grid, block, lds, ...)                             \
  do {                                                                                         \
    timing_before(phase, stream);                                                              \
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(block), lds, (hipStream_t)(stream), __VA_ARGS__); \
    const int err_ = (int)hipGetLastError();                                                   \
    timing_after(phase, stream);                                                               \
    return err_;                                                                               \
  } while (0)

int launch_pack(const PackArgs& a, int phase, void* stream) {
  DMUON_LAUNCH(phase, stream, k_pack, stride_grid(round_up(a.rows, 8) * (a.ldd / 8)), kThreads, 0, a);
}
int launch_ce_scan(const CeScanArgs& a, void* stream) {
  DMUON_LAUNCH(PH_CE_PACK, stream, k_ce_scan, 1, kScanThreads, 0, a);
}
template <typename S, bool BACKWARD, bool F32>
static int ce_logits(const CeLogitsArgs& a, void* stream) {
  static std::atomic<uint64_t> ready{0};
  const int e = raise_lds((const void*)k_ce_logits<S, BACKWARD, F32>, S::Lds, ready);
  if (e) return e;
  DMUON_LAUNCH(PH_CE_LOGITS, stream, (k_ce_logits<S, BACKWARD, F32>), (unsigned)(a.tiles_t * a.tiles_v), S::Threads, S::Lds, a);
}
int launch_ce_logits(const CeLogitsArgs& a, int backward, int f32, void* stream) {
  if (a.tile == Large::M) {
    if (!backward) return ce_logits<Large, false, false>(a, stream);
    return f32 ? ce_logits<Large, true, true>(a, stream) : ce_logits<Large, true, false>(a, stream);
  }
  if (!backward) return ce_logits<Small, false, false>(a, stream);
  return f32 ? ce_logits<Small, true, true>(a, stream) : ce_logits<Small, true, false>(a, stream);
}
int launch_ce_few_start(const CeScanArgs& a, const PackArgs& p, void* stream) {
  DMUON_LAUNCH(PH_CE_PACK, stream, k_ce_few_start, (unsigned)cdiv(cdiv(a.tokens, 8) * (p.ldd / 64), kThreads / 64), kThreads, 0, a, p);
}
int launch_ce_few(const CeFewArgs& a, int f32, void* stream) {
  const unsigned grid = (unsigned)cdiv(a.vocab, kFewRows);
  const int nt = few_tiles(a.tokens);
  if (f32) {
    if (nt == 1) DMUON_LAUNCH(PH_CE_LOGITS, stream, (k_ce_few<float, 1, 2>), grid, kThreads, 0, a);
    if (nt == 2) DMUON_LAUNCH(PH_CE_LOGITS, stream, (k_ce_few<float, 2, 2>), grid, kThreads, 0, a);
    DMUON_LAUNCH(PH_CE_LOGITS, stream, (k_ce_few<float, 4, 2>), grid, kThreads, 0, a);
  }
  if (nt == 1) DMUON_LAUNCH(PH_CE_LOGITS, stream, (k_ce_few<uint16_t, 1, 8>), grid, kThreads, 0, a);
  DMUON_LAUNCH(PH_CE_LOGITS, stream, (k_ce_few<uint16_t, 2, 8>), grid, kThreads, 0, a);
}
int launch_ce_rows(const CeRowsArgs& a, void* stream) {
  if (a.tokens <= kFewTokens) DMUON_LAUNCH(PH_CE_ROWS, stream, k_ce_rows<4>, (unsigned)cdiv(a.tokens, 4), kThreads, 0, a);
  DMUON_LAUNCH(PH_CE_ROWS, stream, k_ce_rows<16>, (unsigned)cdiv(a.tokens, 16), kThreads, 0, a);
}
template <typename S, bool TB>
static int product(const ProductArgs& a, int phase, void* stream) {
  static std::atomic<uint64_t> ready{0};
  const int e = raise_lds((const void*)k_product<S, TB>, S::Lds, ready);
  if (e) return e;
  DMUON_LAUNCH(phase, stream, (k_product<S, TB>), (unsigned)(a.tiles_r * a.tiles_c * a.groups * a.splits), S::Threads, S::Lds, a);
}
int launch_product(const ProductArgs& a, int phase, void* stream) {
  if (a.tile == Large::M) return a.b_rows ? product<Large, false>(a, phase, stream) : product<Large, true>(a, phase, stream);
  return a.b_rows ? product<Small, false>(a, phase, stream) : product<Small, true>(a, phase, stream);
}
int launch_join(const JoinArgs& a, int phase, void* stream) {
  DMUON_LAUNCH(phase, stream, k_join, stride_grid(a.rows * cdiv(a.cols, 8)), kThreads, 0, a);
}
template <typename T>
static int embed_rows(const EmbedArgs& a, void* stream) {
  const unsigned grid = stride_grid(a.tokens * cdiv(a.width, a.unit));
  if (a.unit == 8) DMUON_LAUNCH(PH_EMBED, stream, k_embed<T>, grid, kThreads, 0, a);
  if (a.unit == 4) DMUON_LAUNCH(PH_EMBED, stream, (k_embed_units<T, 4>), grid, kThreads, 0, a);
  if (a.unit == 2) DMUON_LAUNCH(PH_EMBED, stream, (k_embed_units<T, 2>), grid, kThreads, 0, a);
  DMUON_LAUNCH(PH_EMBED, stream, (k_embed_units<T, 1>), grid, kThreads, 0, a);
}
int launch_embed(const EmbedArgs& a, void* stream) {
  return a.f32 ? embed_rows<float>(a, stream) : embed_rows<uint16_t>(a, stream);
}
int launch_sort_runs(const SortArgs& a, void* stream) {
  const dim3 grid((unsigned)cdiv(a.tokens, kSortRun)), block(kScanThreads);
  hipStream_t st = (hipStream_t)stream;
  timing_before(PH_EMBED_GRAD, stream);
  if (a.tokens <= kScanThreads) hipLaunchKernelGGL(k_sort_block<1>, grid, block, 0, st, a);
  else if (a.tokens <= 4 * kScanThreads) hipLaunchKernelGGL(k_sort_block<4>, grid, block, 0, st, a);
  else hipLaunchKernelGGL(k_sort_block<kSortRun / kScanThreads>, grid, block, 0, st, a);
  if (a.tokens > kSortRun) hipLaunchKernelGGL(k_sort_merge, dim3((unsigned)cdiv(a.tokens, kThreads)), dim3(kThreads), 0, st, a);
  const int e = (int)hipGetLastError();
  timing_after(PH_EMBED_GRAD, stream);
  return e;
}
int launch_sort_pass(const SortArgs& a, void* stream) {
  timing_before(PH_EMBED_GRAD, stream);
  hipLaunchKernelGGL(k_sort_count, dim3(a.blocks), dim3(kThreads), 0, (hipStream_t)stream, a);
  hipLaunchKernelGGL(k_sort_scan, dim3(1), dim3(kScanThreads), 0, (hipStream_t)stream, a);
  hipLaunchKernelGGL(k_sort_place, dim3(a.blocks), dim3(kThreads), 0, (hipStream_t)stream, a);
  const int e = (int)hipGetLastError();
  timing_after(PH_EMBED_GRAD, stream);
  return e;
}
int launch_embed_run(const EmbedGradArgs& a, int level, void* stream) {
  const dim3 grid((unsigned)(a.tokens / (level == 0 ? kRun : kRun * kRun)), (unsigned)cdiv(a.width, 512));
  if (level == 1) DMUON_LAUNCH(PH_EMBED_GRAD, stream, (k_embed_run<float, 1>), grid, kThreads, 0, a);
  if (a.grad_f32) DMUON_LAUNCH(PH_EMBED_GRAD, stream, (k_embed_run<float, 0>), grid, kThreads, 0, a);
  DMUON_LAUNCH(PH_EMBED_GRAD, stream, (k_embed_run<uint16_t, 0>), grid, kThreads, 0, a);
}
int launch_embed_grad(const EmbedGradArgs& a, void* stream) {
  const unsigned grid = (unsigned)(a.seg_wg + (a.accumulate ? 0 : cdiv(a.rows, a.zero_rows)));
  if (a.grad_f32) {
    if (a.out_f32) DMUON_LAUNCH(PH_EMBED_GRAD, stream, (k_embed_grad<float, float>), grid, kThreads, 0, a);
    DMUON_LAUNCH(PH_EMBED_GRAD, stream, (k_embed_grad<float, uint16_t>), grid, kThreads, 0, a);
  }
  if (a.out_f32) DMUON_LAUNCH(PH_EMBED_GRAD, stream, (k_embed_grad<uint16_t, float>), grid, kThreads, 0, a);
  DMUON_LAUNCH(PH_EMBED_GRAD, stream, (k_embed_grad<uint16_t, uint16_t>), grid, kThreads, 0, a);
}
int launch_ckpt_quantize(const CodecArgs& a, void* stream) {
  const unsigned grid = stride_grid(a.rows * a.blocks * 4);
  if (a.f32) DMUON_LAUNCH(PH_CKPT_CODEC, stream, k_ckpt_quantize<float>, grid, kThreads, 0, a);
  DMUON_LAUNCH(PH_CKPT_CODEC, stream, k_ckpt_quantize<uint16_t>, grid, kThreads, 0, a);
}
int launch_ckpt_read(const CodecArgs& a, int phase, void* stream) {
  const unsigned grid = stride_grid(a.rows * cdiv(a.cols, 8));
  if (phase == PH_CKPT_WGRAD) DMUON_LAUNCH(phase, stream, (k_ckpt_read<uint16_t, false>), grid, kThreads, 0, a);   // an operand copy
  if (a.f32) DMUON_LAUNCH(phase, stream, (k_ckpt_read<float, true>), grid, kThreads, 0, a);
  DMUON_LAUNCH(phase, stream, (k_ckpt_read<uint16_t, true>), grid, kThreads, 0, a);
}

}  // namespace dmuon
