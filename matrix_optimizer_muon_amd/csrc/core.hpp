// Device code shared by the HIP sources for gfx950 (MI355X): small conversions,
// range-checked buffer access, and the step's matrix-core contraction core with its
// tile orders, parts of which the training gradients' cores use too.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>
#include <utility>

#include "internal.hpp"

namespace dmuon {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef short v4i16_t __attribute__((ext_vector_type(4)));

// Global-memory (address space 1) view of a pointer.  Pointers read out of the
// device-side problem table are generic to the compiler, which would otherwise
// emit flat accesses (counted on both vmcnt and lgkmcnt, hence coarse waits).
template <typename T> using gptr = __attribute__((address_space(1))) T*;
template <typename T> __device__ __forceinline__ gptr<T> glob(T* p) { return (gptr<T>)p; }

// ---------------------------------------------------------------------------
// small helpers
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  // v_cvt_pk_bf16_f32: round to nearest even, NaN stays NaN
  const __bf16 b = (__bf16)f;
  uint16_t u;
  __builtin_memcpy(&u, &b, 2);
  return u;
}
__device__ __forceinline__ float bf16_to_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// bf16 pair (lo, hi) packed into one dword, round to nearest even
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  const bf16x2_t b = __builtin_convertvector(v, bf16x2_t);
  uint32_t u;
  __builtin_memcpy(&u, &b, 4);
  return u;
}

// Buffer resource over [p, p + bytes) (a null p gives an empty range).  Buffer
// accesses are range checked: a load beyond the range reads zero and a store
// beyond it is dropped, which replaces per-element predicates (and the branches
// they would need) in the apply epilogue.
constexpr unsigned kOob = 0x7ffffff0u;       // an offset beyond every range used here
// Word 3 of a buffer descriptor: data format 32 (bits 15–18 = 4), which raw
// (untyped) buffer accesses need to be non-zero; no swizzle, no index stride.
constexpr int kRsrcFlags = 0x00020000;
// The fields are workgroup-uniform; readfirstlane tells the compiler so (a
// descriptor it cannot prove uniform is rebuilt per lane in a loop).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t range_rsrc(const void* p, int64_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)a);
  const unsigned hi = __builtin_amdgcn_readfirstlane((unsigned)(a >> 32));
  const int n = __builtin_amdgcn_readfirstlane(p ? (int)bytes : 0);
  return __builtin_amdgcn_make_buffer_rsrc((void*)(((uint64_t)hi << 32) | lo), 0, n, kRsrcFlags);
}
__device__ __forceinline__ float buf_ld(__amdgpu_buffer_rsrc_t r, unsigned off) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
}
__device__ __forceinline__ void buf_st(__amdgpu_buffer_rsrc_t r, unsigned off, float v) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, (int)off, 0, 0);
}
__device__ __forceinline__ void buf_st(__amdgpu_buffer_rsrc_t r, unsigned off, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b32(v, r, (int)off, 0, 0);
}

// ---------------------------------------------------------------------------
// Contraction core on the matrix cores: C[i][j] = Σ_k A(i, k)·B(j, k).
//
// One workgroup = 8 wave64s (two per SIMD) computing a 256×256 output tile; each
// wave owns a 128×64 sub-tile (4×2 blocks of 32×32 fp32 accumulators; on the bf16
// path each block is computed as four 16×16×32 quarters, see mfma_quarter).  K is staged
// through LDS in 64-byte rows (32 bf16 or 16 fp32 per row and stage), four stages
// deep, filled by buffer_load … lds (global → LDS without VGPRs; rows beyond the
// operand read as zero through the buffer's range check).  The four 16-byte
// chunks of a row are XOR-swizzled with (row >> 2) & 3 so that 16 consecutive
// rows read at one logical chunk cover all 64 LDS banks.
//
// An operand is read either row-major ("NT": row i holds A(i, 0..K), staged as
// 256 rows of 64 bytes) or K-major (row k holds A(0..255, k) of the tile,
// staged as 32 rows of 512 bytes, bf16 only).  A K-major stage is filled with
// whole 512-byte row segments, so each DMA instruction moves 8 full cache lines
// (the NT stage moves 16 half lines); its MFMA fragments are read with the
// transposing ds_read_b64_tr_b16 (two 8-byte reads per 16-byte fragment).  Its
// 32-byte segments are XOR-swizzled by kmaj_swz(row), which spreads the rows and
// segments one half-wave of a fragment read touches over all 64 banks.  A K-major B operand
// made plain 2048- to 8192-sized products 5–16% faster than NT; with both
// operands K-major (twice the fragment reads) it is about even.  On the bf16
// path X is kept only in storage layout, so the apply reads X (wide) or the
// symmetric B′ (tall) K-major and the tall Gram reads both operands K-major; the
// square stays NT (measured faster there).
//
// Ping-pong schedule: the two waves sharing a SIMD belong to different groups
// (group = wave >> 2, the 128-row half of the tile they own), and the groups run
// one phase apart.  A phase is either an MFMA phase (the MFMAs on the fragments
// of one stage: 32 of 16×16×32 on bf16, 64 of 32×32×2 on fp32) or a memory
// phase (wait for the stage's DMA, read all of its fragments, issue the DMA of
// the stage three ahead); a workgroup barrier ends every phase.  While one group's waves keep the matrix cores busy, the other
// group's waves move data, so no barrier drains the MFMA pipeline.
// ---------------------------------------------------------------------------
constexpr int kGemmWaves = 8;
constexpr int kGemmThreads = 64 * kGemmWaves;
constexpr int kRowBytes = 64;                          // staged bytes per operand row
constexpr int kStageBytes = 2 * kTile * kRowBytes;     // A rows + B rows: 32 KiB
constexpr int kStages = 4;
constexpr int kGemmLds = kStages * kStageBytes;        // 128 KiB
constexpr int kDmaPerStage = 4;                        // buffer_load … lds per thread per stage
static_assert(kTile == 256 && kGemmWaves == 8, "fragment layout assumes 8 waves on a 256 tile");

struct Operands {
  const char* a;     // NT: first A row of the tile; K-major: start of k-row 0
  const char* b;     // NT: first B row of the tile; K-major: start of k-row 0
  int lda_b;         // leading dims in bytes (multiples of 128)
  int ldb_b;
  int rows_a;        // NT: valid rows from the tile start; K-major: valid k rows
  int rows_b;
  int cola_b;        // K-major: byte offset of the tile's first column in a k-row
  int colb_b;
  int ktiles;        // stages: K elements / 32 (bf16) or / 16 (fp32)
};

// K-major stage layout: 32-byte segment s of k-row r sits at segment s ^ kmaj_swz(r).
// A transposing fragment read has 16-lane groups read four consecutive k-rows of
// one 16-column segment, the two groups of a half-wave k-rows 8 apart: bits 0-1
// of r spread a group's rows over four segment pairs and bit 3 moves the other
// group's rows to the odd segments, so a half-wave touches 8 distinct segments.
__device__ __forceinline__ int kmaj_swz(int r) { return (2 * (r & 3)) ^ ((r >> 3) & 1); }

// f(std::integral_constant<int, 0>{}) … f(std::integral_constant<int, N − 1>{})
template <typename F, int... I>
__device__ __forceinline__ void static_for_seq(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_seq(f, std::make_integer_sequence<int, N>{});
}

// bf16 contraction step on one 16×16 quarter of a 32×32 accumulator block.
// During the K loop quarter (R, C) (rows 16R.., columns 16C.. of the block) lives
// in registers 4(2R + C) .. 4(2R + C) + 3 in the 16×16×32 output layout: lane l,
// register i holds row 4(l >> 4) + i, column l & 15.  The operands: lane l holds
// row (A) or column (B) l & 15 and k = 8(l >> 4) .. 8(l >> 4) + 7 of the 32-deep
// stage.  quarters_to_32x32 turns the block into the 32×32×16 output layout the
// epilogues read (acc_row / acc_col).
template <int Q>
__device__ __forceinline__ void mfma_quarter(f32x16_t& acc, const u32x4_t& a, const u32x4_t& b) {
  bf16x8_t va, vb;
  __builtin_memcpy(&va, &a, 16);
  __builtin_memcpy(&vb, &b, 16);
  f32x4_t q = {acc[4 * Q], acc[4 * Q + 1], acc[4 * Q + 2], acc[4 * Q + 3]};
  q = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, vb, q, 0, 0, 0);
  acc[4 * Q] = q[0];
  acc[4 * Q + 1] = q[1];
  acc[4 * Q + 2] = q[2];
  acc[4 * Q + 3] = q[3];
}

// Quarter layout → 32×32×16 layout, in place.  In the 32×32 layout lane l,
// register 4g + i holds row 8g + 4(l >> 5) + i, column l & 31; that value sits in
// quarter (g >> 1, (l >> 4) & 1) at lane 32(g & 1) + 16(l >> 5) + (l & 15),
// register i.  Per register pair (quarters (R, 0) and (R, 1)) this is a swap of
// lane bit 4 with the pair index followed by a swap of lane bit 5 with it:
// v_permlane16_swap then v_permlane32_swap.
__device__ __forceinline__ void quarters_to_32x32(f32x16_t& acc) {
#pragma unroll
  for (int R = 0; R < 2; ++R)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto s16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[8 * R + i]),
                                                        __float_as_uint(acc[8 * R + 4 + i]), false, false);
      const auto s32 = __builtin_amdgcn_permlane32_swap(s16[0], s16[1], false, false);
      acc[8 * R + i] = __uint_as_float(s32[0]);
      acc[8 * R + 4 + i] = __uint_as_float(s32[1]);
    }
}

// fp32 contraction step on one 32×32 block: a 16-byte chunk holds 4 consecutive
// k; element e of the two lane halves forms one K = 2 step.  A and B use the same
// k permutation, so the sum covers the same products.
__device__ __forceinline__ void mfma_chunk_f32(f32x16_t& acc, const u32x4_t& a, const u32x4_t& b) {
  acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), acc, 0, 0, 0);
  acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), acc, 0, 0, 0);
}

// s_waitcnt with only vmcnt constrained (expcnt 7, lgkmcnt 15 = no wait)
#define DMUON_WAIT_VM(n) __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xF << 8) | ((n) & 15) | ((((n) >> 4) & 3) << 14))

// s_waitcnt with only lgkmcnt constrained to 0 (vmcnt 63, expcnt 7 = no wait)
#define DMUON_WAIT_LGKM0() __builtin_amdgcn_s_waitcnt(0xF | (0x3 << 14) | (0x7 << 4))

// The apply's α·X term on the matrix cores (bf16 path).  X enters the apply's
// contraction as its bf16 operand copy hi; α·hi is α·I times that operand, so
// in the K stages that cover the tile's own rows (wide: the diagonal block of
// the B′ operand) or columns (tall: of the B′ operand on the B side) each wave
// issues extra MFMAs against a diagonal fragment built in registers.  α is split
// into two bf16 values α1 = bf16(α), α2 = bf16(α − α1), so α1·hi + α2·hi is
// α·hi to about 2⁻¹⁷ relative; the products are exact and accumulate in fp32.
struct DiagTerm {
  int kd0;           // first K stage of the tile's diagonal block
  uint32_t a1, a2;   // bf16 bit patterns of α1, α2
};

template <typename T, bool TA = false, bool TB = false, int DIAG = 0>
__device__ __forceinline__ void gemm_mainloop(const Operands& op, char* smem, f32x16_t (&acc)[4][2],
                                              const DiagTerm& dg = DiagTerm{0, 0u, 0u}) {
  static_assert(!(TA || TB) || sizeof(T) == 2, "K-major operands are bf16");
  static_assert(DIAG == 0 || sizeof(T) == 2, "the diagonal term is for bf16 operands");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);    // wave-uniform
  const int wr = wave >> 2, wc = wave & 3, h = lane >> 5, r32 = lane & 31;
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      (void*)op.a, 0, (op.rows_a < kTile ? op.rows_a : kTile) * op.lda_b, kRsrcFlags);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      (void*)op.b, 0, (op.rows_b < kTile ? op.rows_b : kTile) * op.ldb_b, kRsrcFlags);
  // DMA: wave w fills rows [32w, 32w + 32) of A and of B, 16 rows per instruction;
  // lane l lands at byte 16·l of the instruction's 1 KiB = row l/4, physical chunk l%4.
  // K-major: the instruction's 1 KiB is k-rows 2(2w + q) and 2(2w + q) + 1; lane l
  // lands in k-row l/32 at physical 16-byte unit l%32.
  int offa[2], offb[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int row = (wave * 2 + q) * 16 + (lane >> 2);
    const int c = (lane & 3) ^ ((row >> 2) & 3);
    const int kr = 2 * (wave * 2 + q) + (lane >> 5), un = lane & 31;
    const int lun = (((un >> 1) ^ kmaj_swz(kr)) << 1) | (un & 1);    // logical unit
    offa[q] = TA ? kr * op.lda_b + op.cola_b + lun * 16 : row * op.lda_b + c * 16;
    offb[q] = TB ? kr * op.ldb_b + op.colb_b + lun * 16 : row * op.ldb_b + c * 16;
  }
  // Fragments of one stage.  bf16 (16×16×32 quarters): fa[ss][i] is rows
  // 16(4ss + i) .. +15 of the wave's 128 and fb[ss][j] columns 16(2ss + j) .. +15
  // of its 64, all 32 k, lane l reading logical chunk l >> 4 of row l & 15.
  // fp32 (32×32×2): fa[ss][i] / fb[ss][j] are 32-row / 32-column blocks i / j and
  // 16-k chunk ss, lane l reading logical chunk 2·ss + (l >> 5) of row l & 31.
  constexpr bool kQ = sizeof(T) == 2;
  int fa_off[2][4], fb_off[2][2];
#pragma unroll
  for (int ss = 0; ss < 2; ++ss) {
    const int c = kQ ? lane >> 4 : 2 * ss + h;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = kQ ? wr * 128 + 16 * (4 * ss + i) + (lane & 15) : wr * 128 + i * 32 + r32;
      fa_off[ss][i] = row * kRowBytes + ((c ^ ((row >> 2) & 3)) * 16);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = kQ ? wc * 64 + 16 * (2 * ss + j) + (lane & 15) : wc * 64 + j * 32 + r32;
      fb_off[ss][j] = kTile * kRowBytes + row * kRowBytes + ((c ^ ((row >> 2) & 3)) * 16);
    }
  }
  // K-major fragments (bf16, quarter layout): two transposing 8-byte reads (k
  // 0..3 and 4..7 of the lane's 8-k block 8(l >> 4)); in each 16-lane group,
  // source lane i reads k-row 8(l >> 4) + 4t + (i >> 2), columns 4(i & 3) .. +3 of
  // the quarter's 16 columns, and lane i receives column i of the quarter, four
  // consecutive k
  int ta_off[TA ? 2 : 1][4][2], tb_off[TB ? 2 : 1][2][2];
#pragma unroll
  for (int ss = 0; ss < 2; ++ss)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int kr = 8 * (lane >> 4) + 4 * t + ((lane & 15) >> 2);
      const int sub = 4 * (lane & 3);
      if (TA) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = wr * 128 + 16 * (4 * ss + i) + sub;
          ta_off[TA ? ss : 0][i][t] = kr * 512 + (((n >> 4) ^ kmaj_swz(kr)) << 5) + ((2 * n) & 31);
        }
      }
      if (TB) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int n = wc * 64 + 16 * (2 * ss + j) + sub;
          tb_off[TB ? ss : 0][j][t] = kTile * kRowBytes + kr * 512 + (((n >> 4) ^ kmaj_swz(kr)) << 5) + ((2 * n) & 31);
        }
      }
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  u32x4_t fa[2][4], fb[2][2];     // all fragments of one stage
  // K-major operands take a range per stage: exactly its 32 k-rows (fewer at the
  // K tail, whose missing rows read as zero), so byte offsets stay small for any
  // K and no read leaves the operand.  Reads past a row's end (tile columns past
  // the leading dim) see the next row or zero; they feed only output columns
  // past the matrix, which the epilogues drop.
  auto kmaj_rsrc = [&](const char* p, int ld_b, int rows, int kt) {
    const int left = rows - 32 * kt;
    return range_rsrc(p + (int64_t)kt * 32 * ld_b, (int64_t)(left < 0 ? 0 : (left < 32 ? left : 32)) * ld_b);
  };
  auto issue = [&](int kt) {
    char* base = smem + (kt % kStages) * kStageBytes;
    const __amdgpu_buffer_rsrc_t sa = TA ? kmaj_rsrc(op.a, op.lda_b, op.rows_a, kt) : ra;
    const __amdgpu_buffer_rsrc_t sb = TB ? kmaj_rsrc(op.b, op.ldb_b, op.rows_b, kt) : rb;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      char* da = base + (wave * 2 + q) * 16 * kRowBytes;
      char* db = da + kTile * kRowBytes;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sa, (__attribute__((address_space(3))) void*)da, 16,
                                               offa[q] + (TA ? 0 : kt * kRowBytes), 0, 0, 0);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(sb, (__attribute__((address_space(3))) void*)db, 16,
                                               offb[q] + (TB ? 0 : kt * kRowBytes), 0, 0, 0);
    }
  };
  const int KT = op.ktiles;        // ≥ 2 (leading dims are multiples of 64 elements)
  const bool lead = wr == 1;       // group 1 runs one phase ahead of group 0

  // Memory phase of stage kt.  Every wave waited for its own share of stage kt
  // in its previous memory phase (or before the first barrier), so each share
  // a wave reads here landed before at least one barrier, like the other
  // group's share.  Here it waits for its share of stage kt + 1; stages up to
  // min(kt + 2, KT − 1) have been issued.
  auto mem_phase = [&](int kt) {
    if (kt + 2 < KT) DMUON_WAIT_VM(kDmaPerStage);
    else DMUON_WAIT_VM(0);
    const char* base = smem + (kt % kStages) * kStageBytes;
    auto tr16 = [&](int off0, int off1) {    // two transposing reads → one 16-byte fragment
      const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)(base + off0));
      const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4i16_t*)(base + off1));
      u32x4_t r;
      r.x = (uint32_t)(uint16_t)lo.x | ((uint32_t)(uint16_t)lo.y << 16);
      r.y = (uint32_t)(uint16_t)lo.z | ((uint32_t)(uint16_t)lo.w << 16);
      r.z = (uint32_t)(uint16_t)hi.x | ((uint32_t)(uint16_t)hi.y << 16);
      r.w = (uint32_t)(uint16_t)hi.z | ((uint32_t)(uint16_t)hi.w << 16);
      return r;
    };
#pragma unroll
    for (int ss = 0; ss < 2; ++ss) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        fa[ss][i] = TA ? tr16(ta_off[TA ? ss : 0][i][0], ta_off[TA ? ss : 0][i][1])
                       : *(const u32x4_t*)(base + fa_off[ss][i]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        fb[ss][j] = TB ? tr16(tb_off[TB ? ss : 0][j][0], tb_off[TB ? ss : 0][j][1])
                       : *(const u32x4_t*)(base + fb_off[ss][j]);
    }
    // the slot of stage kt − 1, read by both groups in earlier phases
    if (kt + kStages - 1 < KT) issue(kt + kStages - 1);
    // fragment reads complete before the barrier that releases this slot
    DMUON_WAIT_LGKM0();
  };
  // diagonal fragment of quarter R (A side: rows 16R .. of the 32-row block the
  // stage's k cover; B side: columns): this lane holds k = 8(l >> 4) + e (e < 8)
  // for row / column 16R + (l & 15); its only nonzero element is e = e0 + 16R
  // with e0 = (l & 15) − 8(l >> 4).
  // e0 passes through an empty asm so that the fragments are built inside the
  // (rarely taken) diagonal branch instead of being hoisted out of the K loop,
  // where they would hold registers for the whole contraction.
  auto diag_frag = [&](int e, uint32_t bits) {
    const uint32_t v = (e & 1) ? bits << 16 : bits;
    u32x4_t f;
    f.x = (unsigned)e < 2u ? v : 0u;
    f.y = (unsigned)(e - 2) < 2u ? v : 0u;
    f.z = (unsigned)(e - 4) < 2u ? v : 0u;
    f.w = (unsigned)(e - 6) < 2u ? v : 0u;
    return f;
  };
  auto mfma_phase = [&]() {
    __builtin_amdgcn_s_setprio(1);
    if constexpr (kQ) {
      // quarter (s, t): rows 16s of the wave's 128, columns 16t of its 64
      static_for<8>([&](auto S) {
        constexpr int qs = decltype(S)::value;
        static_for<4>([&](auto Tq) {
          constexpr int qt = decltype(Tq)::value;
          mfma_quarter<2 * (qs & 1) + (qt & 1)>(acc[qs >> 1][qt >> 1], fa[qs >> 2][qs & 3], fb[qt >> 1][qt & 1]);
        });
      });
    } else {
#pragma unroll
      for (int ss = 0; ss < 2; ++ss)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) mfma_chunk_f32(acc[i][j], fa[ss][i], fb[ss][j]);
    }
    __builtin_amdgcn_s_setprio(0);
  };
  // the extra MFMAs of a diagonal stage: block I of the wave's rows (A side) or
  // columns (B side)
  auto diag_phase = [&](auto I) {
    constexpr int b = decltype(I)::value;
    int e0 = (lane & 15) - 8 * (lane >> 4);
    asm volatile("" : "+v"(e0));
    __builtin_amdgcn_s_setprio(1);
    static_for<2>([&](auto Rq) {
      constexpr int R = decltype(Rq)::value;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const u32x4_t df = diag_frag(e0 + 16 * R, p ? dg.a2 : dg.a1);
        if constexpr (DIAG == 1) {
          // rows of quarter row R of block b against every column quarter
          static_for<4>([&](auto Tq) {
            constexpr int qt = decltype(Tq)::value;
            mfma_quarter<2 * R + (qt & 1)>(acc[b][qt >> 1], df, fb[qt >> 1][qt & 1]);
          });
        } else {
          // columns of quarter column R of block b against every row quarter
          static_for<8>([&](auto S) {
            constexpr int qs = decltype(S)::value;
            mfma_quarter<2 * (qs & 1) + R>(acc[qs >> 1][b], fa[qs >> 2][qs & 3], df);
          });
        }
      }
    });
    __builtin_amdgcn_s_setprio(0);
  };

  const int pro = KT < kStages - 1 ? KT : kStages - 1;
  for (int st = 0; st < pro; ++st) issue(st);
  if (pro == 3) DMUON_WAIT_VM(2 * kDmaPerStage);      // own share of stage 0
  else if (pro == 2) DMUON_WAIT_VM(kDmaPerStage);
  else DMUON_WAIT_VM(0);
  __builtin_amdgcn_s_barrier();
  if (!lead) __builtin_amdgcn_s_barrier();             // trailing group: one phase late
  __builtin_amdgcn_sched_barrier(0);
  auto step = [&](int kt) {
    mem_phase(kt);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    mfma_phase();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  if constexpr (DIAG == 0) {
#pragma unroll 1
    for (int kt = 0; kt < KT; ++kt) step(kt);
  } else {
    // every wave runs KT steps with the same barriers; its diagonal stages
    // [kb, kb + nb) (wide: its 4 row blocks, tall: its 2 column blocks) are
    // unrolled so that each names its accumulator block at compile time
    constexpr int nb = DIAG == 1 ? 4 : 2;
    const int kb = dg.kd0 + (DIAG == 1 ? 4 * wr : 2 * wc);
    const int k1 = kb < KT ? kb : KT;
#pragma unroll 1
    for (int kt = 0; kt < k1; ++kt) step(kt);
    auto dstep = [&](auto I) {
      const int kt = kb + decltype(I)::value;
      if (kt >= KT) return;
      mem_phase(kt);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      mfma_phase();
      diag_phase(I);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
    };
    dstep(std::integral_constant<int, 0>{});
    dstep(std::integral_constant<int, 1>{});
    if constexpr (nb == 4) {
      dstep(std::integral_constant<int, 2>{});
      dstep(std::integral_constant<int, 3>{});
    }
#pragma unroll 1
    for (int kt = kb + nb < KT ? kb + nb : KT; kt < KT; ++kt) step(kt);
  }
  if (lead) __builtin_amdgcn_s_barrier();              // every wave passes 2·KT + 2 barriers
  if constexpr (kQ) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) quarters_to_32x32(acc[i][j]);
  }
  // all LDS reads done before the caller reuses LDS
  __syncthreads();
}

// Position of accumulator register r of block (i, j) inside the 256×256 tile.
__device__ __forceinline__ int acc_row(int i, int rq) {   // rq = r >> 2; rows rq·8 + h·4 + 0..3
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  return (wave >> 2) * 128 + i * 32 + rq * 8 + (lane >> 5) * 4;
}
__device__ __forceinline__ int acc_col(int j) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  return (wave & 3) * 64 + j * 32 + (lane & 31);
}

// Tile orders.  Consecutive logical tiles run on one XCD in runs of 16 or 64 (see
// xcd_logical_block), so the order decides how many operand panels one XCD's L2
// has to hold at once.  Both orders walk bands of tiles along one side of the
// output and advance the other side every band height, so the 32 apply tiles
// one XCD runs at once cover about 8 × 4 tiles and touch ~12 panels (a
// row-by-row order touched ~33: for an 8192 × 28672 matrix, all 32 panels of B'
// per XCD and round).  The Gram and the square, in runs of 16, walk bands of 4:
// a run covers about 4 × 4 tiles (8 panels, against 10 for 8 × 2).
constexpr int kBand = 8;
constexpr int kTriBand = 4;

// apply: R tiles along the short side, C along the long one; returns the
// short-side and long-side tile indices of logical tile u
__device__ __forceinline__ void band_tile(int u, int R, int C, int& ts, int& tl) {
  const int b = u / (kBand * C);
  const int r0 = b * kBand;
  const int gb = R - r0 < kBand ? R - r0 : kBand;
  const int v = u - b * kBand * C;
  ts = r0 + v % gb;
  tl = v / gb;
}

// Gram / square: upper-triangle tile u (ti ≤ tj) of a T×T grid.  Band b holds
// rows [BAND·b, BAND·b + h): first its triangle (tj from BAND·b to BAND·b + h − 1,
// each with the rows up to tj), then h rows for every later tj.
template <int BAND>
__device__ __forceinline__ void tri_tile(int u, int T, int& ti, int& tj) {
  int r0 = 0, start = 0;
  for (;;) {
    const int h = T - r0 < BAND ? T - r0 : BAND;
    const int n = h * (h + 1) / 2 + h * (T - r0 - h);
    if (u < start + n) {
      int v = u - start;
      const int tri = h * (h + 1) / 2;
      if (v < tri) {
        int k = 0;
        while ((k + 1) * (k + 2) / 2 <= v) ++k;
        ti = r0 + (v - k * (k + 1) / 2);
        tj = r0 + k;
      } else {
        v -= tri;
        ti = r0 + v % h;
        tj = r0 + h + v / h;
      }
      return;
    }
    start += n;
    r0 += BAND;
  }
}

// Logical workgroup index.  Workgroups are handed to the 8 XCDs round-robin in
// launch order, so workgroup b runs on XCD b % 8 as its (b / 8)-th workgroup.
// The logical tile list is consumed in windows of 8·RUN tiles: inside a window
// each XCD takes RUN consecutive tiles (neighbours share operand panels in that
// XCD's L2), and all XCDs advance through the list together, so tiles of
// unequal cost (long-K problems first) are spread over every XCD.  A last
// partial window of R tiles is split the same way into 8 contiguous runs (the
// first R % 8 XCDs take one tile more).  The map is a bijection on [0, G).
// Runs of 64 suit the apply (two rounds of 8 × 4 tiles per XCD); the Gram and
// the square (triangle tiles in bands of 4) measured faster with runs of 16.
template <int RUN>
__device__ __forceinline__ int xcd_logical_block() {
  const int G = gridDim.x, b = blockIdx.x;
  constexpr int win = 8 * RUN;
  const int w = b / win;
  const int xcd = b & 7, slot = (b >> 3) - w * RUN;
  if ((w + 1) * win <= G) return w * win + xcd * RUN + slot;
  const int R = G - w * win, per = R >> 3, rem = R & 7;
  return w * win + (xcd < rem ? xcd * (per + 1) : rem * (per + 1) + (xcd - rem) * per) + slot;
}

}  // namespace dmuon
