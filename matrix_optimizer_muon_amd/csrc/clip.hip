// HIP kernels of the global norm over many gradients and of clipping by it, for gfx950
// (MI355X).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "clip.hpp"
#include "core.hpp"
#include "elements.hpp"

namespace dmuon {

// ---------------------------------------------------------------------------
// the list of tensors, in chunks of 8192 elements: workgroup b takes the chunks b,
// b + groups, …, so that all of them work in one moving window of memory (contiguous ranges
// per workgroup, 2048 places at once: 1122 M bf16 elements clipped 1176 µs, so 1140), and looks a
// chunk's tensor up with a search of 64 probes a step when the last one is passed.
// f(problem, first element, end).
// ---------------------------------------------------------------------------
__device__ __forceinline__ int first_problem(const ClipTable& tab, int chunk) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = tab.n;                                 // the last p with chunk0[p] ≤ chunk lies in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 63) >> 6;
    const int i = lane * step;
    const bool in = i < n && tab.chunk0[lo + i] <= chunk;
    const int k = (__popcll(__ballot(in)) - 1) * step;
    lo += k;
    n = n - k < step ? n - k : step;
  }
  return lo;
}

// false: the workspace holds another table
template <typename F>
__device__ __forceinline__ bool walk(const ClipTable& tab, F f) {
  if (tab.probs[0].tag != tab.tag) return false;
  int p = 0, base = 0, next = 0;
  for (int c = blockIdx.x; c < tab.chunks; c += tab.groups) {
    if (c >= next) {
      p = first_problem(tab, c);
      base = tab.chunk0[p];
      next = tab.chunk0[p + 1];
    }
    const ClipProblem& P = tab.probs[p];
    if (P.tag != tab.tag) return false;
    const int64_t e0 = (int64_t)(c - base) * kClipChunk;
    f(P, e0, e0 + kClipChunk < P.numel ? e0 + kClipChunk : P.numel);
  }
  return true;
}

// ---------------------------------------------------------------------------
// sums of squares in 64 bits: a square of an fp32 value is exact there, nothing overflows or
// vanishes, and the order is fixed.  Memory bound: 1045 M bf16 elements in 351 µs, 5.95 TB/s.
// ---------------------------------------------------------------------------
__device__ __forceinline__ double sum_workgroup(double v, double* shared) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
  __syncthreads();
  return (shared[0] + shared[1]) + (shared[2] + shared[3]);
}

// one chunk: a thread's units of 16 bytes 256 apart, so that every access of a wave is whole
// lines (fp32 units of 8 elements, two accesses of each: 5 × 200 M clipped in 2351 µs, so
// 2062), 4 loads in flight (8: 78 registers for 50, and bf16 5% slower), and at a tensor's
// end at most 7 elements.  ONCE: nontemporal, for the last reading of the data; the sums'
// loads leave what fits in the caches for the scaling (29 × 16 Mi bf16: 482 µs, with
// nontemporal loads in both 483, in neither 553; 7 × 11 Mi: 75, 83 and 77).
template <bool ONCE, typename T, typename F, typename G>
__device__ __forceinline__ void chunk(gptr<const T> p, int n, F unit, G single) {
  constexpr int W = 16 / sizeof(T), B = 4;
  const int units = n / W;
#pragma unroll 1
  for (int h = 0; h < kClipChunk / (B * W * kThreads); ++h) {
    const int j0 = threadIdx.x + h * (B * kThreads);
    Unit<T, W> x[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int j = j0 + k * kThreads;
      if (j < units) {
        if (ONCE) x[k].load_once(p + j * W);
        else x[k].load(p + j * W);
      }
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int j = j0 + k * kThreads;
      if (j >= units) break;
      float v[W];
      x[k].values(v);
      unit(j * W, v);
    }
  }
  const int e = units * W + threadIdx.x;
  if (e < n) single(e, element(p + e));
}

template <typename T>
__device__ __forceinline__ void add_squares(gptr<const T> p, int64_t e0, int64_t e1, double (&sum)[2]) {
  chunk<false>(p + e0, (int)(e1 - e0),
        [&](int, const auto& v) {
#pragma unroll
          for (int e = 0; e < 16 / (int)sizeof(T); ++e) sum[e & 1] = fma((double)v[e], (double)v[e], sum[e & 1]);
        },
        [&](int, float v) { sum[0] = fma((double)v, (double)v, sum[0]); });
}

__global__ __launch_bounds__(kThreads) void k_grad_norm(ClipTable tab) {
  __shared__ double shared[kThreads / 64];
  double sum[2] = {0.0, 0.0};
  const bool ok = walk(tab, [&](const ClipProblem& P, int64_t e0, int64_t e1) {
    if (P.f32) add_squares(glob((const float*)P.grad), e0, e1, sum);
    else add_squares(glob((const uint16_t*)P.grad), e0, e1, sum);
  });
  const double all = sum_workgroup(sum[0] + sum[1], shared);
  if (ok && threadIdx.x == 0) tab.part[blockIdx.x] = all;
}

// the norm of all partial sums, the same bits wherever it is computed
__device__ __forceinline__ float joined_norm(const ClipTable& tab, double* shared) {
  double v[kClipGroups / kThreads];
#pragma unroll
  for (int k = 0; k < kClipGroups / kThreads; ++k) {
    const int i = threadIdx.x + k * kThreads;
    v[k] = i < tab.groups ? tab.part[i] : 0.0;
  }
  double sum = 0.0;
#pragma unroll
  for (int k = 0; k < kClipGroups / kThreads; ++k) sum += v[k];
  return (float)sqrt(sum_workgroup(sum, shared));
}

__global__ __launch_bounds__(kThreads) void k_grad_norm_join(ClipTable tab, float* norm) {
  __shared__ double shared[kThreads / 64];
  if (tab.n > 0 && tab.probs[0].tag != tab.tag) return;  // no tensors: 0
  const float n = joined_norm(tab, shared);
  if (threadIdx.x == 0) *norm = n;
}

// ---------------------------------------------------------------------------
// out = c·g, c = min(1, max_norm/(norm + eps)), 1 where the norm is not finite: one
// rounding to fp32 and one to the output's type.  Where c lies below fp32's normal numbers it
// is a fraction and a power of 2 that follows the product, so that gradients near fp32's end
// keep their digits (an instruction per element; no time, it passes behind the loads).  Every
// workgroup joins the partial sums for itself (16 KiB from the caches) instead of waiting for
// another launch.  In place nothing is written where c is 1.  Memory bound: what exceeds the
// caches is read twice (1045 M bf16 elements: 706 µs, 5.9 TB/s; with the norm 1057 to 1064;
// 65 × 4096: 3.6 + 4.3 µs).  Into fp32 bf16 gradients take 1914, 4.4 TB/s: a thread's two
// stores of 16 bytes lie next to each other, so that each of a wave's is half of every line.
// ---------------------------------------------------------------------------
struct Factor {
  float c;
  int shift;
  __device__ __forceinline__ explicit Factor(double quotient) : c((float)quotient), shift(0) {
    if (quotient < 0x1p-126) c = (float)frexp(quotient, &shift);
  }
  __device__ __forceinline__ float times(float v) const { return ldexpf(v * c, shift); }
};
template <typename T, typename O>
__device__ __forceinline__ void scale_chunk(gptr<const T> p, gptr<O> out, int64_t e0, int64_t e1, Factor c) {
  out += e0;
  chunk<true>(p + e0, (int)(e1 - e0),
        [&](int at, auto& v) {
#pragma unroll
          for (int e = 0; e < 16 / (int)sizeof(T); ++e) v[e] = c.times(v[e]);
          store_unit(out + at, v);
        },
        [&](int at, float v) { store_element(out + at, c.times(v)); });
}

__global__ __launch_bounds__(kThreads) void k_grad_clip(ClipTable tab, ClipScalars s) {
  __shared__ double shared[kThreads / 64];
  if (tab.probs[0].tag != tab.tag) return;
  const float norm = s.measured ? joined_norm(tab, shared) : *s.norm;
  if (s.measured && blockIdx.x == 0 && threadIdx.x == 0) *s.norm = norm;
  const double quotient = (double)s.max_norm / ((double)norm + (double)s.eps);
  const Factor c(!(fabsf(norm) < INFINITY) || !(quotient < 1.0) ? 1.0 : quotient);
  walk(tab, [&](const ClipProblem& P, int64_t e0, int64_t e1) {
    if (P.out == P.grad && c.c == 1.f && c.shift == 0) return;
    if (P.f32) {
      if (P.out_f32) scale_chunk(glob((const float*)P.grad), glob((float*)P.out), e0, e1, c);
      else scale_chunk(glob((const float*)P.grad), glob((uint16_t*)P.out), e0, e1, c);
    } else {
      if (P.out_f32) scale_chunk(glob((const uint16_t*)P.grad), glob((float*)P.out), e0, e1, c);
      else scale_chunk(glob((const uint16_t*)P.grad), glob((uint16_t*)P.out), e0, e1, c);
    }
  });
}

int launch_grad_norm(const ClipTable& tab, void* stream) {
  DMUON_LAUNCH(PH_GRAD_NORM, stream, k_grad_norm, (unsigned)tab.groups, kThreads, 0, tab);
}
int launch_grad_norm_join(const ClipTable& tab, float* norm, void* stream) {
  DMUON_LAUNCH(PH_GRAD_NORM, stream, k_grad_norm_join, 1, kThreads, 0, tab, norm);
}
int launch_grad_clip(const ClipTable& tab, const ClipScalars& s, void* stream) {
  DMUON_LAUNCH(PH_GRAD_CLIP, stream, k_grad_clip, (unsigned)tab.groups, kThreads, 0, tab, s);
}

}  // namespace dmuon
