// Device code and launch helpers shared by the HIP sources of the training operators
// (grads.hip, logprobs.hip, clip.hip): rows of bf16 or fp32 in units of 8, indices, grids.
#pragma once

#include "core.hpp"

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

// l = x − lse as the gradients of log probabilities take it: from −200 on, where e^l is 0 in
// fp32, so that 0·−∞ does not arise.  lse is rounded to fp32, and the largest x of a row may come
// out above it by half a step.  From |lse| = 2^16 on, where that is more than a rounding to
// bf16, l is at most 0: e^l stays at most 1 for any finite logits (x = −1.25·10⁹ throughout,
// a row masked out: l up to 64 else).  A NaN stays.
__device__ __forceinline__ float log_p_of(float x_less_lse, float lse) {
  return x_less_lse == x_less_lse ? __builtin_amdgcn_fmed3f(x_less_lse, -200.f, fabsf(lse) < 0x1p16f ? 1.f : 0.f) : x_less_lse;
}

// ---------------------------------------------------------------------------
// units: 8 consecutive elements (fp32: or 4) as they were loaded, from any element on, so that
// rows of every alignment move 16 bytes at a time: the types are aligned to one element only.
// ---------------------------------------------------------------------------
typedef u32x4_t u32x4_any __attribute__((aligned(2)));
typedef f32x4_t f32x4_any __attribute__((aligned(4)));

template <typename T, int UNIT>
struct Unit;
template <>
struct Unit<uint16_t, 8> {
  u32x4_t u;
  __device__ __forceinline__ void load(gptr<const uint16_t> p) { u = *(gptr<const u32x4_any>)p; }
  __device__ __forceinline__ void load_once(gptr<const uint16_t> p) { u = __builtin_nontemporal_load((gptr<const u32x4_any>)p); }
  __device__ __forceinline__ void set(const float (&v)[8]) { u = pack8(v); }
  __device__ __forceinline__ void clear() { u = u32x4_t{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u}; }     // −∞
  __device__ __forceinline__ void values(float (&v)[8]) const { unpack8(u, v); }
};
template <>
struct Unit<float, 8> {
  f32x4_t a, b;
  __device__ __forceinline__ void load(gptr<const float> p) {
    a = ((gptr<const f32x4_any>)p)[0];
    b = ((gptr<const f32x4_any>)p)[1];
  }
  __device__ __forceinline__ void load_once(gptr<const float> p) {
    a = __builtin_nontemporal_load((gptr<const f32x4_any>)p);
    b = __builtin_nontemporal_load((gptr<const f32x4_any>)p + 1);
  }
  // two quads that do not follow each other
  template <bool ONCE>
  __device__ __forceinline__ void load_quads(gptr<const float> p, gptr<const float> q) {
    a = ONCE ? __builtin_nontemporal_load((gptr<const f32x4_any>)p) : *(gptr<const f32x4_any>)p;
    b = ONCE ? __builtin_nontemporal_load((gptr<const f32x4_any>)q) : *(gptr<const f32x4_any>)q;
  }
  __device__ __forceinline__ void clear_quads(bool first, bool second) {
    if (first) a = f32x4_t{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (second) b = f32x4_t{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = f32x4_t{v[0], v[1], v[2], v[3]};
    b = f32x4_t{v[4], v[5], v[6], v[7]};
  }
  __device__ __forceinline__ void clear() { a = b = f32x4_t{-INFINITY, -INFINITY, -INFINITY, -INFINITY}; }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <>
struct Unit<float, 4> {
  f32x4_t a;
  __device__ __forceinline__ void load(gptr<const float> p) { a = *(gptr<const f32x4_any>)p; }
  __device__ __forceinline__ void load_once(gptr<const float> p) { a = __builtin_nontemporal_load((gptr<const f32x4_any>)p); }
  __device__ __forceinline__ void set(const float (&v)[4]) { a = f32x4_t{v[0], v[1], v[2], v[3]}; }
  __device__ __forceinline__ void values(float (&v)[4]) const { v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; }
};
__device__ __forceinline__ float element(gptr<const uint16_t> p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float element(gptr<const float> p) { return *p; }
__device__ __forceinline__ void store_unit(gptr<uint16_t> p, const float (&v)[8]) {
  __builtin_nontemporal_store(pack8(v), (gptr<u32x4_any>)p);
}
__device__ __forceinline__ void store_unit(gptr<float> p, const float (&v)[8]) {
  __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (gptr<f32x4_any>)p);
  __builtin_nontemporal_store(f32x4_t{v[4], v[5], v[6], v[7]}, (gptr<f32x4_any>)p + 1);
}
__device__ __forceinline__ void store_unit(gptr<uint16_t> p, const float (&v)[4]) {
  typedef uint16_t quad __attribute__((ext_vector_type(4)));
  typedef quad quad_any __attribute__((aligned(2)));
  __builtin_nontemporal_store(quad{f32_to_bf16(v[0]), f32_to_bf16(v[1]), f32_to_bf16(v[2]), f32_to_bf16(v[3])}, (gptr<quad_any>)p);
}
__device__ __forceinline__ void store_unit(gptr<float> p, const float (&v)[4]) {
  __builtin_nontemporal_store(f32x4_t{v[0], v[1], v[2], v[3]}, (gptr<f32x4_any>)p);
}
__device__ __forceinline__ void store_element(gptr<uint16_t> p, float v) { *p = f32_to_bf16(v); }
__device__ __forceinline__ void store_element(gptr<float> p, float v) { *p = v; }

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// Workgroups of a grid-stride kernel: enough to fill 256 CUs several times over
inline unsigned stride_grid(int64_t items) {
  const int64_t wg = cdiv(items, kThreads);
  return (unsigned)(wg < 1 ? 1 : (wg < 16384 ? wg : 16384));
}

#define DMUON_LAUNCH(phase, stream, kernel, grid, block, lds, ...)                             \
  do {                                                                                         \
    timing_before(phase, stream);                                                              \
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(block), lds, (hipStream_t)(stream), __VA_ARGS__); \
    const int err_ = (int)hipGetLastError();                                                   \
    timing_after(phase, stream);                                                               \
    return err_;                                                                               \
  } while (0)

}  // namespace dmuon
