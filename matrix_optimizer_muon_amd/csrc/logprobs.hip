// HIP kernels of log probabilities from logits in memory for gfx950 (MI355X): the given
// token's log probability, the entropy and the most likely alternatives of every row, and
// the gradient.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "core.hpp"
#include "elements.hpp"
#include "grads.hpp"
#include "logprobs.hpp"

namespace dmuon {

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLowest = -3.402823466e38f;
constexpr float kNan = __builtin_nanf("");

// ---------------------------------------------------------------------------
// units of a row
// ---------------------------------------------------------------------------
// unit j of a piece of len elements, −∞ past its end
template <typename T, int UNIT>
__device__ __forceinline__ void edge_unit(gptr<const T> row, int j, int len, float (&v)[UNIT]) {
#pragma unroll
  for (int e = 0; e < UNIT; ++e) v[e] = j * UNIT + e < len ? element(row + j * UNIT + e) : -INFINITY;
}
template <typename T, int UNIT>
__device__ __forceinline__ void any_unit(gptr<const T> row, int j, int len, float (&v)[UNIT]) {
  if ((j + 1) * UNIT <= len) {
    Unit<T, UNIT> x;
    x.load(row + j * UNIT);
    x.values(v);
  } else {
    edge_unit<T, UNIT>(row, j, len, v);
  }
}

// ---------------------------------------------------------------------------
// one pass over a row: with m the largest logit so far,
//   s = Σ e^{c(z − m)},   u = Σ (z − m)·e^{c(z − m)}   (c: the scale)
// and both multiplied by e^{c(m − m')} when m grows to m' (u first becomes
// Σ (z − m')·…, that is u + (m − m')·s).  m starts at the lowest finite value, so that no
// difference is −∞ − −∞: a logit of −∞ has e = 0, and its difference is kept finite for
// the product 0·(z − m).  A NaN reaches s through its e.
// ---------------------------------------------------------------------------
constexpr float kFar = -1e30f;           // a difference whose exponential is 0

struct Running {
  float m, s, u;
  __device__ __forceinline__ void grow(float to, float c2) {
    const float d = m - to;
    const float a = __builtin_amdgcn_exp2f(d * c2);
    u = a * fmaf(fmaxf(d, kFar), s, u);
    s *= a;
    m = to;
  }
  template <int N>
  __device__ __forceinline__ float add(const float (&v)[N], float c2) {        // returns the largest of v
    float most = v[0];
#pragma unroll
    for (int e = 1; e < N; ++e) most = fmaxf(most, v[e]);
    if (most > m) grow(most, c2);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = v[e] - m;
      const float p = __builtin_amdgcn_exp2f(d * c2);
      s += p;
      u = fmaf(p, fmaxf(d, kFar), u);
    }
    return most;
  }
};

// the statistics of all lanes of a wave, in every lane
__device__ __forceinline__ void join_wave(Running& r, float c2) {
  float m = r.m;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  r.grow(m, c2);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    r.s += __shfl_xor(r.s, o, 64);
    r.u += __shfl_xor(r.u, o, 64);
  }
}

// A finished row.  Where no logit is finite (s = 0: all are −∞) lse and every log
// probability are −∞ and the entropy is 0.
struct Row {
  float m, log_s, lse, entropy, scale;
  __device__ __forceinline__ Row(const Running& r, float c) : m(r.m), scale(c) {
    const bool none = r.s == 0.f;
    log_s = none ? 0.f : logf(r.s);
    lse = none ? -INFINITY : fmaf(r.m, c, log_s);
    entropy = none ? 0.f : log_s - r.u * c / r.s;
  }
  // (z − m)·c − log s: neither term is positive, and the logarithm keeps its digits
  // beside a large m
  __device__ __forceinline__ float log_p(float z) const { return (z - m) * scale - log_s; }
};

// ordered bits: rise with the value
__device__ __forceinline__ uint32_t ordered(float z) {
  const uint32_t b = __float_as_uint(z);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// Keys order by value, then by lower index: the value's bits as a whole number in the
// high half, ~index in the low one.  NaN counts as −∞, −0 as 0.  No key is 0.
__device__ __forceinline__ float rankable(float z) { return fmaxf(z, -INFINITY) + 0.f; }
__device__ __forceinline__ uint64_t key_of(float z, int32_t index) { return (uint64_t)ordered(z) << 32 | (uint32_t)~index; }
__device__ __forceinline__ float key_value(uint64_t key) { return from_ordered((uint32_t)(key >> 32)); }
__device__ __forceinline__ int32_t key_index(uint64_t key) { return (int32_t)~(uint32_t)key; }

// what a row's target asks for
enum : int { kIgnored, kInside, kShard, kOutside };
__device__ __forceinline__ int target_kind(int64_t y, int64_t ignore, int32_t vocab) {
  return y == ignore ? kIgnored : y >= 0 && y < vocab ? kInside : y == kElsewhere ? kShard : kOutside;
}

template <typename T>
__device__ __forceinline__ void write_row(const LogprobsArgs& a, int64_t row, int64_t y, int kind, const Row& r) {
  a.lse[row] = r.lse;
  a.entropy[row] = r.entropy;
  if (!a.targets) return;
  a.logprobs[row] = kind == kInside ? r.log_p(element(glob((const T*)a.logits) + row * a.ld + y)) : kind == kShard ? -r.lse : kNan;
}

// ---------------------------------------------------------------------------
// the k largest of a piece.  The k-th largest of the threads' maxima, tau, is not above
// the k-th largest element, and few elements reach it.  Every wave finds it by itself, bit
// by bit from ballots over the 256 maxima.  If more elements than the list holds are
// greater than tau, the k-th largest of those it took becomes the new tau (it is greater:
// each round drops at least the rest of the list).  Elements equal to tau are needed where
// fewer than k are greater; where many are (equal logits, words masked out by −∞) the
// first of them in order are looked for.  Places come from counting the greater keys:
// keys are distinct, so the result does not depend on the list's order.
// ---------------------------------------------------------------------------
constexpr int kStrict = 512, kTies = 256;

struct TopShared {
  alignas(16) uint64_t list[kStrict + kTies];
  float most[kThreads];                  // each thread's largest
  int flags, strict, ties, wave[kThreads / 64];
  float tau;
};
struct GroupShared {
  float group[kGroups][kThreads];        // largest of each thread's groups
  uint16_t flag[kGroups * kThreads];     // groups to read again
};

// the k-th largest of 256 values in LDS, in every lane (k ≤ 256)
template <typename T>
__device__ __forceinline__ float kth_of_threads(const float* most, int k) {
  constexpr int N = kThreads / 64, low = sizeof(T) == 2 ? 16 : 0;     // bf16: 16 bits tell the values apart
  const int lane = threadIdx.x & 63;
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = ordered(most[lane + 64 * i]) >> low;
  uint32_t t = 0;
#pragma unroll
  for (int b = 31 - low; b >= 0; --b) {
    const uint32_t c = t | 1u << b;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += __popcll(__ballot(key[i] >= c));
    if (n >= k) t = c;
  }
  t = __builtin_amdgcn_readfirstlane(t);
  return from_ordered(low ? t << 16 | (t & 0x8000u ? 0u : 0xffffu) : t);
}

// the number of keys greater than `key` in list[0, n)
__device__ __forceinline__ int places_above(const uint64_t* list, int n, uint64_t key) {
  int r = 0;
  int i = 0;
  for (; i + 8 <= n; i += 8) {
    ulonglong2 o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = *(const ulonglong2*)(list + i + 2 * u);
#pragma unroll
    for (int u = 0; u < 4; ++u) r += (o[u].x > key) + (o[u].y > key);
  }
  for (; i < n; ++i) r += list[i] > key;
  return r;
}

__device__ __forceinline__ void put_candidate(TopShared& sh, float raw, float tau, bool inside, int index) {
  const float z = rankable(raw);
  if (z > tau) {
    const int i = atomicAdd(&sh.strict, 1);
    if (i < kStrict) sh.list[i] = key_of(z, index);
  } else if (z == tau && inside) {
    const int i = atomicAdd(&sh.ties, 1);
    if (i < kTies) sh.list[kStrict + i] = key_of(z, index);
  }
}

// emit(place, key) for the min(k, len) largest of the piece, whose threads' maxima are in
// sh.most and whose counters are 0 (behind a barrier); returns their number.  gather(tau)
// puts the piece's elements from tau on into the list.
template <typename T, typename G, typename F>
__device__ __forceinline__ int select_top(TopShared& sh, gptr<const T> row, int len, int first, int k, G gather, F emit) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int want = k < len ? k : len;
  float tau = kth_of_threads<T>(sh.most, k);
  int strict, ties;
  for (;;) {
    gather(tau);
    __syncthreads();
    strict = sh.strict;
    ties = sh.ties;
    if (strict <= kStrict) break;
    for (int i = tid; i < kStrict; i += kThreads)
      if (places_above(sh.list, kStrict, sh.list[i]) == k - 1) sh.tau = key_value(sh.list[i]);
    __syncthreads();
    tau = sh.tau;
    if (tid == 0) sh.flags = sh.strict = sh.ties = 0;
    __syncthreads();
  }
  if (strict >= want) {
    ties = 0;
  } else if (ties > kTies) {
    const int need = want - strict;
    int have = 0;
    for (int base = 0; have < need && base * 8 < len; base += kThreads) {
      float v[8];
      any_unit<T, 8>(row, base + tid, len, v);
      uint32_t in = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) in |= (uint32_t)(rankable(v[e]) == tau && (base + tid) * 8 + e < len) << e;
      int incl = __popc(in);
      const int n = incl;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(incl, o, 64);
        if (lane >= o) incl += up;
      }
      if (lane == 63) sh.wave[wave] = incl;
      __syncthreads();
      int at = have + incl - n, all = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wave) at += sh.wave[w];
        all += sh.wave[w];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (in >> e & 1) {
          if (at < need) sh.list[kStrict + at] = key_of(tau, first + (base + tid) * 8 + e);
          ++at;
        }
      have += all;
      __syncthreads();
    }
    ties = need;
  }
  if (ties > 0) {                        // one list: the ties behind the others
    uint64_t moved = 0;
    if (tid < ties) moved = sh.list[kStrict + tid];
    __syncthreads();
    if (tid < ties) sh.list[strict + tid] = moved;
    __syncthreads();
  }
  const int n = strict + ties;
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t key = sh.list[i];
    const int place = places_above(sh.list, n, key);
    if (place < want) emit(place, key);
  }
  return want;
}

// ---------------------------------------------------------------------------
// G threads per row (or piece of one): a wave where rows are short, else a workgroup.
// Memory bound: a thread has kGroupUnits loads of 16 bytes in flight.  With alternatives,
// pieces of up to 2048 stay in registers, 8 elements per thread (kShort; kNarrow, for
// vocabularies below that, takes them 256 apart, so that as many threads as possible hold
// a maximum); of longer ones (kLong) the maxima of each thread's groups stay in LDS, and
// only groups that reach tau are read again.
// ---------------------------------------------------------------------------
enum : int { kNoTop, kLong, kShort, kNarrow };

template <typename T, int G, int TOP>
__global__ __launch_bounds__(kThreads) void k_logprobs(LogprobsArgs a) {
  __shared__ Running part[kThreads / 64];
  const int tid = G == 64 ? threadIdx.x & 63 : threadIdx.x;
  const uint32_t id = blockIdx.x * (kThreads / G) + (G == 64 ? threadIdx.x >> 6 : 0);
  const int64_t row = id / (uint32_t)a.pieces;
  const int piece = (int)(id - (uint32_t)row * a.pieces);
  if (row >= a.rows) return;                             // only where a wave has its own row
  const int64_t y = a.targets ? load_index(a.targets, a.idx64, row) : 0;
  const int kind = a.targets ? target_kind(y, a.ignore, a.vocab) : kInside;
  if (kind == kIgnored) {
    if (piece == 0) {
      if (tid == 0) a.logprobs[row] = a.entropy[row] = a.lse[row] = 0.f;
      for (int i = tid; i < a.top; i += G) {
        a.top_ids[row * a.top + i] = -1;
        a.top_logprobs[row * a.top + i] = 0.f;
      }
    }
    return;
  }
  const int first = piece * a.piece;
  const int len = a.vocab - first < a.piece ? a.vocab - first : a.piece;
  const gptr<const T> src = glob((const T*)a.logits) + row * a.ld + first;
  const float c2 = a.scale * kLog2e;
  Running r = {kLowest, 0.f, 0.f};
  extern __shared__ __align__(16) char top_smem[];
  TopShared& sh = *(TopShared*)top_smem;
  GroupShared& groups = *(GroupShared*)(top_smem + sizeof(TopShared));
  float most = -INFINITY;                                // of this thread
  float held[8];                                         // kShort, kNarrow: its elements
  constexpr int B = sizeof(T) == 2 ? kGroupUnits : kGroupUnits / 2;       // loads in flight
  const int ngroups = (len + G * kGroupUnits * 8 - 1) / (G * kGroupUnits * 8);
  if constexpr (TOP == kShort) {
    any_unit<T, 8>(src, tid, len, held);
    most = r.add(held, c2);
  } else if constexpr (TOP == kNarrow) {
#pragma unroll
    for (int e = 0; e < 8; ++e) held[e] = e * kThreads + tid < len ? element(src + e * kThreads + tid) : -INFINITY;
    most = r.add(held, c2);
  } else {
    for (int g = 0; g < ngroups; ++g) {
      float top = -INFINITY;
      if ((g + 1) * G * kGroupUnits * 8 <= len) {
#pragma unroll
        for (int b = 0; b < kGroupUnits; b += B) {
          Unit<T, 8> x[B];
#pragma unroll
          for (int k = 0; k < B; ++k) x[k].load(src + (int64_t)((g * kGroupUnits + b + k) * G + tid) * 8);
#pragma unroll
          for (int k = 0; k < B; ++k) {
            float v[8];
            x[k].values(v);
            const float o = r.add(v, c2);
            if (TOP) top = fmaxf(top, o);
          }
        }
      } else {
#pragma unroll 1
        for (int k = 0; k < kGroupUnits; ++k) {
          const int j = (g * kGroupUnits + k) * G + tid;
          if (j * 8 >= len) break;
          float v[8];
          any_unit<T, 8>(src, j, len, v);
          const float o = r.add(v, c2);
          if (TOP) top = fmaxf(top, o);
        }
      }
      if (TOP) {
        top = rankable(top);
        groups.group[g][tid] = top;
        most = fmaxf(most, top);
      }
    }
  }
  if constexpr (TOP) {
    sh.most[tid] = rankable(most);
    if (tid == 0) sh.flags = sh.strict = sh.ties = 0;
  }
  join_wave(r, c2);
  if constexpr (G > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = r;
    __syncthreads();
    Running all = part[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w) {
      Running o = part[w];
      const float m = fmaxf(all.m, o.m);
      all.grow(m, c2);
      o.grow(m, c2);
      all.s += o.s;
      all.u += o.u;
    }
    r = all;
  }
  const Row done(r, a.scale);
  if (tid == 0) {
    if (a.pieces == 1) write_row<T>(a, row, y, kind, done);
    else a.stats[row * a.pieces + piece] = RowStat{r.m, r.s, r.u};
  }
  if constexpr (TOP) {
    auto gather = [&](float tau) {
      if constexpr (TOP == kLong) {
        for (int g = 0; g < ngroups; ++g)
          if (groups.group[g][tid] >= tau) groups.flag[atomicAdd(&sh.flags, 1)] = (uint16_t)(g * kThreads + tid);
        __syncthreads();
        const int units = sh.flags * kGroupUnits;
        for (int w = tid; w < units; w += kThreads) {
          const int f = groups.flag[w / kGroupUnits];
          const int j = (f / kThreads * kGroupUnits + w % kGroupUnits) * kThreads + f % kThreads;
          if (j * 8 >= len) continue;
          float v[8];
          any_unit<T, 8>(src, j, len, v);
#pragma unroll
          for (int e = 0; e < 8; ++e) put_candidate(sh, v[e], tau, j * 8 + e < len, first + j * 8 + e);
        }
      } else if (sh.most[tid] >= tau) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = TOP == kShort ? tid * 8 + e : e * kThreads + tid;
          put_candidate(sh, held[e], tau, at < len, first + at);
        }
      }
    };
    if (a.pieces == 1) {
      select_top(sh, src, len, first, a.top, gather, [&](int place, uint64_t key) {
        a.top_ids[row * a.top + place] = key_index(key);
        a.top_logprobs[row * a.top + place] = done.log_p(key_value(key));
      });
    } else {
      uint64_t* out = a.cand + (row * a.pieces + piece) * a.top;
      const int n = select_top(sh, src, len, first, a.top, gather, [&](int place, uint64_t key) { out[place] = key; });
      for (int i = n + tid; i < a.top; i += kThreads) out[i] = 0;
    }
  }
}

// ---------------------------------------------------------------------------
// the pieces of a row joined: statistics by one wave, then the k largest of the pieces'
// sorted candidates, all in LDS, by the same rule as in a piece.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void k_logprobs_join(LogprobsArgs a) {
  extern __shared__ __align__(16) char join_smem[];
  __shared__ Running whole;
  __shared__ alignas(16) uint64_t list[kStrict];
  __shared__ float most[kThreads];
  __shared__ uint64_t next_tau;
  __shared__ int count;
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const int64_t y = a.targets ? load_index(a.targets, a.idx64, row) : 0;
  const int kind = a.targets ? target_kind(y, a.ignore, a.vocab) : kInside;
  if (kind == kIgnored) return;                          // written by the first piece's workgroup
  const float c2 = a.scale * kLog2e;
  if (tid < 64) {
    Running r = {kLowest, 0.f, 0.f};
    if (tid < a.pieces) {
      const RowStat s = a.stats[row * a.pieces + tid];
      r.m = s.m;
      r.s = s.s;
      r.u = s.u;
    }
    join_wave(r, c2);
    if (tid == 0) {
      whole = r;
      write_row<T>(a, row, y, kind, Row(r, a.scale));
    }
  }
  if (a.top == 0) return;
  uint64_t* keys = (uint64_t*)join_smem;
  const int n = a.pieces * a.top;
  uint64_t mine = 0;
#pragma unroll 8
  for (int i = tid; i < n; i += kThreads) {
    const uint64_t key = a.cand[row * n + i];
    keys[i] = key;
    mine = key > mine ? key : mine;
  }
  most[tid] = mine ? key_value(mine) : -INFINITY;
  if (tid == 0) count = 0;
  __syncthreads();
  const Row done(whole, a.scale);
  uint64_t tau = key_of(kth_of_threads<T>(most, a.top), -1);       // the least key of that value
  for (;;) {
    for (int i = tid; i < n; i += kThreads)
      if (keys[i] >= tau) {
        const int at = atomicAdd(&count, 1);
        if (at < kStrict) list[at] = keys[i];
      }
    __syncthreads();
    const int have = count;
    if (have <= kStrict) {
      for (int i = tid; i < have; i += kThreads) {
        const int place = places_above(list, have, list[i]);
        if (place < a.top) {
          a.top_ids[row * a.top + place] = key_index(list[i]);
          a.top_logprobs[row * a.top + place] = done.log_p(key_value(list[i]));
        }
      }
      return;
    }
    for (int i = tid; i < kStrict; i += kThreads)
      if (places_above(list, kStrict, list[i]) == a.top - 1) next_tau = list[i];
    __syncthreads();
    tau = next_tau;
    if (tid == 0) count = 0;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// the gradient, element by element: with l = c·z − lse and p = e^l,
//   dz = c·(g·[v = target] − p·(g + h·(l + H)))     (g, h: of the log probability, the entropy)
// l is kept from −200 on (e^−200 is 0 in fp32), so that 0·−∞ does not arise.  Rows that
// take no part are zeros and their logits are not read.  Memory bound.
// ---------------------------------------------------------------------------
template <typename T, int G>
__global__ __launch_bounds__(kThreads) void k_logprobs_grad(LogprobsGradArgs a) {
  const int tid = G == 64 ? threadIdx.x & 63 : threadIdx.x;
  const uint32_t id = blockIdx.x * (kThreads / G) + (G == 64 ? threadIdx.x >> 6 : 0);
  const int64_t row = id / (uint32_t)a.pieces;
  const int piece = (int)(id - (uint32_t)row * a.pieces);
  if (row >= a.rows) return;
  const int j0 = piece * G * kGradUnits + tid;           // this thread's units: j0 + k·G
  const gptr<const T> src = glob((const T*)a.logits) + row * a.ld;
  const gptr<T> dst = glob((T*)a.out) + row * a.ldo;
  const int64_t y = a.targets ? load_index(a.targets, a.idx64, row) : 0;
  const int kind = a.targets ? target_kind(y, a.ignore, a.vocab) : kShard;
  const float g = a.grad_logprobs ? a.grad_logprobs[row] : 0.f;
  const float h = a.grad_entropy ? a.grad_entropy[row] : 0.f;
  const float lse = a.lse[row];
  const float entropy = a.grad_entropy ? a.entropy[row] : 0.f;
  const bool takes_part = kind != kIgnored && kind != kOutside && !(g == 0.f && h == 0.f) && !(lse == -INFINITY);
  const int target = kind == kInside ? (int)y : -1;
#pragma unroll
  for (int k = 0; k < kGradUnits; ++k) {
    const int j = j0 + k * G;
    if (j * 8 >= a.vocab) break;
    float v[8];
    if (takes_part) {
      any_unit<T, 8>(src, j, a.vocab, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float l = fmaf(v[e], a.scale, -lse);
        l = l < -200.f ? -200.f : l;                     // a NaN stays
        const float p = __builtin_amdgcn_exp2f(l * kLog2e);
        const float d = -p * fmaf(h, l + entropy, g);
        v[e] = a.scale * (j * 8 + e == target ? d + g : d);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
    if ((j + 1) * 8 <= a.vocab) {
      store_unit(dst + j * 8, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j * 8 + e < a.vocab) store_element(dst + j * 8 + e, v[e]);
    }
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
template <typename T>
static int logprobs(const LogprobsArgs& a, void* stream) {
  const unsigned work = (unsigned)(a.rows * a.pieces);
  constexpr unsigned few = sizeof(TopShared), all = sizeof(TopShared) + sizeof(GroupShared);
  if (a.top) {
    if (a.vocab < kPieceLeast) DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs<T, kThreads, kNarrow>), work, kThreads, few, a);
    if (a.piece <= kPieceLeast) DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs<T, kThreads, kShort>), work, kThreads, few, a);
    DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs<T, kThreads, kLong>), work, kThreads, all, a);
  }
  if (a.vocab <= kWaveRow) DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs<T, 64, kNoTop>), (unsigned)cdiv(work, kThreads / 64), kThreads, 0, a);
  DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs<T, kThreads, kNoTop>), work, kThreads, 0, a);
}
int launch_logprobs(const LogprobsArgs& a, int f32, void* stream) { return f32 ? logprobs<float>(a, stream) : logprobs<uint16_t>(a, stream); }
int launch_logprobs_join(const LogprobsArgs& a, int f32, void* stream) {
  const unsigned lds = (unsigned)(a.pieces * a.top * sizeof(uint64_t));
  if (f32) DMUON_LAUNCH(PH_LOGPROBS, stream, k_logprobs_join<float>, (unsigned)a.rows, kThreads, lds, a);
  DMUON_LAUNCH(PH_LOGPROBS, stream, k_logprobs_join<uint16_t>, (unsigned)a.rows, kThreads, lds, a);
}
template <typename T>
static int logprobs_grad(const LogprobsGradArgs& a, void* stream) {
  const int64_t work = a.rows * a.pieces;
  if (a.vocab <= kGradWave) DMUON_LAUNCH(PH_LOGPROBS_GRAD, stream, (k_logprobs_grad<T, 64>), (unsigned)cdiv(work, kThreads / 64), kThreads, 0, a);
  DMUON_LAUNCH(PH_LOGPROBS_GRAD, stream, (k_logprobs_grad<T, kThreads>), (unsigned)work, kThreads, 0, a);
}
int launch_logprobs_grad(const LogprobsGradArgs& a, int f32, void* stream) {
  return f32 ? logprobs_grad<float>(a, stream) : logprobs_grad<uint16_t>(a, stream);
}

}  // namespace dmuon
