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
// Unit j of a piece of len ≥ 8 elements.  The last one is the piece's last 8 elements, of
// which those of the unit before count as −∞, so that it is one load too.
template <typename T>
struct Piece {
  gptr<const T> p;
  int len, units;
  __device__ __forceinline__ Piece(gptr<const T> row, int n) : p(row), len(n), units((n + 7) >> 3) {}
  __device__ __forceinline__ int start(int j) const { return (j + 1) * 8 <= len ? j * 8 : len - 8; }
  __device__ __forceinline__ void load(Unit<T, 8>& x, int j) const { x.load(p + start(j)); }
  // its values; element e is number start(j) + e of the piece
  __device__ __forceinline__ void values(const Unit<T, 8>& x, int j, float (&v)[8]) const {
    x.values(v);
    if ((j + 1) * 8 > len) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (len - 8 + e < j * 8) v[e] = -INFINITY;
    }
  }
};

// ---------------------------------------------------------------------------
// one pass over a row.  With m the largest logit so far, c2 = scale·log₂e and the
// reference M = m·c2 rounded once, a logit's exponent is t = z·c2 − M in one fused
// multiply-add, and
//   s = Σ 2^t,   u = Σ t·2^t.
// M's rounding r = m·c2 − M is a factor 2^r of every term.  With R = 2^r, computed as the
// largest logit's own term is,
//   S = Σ e^(scale·(z − m)) = s/R,   entropy = ln S − ln 2·(u − r·s)/s.
// s holds R at least once, so S ≥ 1, and S = 1 where nothing else is left: no log
// probability is above 0 and no entropy below, and both keep their digits for a word that is
// nearly certain (ln S as ln s − r·ln 2 was off by 6·10⁻⁸ of either sign).  When m grows,
// every t moves by e = (m − m')·c2 + r' − r: u becomes 2^e·(u + e·s), s becomes 2^e·s.
// Beyond |M| = 2^24, where r could pass 1/2, t is (z − m)·c2 and r is 0.  m starts
// at the lowest finite value, so that no difference is −∞ − −∞; a logit of −∞ has 2^t = 0
// and its t is kept finite for the product.  A NaN reaches s.  A lane that has seen nothing but
// −∞ counts as beyond 2^24, and its wave takes that slower form meanwhile: 8192 × 32000 bf16 with
// 99% of the words masked out 101 µs, with none 89 (fp32 171 and 165).
// Bound by the instructions: 16 elements are taken together, 6.6 instructions each beside
// the maximum's bookkeeping (unpack, maximum, t, 2^t, clamp, two sums).
// ---------------------------------------------------------------------------
constexpr float kFar = -1e30f;           // an exponent whose power of 2 is 0
constexpr float kBig = 0x1p24f;
constexpr float kLn2 = 0.693147180559945309f;

struct Running {
  float m, M, s, u;
  static __device__ __forceinline__ Running from(float m, float s, float u, float c2) { return {m, m * c2, s, u}; }
  static __device__ __forceinline__ Running none(float c2) { return from(kLowest, 0.f, 0.f, c2); }
  static __device__ __forceinline__ bool big(float M) { return !(fabsf(M) < kBig); }
  static __device__ __forceinline__ float rest(float m, float M, float c2) { return big(M) ? 0.f : fmaf(m, c2, -M); }
  __device__ __forceinline__ void grow(float to, float c2) {
    const float next = to * c2;
    const float e = fmaf(m - to, c2, rest(to, next, c2) - rest(m, M, c2));
    const float a = __builtin_amdgcn_exp2f(e);
    u = a * fmaf(fmaxf(e, kFar), s, u);
    s *= a;
    m = to;
    M = next;
  }
  // units of 8; their maxima go out
  template <int N>
  __device__ __forceinline__ void add(const float (&v)[N], float (&top)[N / 8], float c2) {
#pragma unroll
    for (int k = 0; k < N / 8; ++k) {
      top[k] = v[8 * k];
#pragma unroll
      for (int e = 1; e < 8; ++e) top[k] = fmaxf(top[k], v[8 * k + e]);
    }
    const float most = N == 8 ? top[0] : fmaxf(top[0], top[N / 8 - 1]);
    if (most > m) grow(most, c2);
    if (__any(big(M))) {
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {                      // kept short
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const float z = h ? v[N / 2 + e] : v[e];
          const float t = big(M) ? (z - m) * c2 : fmaf(z, c2, -M);
          const float p = __builtin_amdgcn_exp2f(t);
          s += p;
          u = fmaf(p, fmaxf(t, kFar), u);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float t = fmaf(v[e], c2, -M);
        const float p = __builtin_amdgcn_exp2f(t);
        s += p;
        u = fmaf(p, fmaxf(t, kFar), u);
      }
    }
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
  __device__ __forceinline__ Row(const Running& r, float c, float c2) : m(r.m), scale(c) {
    const bool none = r.s == 0.f;
    const float rest = Running::rest(r.m, r.M, c2);
    log_s = none ? 0.f : logf(r.s / __builtin_amdgcn_exp2f(rest));
    float below = fmaf(-rest, r.s, r.u);                 // Σ (t − r)·2^t: no term is positive
    below = below > 0.f ? 0.f : below;                   // a NaN stays
    lse = none ? -INFINITY : fmaf(r.m, c, log_s);
    entropy = none ? 0.f : log_s - below * kLn2 / r.s;
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

// the target's logit, loaded before the row so that its latency passes beside it
template <typename T>
__device__ __forceinline__ float target_logit(const LogprobsArgs& a, int64_t row, int64_t y, int kind) {
  return a.targets && kind == kInside ? element(glob((const T*)a.logits) + row * a.ld + y) : 0.f;
}
__device__ __forceinline__ void write_row(const LogprobsArgs& a, int64_t row, float z, int kind, const Row& r) {
  a.lse[row] = r.lse;
  a.entropy[row] = r.entropy;
  if (a.targets) a.logprobs[row] = kind == kInside ? r.log_p(z) : kind == kShard ? -r.lse : kNan;
}

// ---------------------------------------------------------------------------
// the k largest of a piece, by G threads (a wave or a workgroup).  The k-th largest of many
// disjoint parts' maxima, tau, is not above the k-th largest element, and few elements reach
// it: only parts that do are looked at again.  If more elements than the list holds are
// greater than tau, the k-th largest of those it took becomes the new tau (it is greater:
// each round drops at least the rest of the list).  Elements equal to tau are needed where
// fewer than k are greater; where many are (equal logits, words masked out by −∞) the
// first of them in order are looked for.  Places come from counting the greater keys:
// keys are distinct, so the result does not depend on the list's order.
// ---------------------------------------------------------------------------
template <int STRICT, int TIES>
struct TopShared {
  static constexpr int kStrict = STRICT, kTies = TIES;
  alignas(16) uint64_t list[STRICT + TIES];
  int wave[kThreads / 64];
  float tau;
};
template <int G>
__device__ __forceinline__ void sync() {
  if constexpr (G > 64) {
    __syncthreads();
  } else {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
}

// the k-th largest of the N values of each lane together, bit by bit from ballots, in every
// lane (bf16: 16 bits tell the values apart)
template <typename T, int N>
__device__ __forceinline__ float kth_largest(const float (&value)[N], int k) {
  constexpr int low = sizeof(T) == 2 ? 16 : 0;
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i) key[i] = ordered(value[i]) >> low;
  uint32_t t = 0;
#pragma unroll 4
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
// of a workgroup's threads' maxima, every wave by itself
template <typename T>
__device__ __forceinline__ float kth_of_threads(const float* most, int k) {
  float v[kThreads / 64];
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) v[i] = most[(threadIdx.x & 63) + 64 * i];
  return kth_largest<T>(v, k);
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

// emit(place, key) for the min(k, len) largest of the piece; returns their number.
// gather(tau, again, strict, ties) puts the piece's elements from tau on into the list
// and counts those greater than and equal to tau (again: the counters are to be cleared),
// behind a barrier.
template <typename T, int G, typename S, typename C, typename F>
__device__ __forceinline__ int select_top(S& sh, const Piece<T>& row, int tid, int first, int k, float tau, C gather, F emit) {
  const int lane = tid & 63, wave = tid >> 6, len = row.len;
  const int want = k < len ? k : len;
  int strict, ties;
  gather(tau, false, strict, ties);
  while (strict > S::kStrict) {
    for (int i = tid; i < S::kStrict; i += G)
      if (places_above(sh.list, S::kStrict, sh.list[i]) == k - 1) sh.tau = key_value(sh.list[i]);
    sync<G>();
    tau = sh.tau;
    sync<G>();
    gather(tau, true, strict, ties);
  }
  if (strict >= want) {
    ties = 0;
  } else if (ties > S::kTies) {                          // then len > 8
    const int need = want - strict;
    int have = 0;
    for (int base = 0; have < need && base < row.units; base += G) {
      const int j = base + tid, at0 = row.start(j);
      uint32_t in = 0;
      if (j < row.units) {
        Unit<T, 8> x;
        float v[8];
        row.load(x, j);
        row.values(x, j, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) in |= (uint32_t)(rankable(v[e]) == tau && at0 + e >= j * 8 && at0 + e < len) << e;
      }
      int incl = __popc(in);
      const int n = incl;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int up = __shfl_up(incl, o, 64);
        if (lane >= o) incl += up;
      }
      int at = have + incl - n, all = 0;
      if constexpr (G > 64) {
        if (lane == 63) sh.wave[wave] = incl;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < G / 64; ++w) {
          if (w < wave) at += sh.wave[w];
          all += sh.wave[w];
        }
      } else {
        all = __shfl(incl, 63, 64);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (in >> e & 1) {
          if (at < need) sh.list[S::kStrict + at] = key_of(rankable(tau), first + at0 + e);
          ++at;
        }
      have += all;
      sync<G>();
    }
    ties = need;
  }
  // one list: the ties behind the others (from the front, so that none is overwritten unread)
  for (int i = 0; i < ties; i += G) {
    uint64_t moved = 0;
    if (i + tid < ties) moved = sh.list[S::kStrict + i + tid];
    sync<G>();
    if (i + tid < ties) sh.list[strict + i + tid] = moved;
    sync<G>();
  }
  const int n = strict + ties;
  for (int i = tid; i < n; i += G) {
    const uint64_t key = sh.list[i];
    const int place = places_above(sh.list, n, key);
    if (place < want) emit(place, key);
  }
  return want;
}

// ---------------------------------------------------------------------------
// a piece (of 8 elements at least) streamed by G threads.  Rows start at any element; loads
// off the 4-byte grid are slow (8192 × 50257 bf16: 193 µs, × 50258 171), so the units lie on
// the 16-byte grid, and the up to 7 elements before and behind them are two more units,
// from the piece's own ends, for the last two threads.  Loads past the last whole unit take
// that one again, so that all of a batch are in flight without a branch, and count as −∞;
// waves that are past it skip them.  ONCE: nontemporal loads, for logits that exceed the
// caches (bf16 8192 × 128000 312 µs, else 356, 4096 × 50257 74 and 79, fp32 4096 × 128000
// 319 and 358; of logits that fit, the gradient that reads them next loses more: 8192 × 2000
// both passes 25 and 23, 512 × 32000 28 and 24).  With alternatives the units that are read
// again miss then: worth it for bf16 rows of more than 1024 words an alternative (4096 ×
// 128000 with 20 of them 178 and 200 µs, with 64 187 and 201; 8192 × 32000 with 20 110 and
// 111, with 64 128 and 121).
// ---------------------------------------------------------------------------
template <typename T, int G, bool AGAIN>
struct Stream {
  const Piece<T>& in;
  int tid, head, full, groups;           // elements before the grid, whole units, groups of units
  bool at_head, at_tail;                 // this thread has one of the ends
  Unit<T, 8> edge;

  __device__ __forceinline__ Stream(const Piece<T>& p, int t) : in(p), tid(t) {
    head = (int)((16u - ((uint32_t)(uintptr_t)p.p & 15u)) & 15u) / (int)sizeof(T);
    full = (p.len - head) >> 3;
    groups = (full + G * kGroupUnits - 1) / (G * kGroupUnits);
    at_head = head > 0 && tid == G - 1;
    at_tail = (p.len - head) % 8 > 0 && tid == G - 2;
    if (at_head || at_tail) edge.load(p.p + (at_head ? 0 : p.len - 8));
  }
  // an end's elements, the others −∞; element e is number edge_at() + e of the piece
  __device__ __forceinline__ int edge_at() const { return at_head ? 0 : in.len - 8; }
  __device__ __forceinline__ void edge_values(float (&v)[8]) const {
    edge.values(v);
    const int rest = (in.len - head) % 8;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at_head ? e >= head : e < 8 - rest) v[e] = -INFINITY;
  }
  // Unit j is 8 elements one after another, or of fp32 that is read once two quads 64 quads
  // apart, so that each load of a wave is whole lines (AGAIN: units are read again one by one,
  // 64 alternatives of 8192 × 32000 207 µs, with quads 228); past the end its elements are
  // not its own.
  static constexpr bool kQuads = sizeof(T) == 4 && !AGAIN;
  __device__ __forceinline__ bool own(int j, int e) const {
    return kQuads ? (j & 63) + (e < 4 ? 0 : 64) < 2 * (full - (j & ~63)) : j < full;
  }
  __device__ __forceinline__ int index(int j, int e) const {
    return head + (kQuads ? (j & ~63) * 8 + (j & 63) * 4 + (e < 4 ? e : 252 + e) : j * 8 + e);
  }
  template <bool ONCE>
  __device__ __forceinline__ void load(Unit<T, 8>& x, int j) const {
    if constexpr (kQuads) {
      const int last = 2 * full - 1, a = (j & ~63) * 2 + (j & 63);
      x.template load_quads<ONCE>(in.p + head + (a < last ? a : last) * 4, in.p + head + (a + 64 < last ? a + 64 : last) * 4);
    } else if (ONCE) {
      x.load_once(in.p + head + (j < full ? j : full - 1) * 8);
    } else {
      x.load(in.p + head + (j < full ? j : full - 1) * 8);
    }
  }
  // left: units from this wave's first one on
  __device__ __forceinline__ void clear(Unit<T, 8>& x, int lane, int left) const {
    if constexpr (kQuads) x.clear_quads(lane >= 2 * left, lane + 64 >= 2 * left);
    else if (lane >= left) x.clear();
  }
  // all of it into r; group(g, largest, largest) of both halves of every group of 8 units;
  // returns the largest of an end
  template <bool ONCE, typename F>
  __device__ __forceinline__ float run(Running& r, float c2, F group) {
    constexpr int B = sizeof(T) == 2 ? kGroupUnits : kGroupUnits / 2;       // loads in flight
    const int wave0 = tid & ~63, lane = tid & 63;
    for (int g = 0; g < groups; ++g) {
      float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int b = 0; b < kGroupUnits; b += B) {
        const int j0 = (g * kGroupUnits + b) * G;
        if (__builtin_amdgcn_readfirstlane(j0 + wave0) >= full) break;
        Unit<T, 8> x[B];
#pragma unroll
        for (int k = 0; k < B; ++k) load<ONCE>(x[k], j0 + k * G + tid);
#pragma unroll
        for (int k = 0; k < B; k += 2) {
          const int left = full - __builtin_amdgcn_readfirstlane(j0 + k * G + wave0);
          if (left <= 0) break;
          if (left < G + 64) {                           // the last units' waves
            clear(x[k], lane, left);
            clear(x[k + 1], lane, left - G);
          }
          float v[16], top[2];
          x[k].values(*(float(*)[8])&v[0]);
          x[k + 1].values(*(float(*)[8])&v[8]);
          r.add(v, top, c2);
          float& half = most[(b + k) / (kGroupUnits / 2)];
          half = fmaxf(half, fmaxf(top[0], top[1]));
        }
      }
      group(g, most[0], most[1]);
    }
    float top[1] = {-INFINITY};
    if (at_head || at_tail) {
      float v[8];
      edge_values(v);
      r.add(v, top, c2);
    }
    return top[0];
  }
};

__device__ __forceinline__ void ignored_row(const LogprobsArgs& a, int64_t row, int tid, int threads) {
  if (tid == 0) a.logprobs[row] = a.entropy[row] = a.lse[row] = 0.f;
  for (int i = tid; i < a.top; i += threads) {
    a.top_ids[row * a.top + i] = -1;
    a.top_logprobs[row * a.top + i] = 0.f;
  }
}

// an alternative of a row, or of a piece: its candidate; the candidates that a piece lacks
__device__ __forceinline__ void put_alternative(const LogprobsArgs& a, int64_t row, int piece, int place, uint64_t key, const Row& r) {
  if (a.pieces == 1) {
    a.top_ids[row * a.top + place] = key_index(key);
    a.top_logprobs[row * a.top + place] = r.log_p(key_value(key));
  } else {
    a.cand[(row * a.pieces + piece) * a.top + place] = key;
  }
}
__device__ __forceinline__ void no_alternatives(const LogprobsArgs& a, int64_t row, int piece, int from, int tid, int threads) {
  for (int i = from + tid; i < a.top; i += threads) a.cand[(row * a.pieces + piece) * a.top + i] = 0;
}

// ---------------------------------------------------------------------------
// a wave per row, without alternatives: no barrier, and four times the rows in flight.
// Against a workgroup per row (300 rows: several), bf16: 8192 × 5000 21 and 28 µs, × 12288 39
// and 41, × 16384 52 and 51, 1500 × 12300 15.1 and 12.5, 300 × 8192 7.0 and 9.4; fp32: 8192 ×
// 3000 21 and 25, × 5000 32 and 30, × 8192 49 and 46, 300 × 8192 7.5 and 9.3.
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ void short_row(gptr<const T> p, int len, Unit<T, 8>& x) {         // fewer than 8 elements
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < len ? element(p + e) : -INFINITY;
  x.set(v);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_logprobs_wave(LogprobsArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (row >= a.rows) return;
  const int64_t y = a.targets ? load_index(a.targets, a.idx64, row) : 0;
  const int kind = a.targets ? target_kind(y, a.ignore, a.vocab) : kInside;
  if (kind == kIgnored) return ignored_row(a, row, lane, 64);
  const Piece<T> in(glob((const T*)a.logits) + row * a.ld, a.vocab);
  const float zy = lane == 0 ? target_logit<T>(a, row, y, kind) : 0.f;
  const float c2 = a.scale * kLog2e;
  Running r = Running::none(c2);
  if (a.vocab >= 16) {
    Stream<T, 64, false> stream(in, lane);
    const auto group = [](int, float, float) {};
    if (a.once) stream.template run<true>(r, c2, group);
    else stream.template run<false>(r, c2, group);
  } else if (lane < in.units) {
    Unit<T, 8> x;
    if (a.vocab < 8) short_row(in.p, a.vocab, x);
    else in.load(x, lane);
    float v[8], top[1];
    if (a.vocab < 8) x.values(v);
    else in.values(x, lane, v);
    r.add(v, top, c2);
  }
  join_wave(r, c2);
  if (lane == 0) write_row(a, row, zy, kind, Row(r, a.scale, c2));
}

// ---------------------------------------------------------------------------
// a wave per row or piece with alternatives, for at most NB·512 units: the units' maxima stay
// in registers, and the units from tau on are read again.  tau comes from 8 maxima per lane
// (of parts of units where the row is short), or for few alternatives from the lanes'.
// ---------------------------------------------------------------------------
template <int NB>
struct WaveShared {
  TopShared<256, 128> top;
  uint16_t flag[NB * 512];
};
template <typename T, int NB>
__global__ __launch_bounds__(kThreads) void k_logprobs_wave_top(LogprobsArgs a) {
  __shared__ WaveShared<NB> shared[kThreads / 64];
  const int lane = threadIdx.x & 63;
  WaveShared<NB>& sh = shared[threadIdx.x >> 6];
  const uint32_t id = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t row = id / (uint32_t)a.pieces;
  const int piece = (int)(id - (uint32_t)row * a.pieces);
  if (row >= a.rows) return;
  const int64_t y = a.targets ? load_index(a.targets, a.idx64, row) : 0;
  const int kind = a.targets ? target_kind(y, a.ignore, a.vocab) : kInside;
  if (kind == kIgnored) {
    if (piece == 0) ignored_row(a, row, lane, 64);
    return;
  }
  const int first = piece * a.piece;
  const int len = a.vocab - first < a.piece ? a.vocab - first : a.piece;
  const Piece<T> in(glob((const T*)a.logits) + row * a.ld + first, len);
  const float zy = lane == 0 && a.pieces == 1 ? target_logit<T>(a, row, y, kind) : 0.f;
  const float c2 = a.scale * kLog2e;
  const bool tiny = len < 8;                         // one unit, not a load
  Running r = Running::none(c2);
  auto take = [&](Unit<T, 8>& x, int j) {
    if (tiny) short_row(in.p, len, x);
    else in.load(x, j < in.units ? j : in.units - 1);
  };
  auto open = [&](Unit<T, 8>& x, int j, float (&v)[8]) {
    if (j >= in.units) x.clear();
    if (tiny || j >= in.units) x.values(v);
    else in.values(x, j, v);
  };
  float top[NB * 8];
  constexpr int B = sizeof(T) == 2 ? 8 : 4;              // loads in flight
#pragma unroll
  for (int b = 0; b < NB * 8; b += B) {
#pragma unroll
    for (int k = 0; k < B; ++k) top[b + k] = -INFINITY;
    if (b * 64 < in.units) {
      Unit<T, 8> x[B];
#pragma unroll
      for (int k = 0; k < B; ++k) take(x[k], (b + k) * 64 + lane);
#pragma unroll
      for (int k = 0; k < B; k += 2) {
        if ((b + k) * 64 >= in.units) break;
        float v[16], t[2];
        open(x[k], (b + k) * 64 + lane, *(float(*)[8])&v[0]);
        open(x[k + 1], (b + k + 1) * 64 + lane, *(float(*)[8])&v[8]);
        r.add(v, t, c2);
        top[b + k] = rankable(t[0]);
        top[b + k + 1] = rankable(t[1]);
      }
    }
  }
  float tau;
  if (a.top <= 32 && in.units >= 64) {
    float one[1] = {top[0]};
#pragma unroll
    for (int k = 1; k < NB * 8; ++k) one[0] = fmaxf(one[0], top[k]);
    tau = kth_largest<T>(one, a.top);
  } else {
    float key[8];
    if (NB == 1 && in.units <= 256) {
      auto parts = [&](auto count) {                     // `count` units per lane, 8 / count maxima of each
        constexpr int N = decltype(count)::value;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          Unit<T, 8> x;
          float v[8];
          take(x, i * 64 + lane);
          open(x, i * 64 + lane, v);
#pragma unroll
          for (int q = 0; q < 8 / N; ++q) {
            float most = v[q * N];
#pragma unroll
            for (int e = 1; e < N; ++e) most = fmaxf(most, v[q * N + e]);
            key[i * (8 / N) + q] = rankable(most);
          }
        }
      };
      if (in.units <= 64) parts(std::integral_constant<int, 1>());
      else if (in.units <= 128) parts(std::integral_constant<int, 2>());
      else parts(std::integral_constant<int, 4>());
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        key[k] = top[k];
#pragma unroll
        for (int b = 1; b < NB; ++b) key[k] = fmaxf(key[k], top[b * 8 + k]);
      }
    }
    tau = kth_largest<T>(key, a.top);
  }
  join_wave(r, c2);
  const Row done(r, a.scale, c2);
  if (lane == 0) {
    if (a.pieces == 1) write_row(a, row, zy, kind, done);
    else a.stats[row * a.pieces + piece] = RowStat{r.m, r.s, r.u};
  }
  const uint64_t below = (1ull << lane) - 1;
  auto gather = [&](float t, bool, int& strict, int& ties) {
    strict = ties = 0;
    int flags = 0;
#pragma unroll
    for (int k = 0; k < NB * 8; ++k) {
      const bool on = top[k] >= t && k * 64 + lane < in.units;
      const uint64_t all = __ballot(on);
      if (on) sh.flag[flags + __popcll(all & below)] = (uint16_t)(k * 64 + lane);
      flags += __popcll(all);
    }
    sync<64>();
    for (int i = lane; i < (flags + 63 & ~63); i += 64) {
      const bool on = i < flags;
      const int j = on ? sh.flag[i] : in.units;
      Unit<T, 8> x;
      float v[8];
      take(x, j);
      open(x, j, v);
      const int at = tiny ? 0 : in.start(j);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = rankable(v[e]);
        const bool own = on && at + e >= j * 8 && at + e < len;
        const uint64_t more = __ballot(own && z > t), same = __ballot(own && z == t);
        if (own && z > t) {
          const int n = strict + __popcll(more & below);
          if (n < sh.top.kStrict) sh.top.list[n] = key_of(z, first + at + e);
        } else if (own && z == t) {
          const int n = ties + __popcll(same & below);
          if (n < sh.top.kTies) sh.top.list[sh.top.kStrict + n] = key_of(z, first + at + e);
        }
        strict += __popcll(more);
        ties += __popcll(same);
      }
    }
    sync<64>();
  };
  const int n = select_top<T, 64>(sh.top, in, lane, first, a.top, tau, gather,
                                  [&](int place, uint64_t key) { put_alternative(a, row, piece, place, key, done); });
  if (a.pieces > 1) no_alternatives(a, row, piece, n, lane, 64);
}

// ---------------------------------------------------------------------------
// a workgroup per row or piece.  With alternatives, pieces of up to 2048 (kShort) stay in
// registers, a unit per thread; of longer ones (kLong) the maxima of every 4 units of a
// thread stay in LDS, and only those that reach tau are read again: with 64 alternatives
// 2001 × 50257 bf16 takes 55 µs without and 62 with one maximum per 8 units, 47 without
// alternatives.  Without them 8192 × 128000 bf16 takes 312 µs (6.7 TB/s) at 2.1 GHz and more,
// where the instructions of a unit still pass behind its load; 378 at the 1.66 GHz that the
// card falls to for some milliseconds when such calls follow each other.
// ---------------------------------------------------------------------------
enum : int { kNoTop, kLong, kShort };
struct GroupTop : TopShared<512, 256> {
  float most[kThreads];                  // each thread's largest
  int flags, strict, ties;
};
struct GroupShared {
  uint16_t bound[2 * kGroups][kThreads]; // largest of each thread's 4 units, ordered bits rounded up
  uint16_t flag[2 * kGroups * kThreads]; // those to read again
};

__device__ __forceinline__ void put_candidate(GroupTop& sh, float raw, float tau, bool own, int index) {
  const float z = rankable(raw);
  if (own && z > tau) {
    const int i = atomicAdd(&sh.strict, 1);
    if (i < sh.kStrict) sh.list[i] = key_of(z, index);
  } else if (own && z == tau) {
    const int i = atomicAdd(&sh.ties, 1);
    if (i < sh.kTies) sh.list[sh.kStrict + i] = key_of(z, index);
  }
}

template <typename T, int TOP>
__global__ __launch_bounds__(kThreads) void k_logprobs(LogprobsArgs a) {
  __shared__ Running part[kThreads / 64];
  extern __shared__ __align__(16) char top_smem[];
  GroupTop& sh = *(GroupTop*)top_smem;
  GroupShared& groups = *(GroupShared*)(top_smem + sizeof(GroupTop));
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x / (uint32_t)a.pieces;
  const int piece = (int)(blockIdx.x - (uint32_t)row * a.pieces);
  const int64_t y = a.targets ? load_index(a.targets, a.idx64, row) : 0;
  const int kind = a.targets ? target_kind(y, a.ignore, a.vocab) : kInside;
  if (kind == kIgnored) {
    if (piece == 0) ignored_row(a, row, tid, kThreads);
    return;
  }
  const int first = piece * a.piece;
  const int len = a.vocab - first < a.piece ? a.vocab - first : a.piece;
  const Piece<T> in(glob((const T*)a.logits) + row * a.ld + first, len);
  const float zy = tid == 0 && a.pieces == 1 ? target_logit<T>(a, row, y, kind) : 0.f;
  const float c2 = a.scale * kLog2e;
  Running r = Running::none(c2);
  float most = -INFINITY;                                // of this thread
  float held[8];                                         // kShort: its unit
  Stream<T, kThreads, TOP == kLong> stream(in, tid);
  if constexpr (TOP == kShort) {
    if (tid < in.units) {
      Unit<T, 8> x;
      in.load(x, tid);
      in.values(x, tid, held);
      float top[1];
      r.add(held, top, c2);
      most = rankable(top[0]);
    }
  } else {
    const auto group = [&](int g, float lo, float hi) {
      if (TOP) {
        lo = rankable(lo);
        hi = rankable(hi);
        groups.bound[2 * g][tid] = (uint16_t)((ordered(lo) + 0xffffu) >> 16);
        groups.bound[2 * g + 1][tid] = (uint16_t)((ordered(hi) + 0xffffu) >> 16);
        most = fmaxf(most, fmaxf(lo, hi));
      }
    };
    const float end = (TOP == kNoTop || sizeof(T) == 2) && a.once ? stream.template run<true>(r, c2, group) : stream.template run<false>(r, c2, group);
    most = fmaxf(most, rankable(end));
  }
  if constexpr (TOP) {
    sh.most[tid] = most;
    if (tid == 0) sh.flags = sh.strict = sh.ties = 0;
  }
  join_wave(r, c2);
  if ((tid & 63) == 0) part[tid >> 6] = r;
  __syncthreads();
  r = part[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) {
    Running o = part[w];
    const float m = fmaxf(r.m, o.m);
    r.grow(m, c2);
    o.grow(m, c2);
    r.s += o.s;
    r.u += o.u;
  }
  const Row done(r, a.scale, c2);
  if (tid == 0) {
    if (a.pieces == 1) write_row(a, row, zy, kind, done);
    else a.stats[row * a.pieces + piece] = RowStat{r.m, r.s, r.u};
  }
  if constexpr (TOP) {
    auto gather = [&](float tau, bool again, int& strict, int& ties) {
      if (again) {
        if (tid == 0) sh.flags = sh.strict = sh.ties = 0;
        __syncthreads();
      }
      if constexpr (TOP == kLong) {
#pragma unroll 1
        for (int g = 0; g < 2 * stream.groups; ++g)
          if (groups.bound[g][tid] >= ordered(tau) >> 16) groups.flag[atomicAdd(&sh.flags, 1)] = (uint16_t)(g * kThreads + tid);
        if (stream.at_head || stream.at_tail) {
          float v[8];
          stream.edge_values(v);
          const int at = stream.edge_at(), rest = (len - stream.head) % 8;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            put_candidate(sh, v[e], tau, stream.at_head ? e < stream.head : e >= 8 - rest, first + at + e);
        }
        __syncthreads();
        constexpr int half = kGroupUnits / 2;
        const int units = sh.flags * half;
#pragma unroll 1
        for (int w = tid; w < units; w += kThreads) {
          const int f = groups.flag[w / half];
          const int j = (f / kThreads * half + w % half) * kThreads + f % kThreads;
          Unit<T, 8> x;
          float v[8];
          stream.template load<false>(x, j);
          x.values(v);
#pragma unroll
          for (int e = 0; e < 8; ++e) put_candidate(sh, v[e], tau, stream.own(j, e), first + stream.index(j, e));
        }
      } else if (tid < in.units && most >= tau) {
        const int at = in.start(tid);
#pragma unroll
        for (int e = 0; e < 8; ++e) put_candidate(sh, held[e], tau, at + e >= tid * 8, first + at + e);
      }
      __syncthreads();
      strict = sh.strict;
      ties = sh.ties;
    };
    const float tau = kth_of_threads<T>(sh.most, a.top);
    const int n = select_top<T, kThreads>(sh, in, tid, first, a.top, tau, gather,
                                          [&](int place, uint64_t key) { put_alternative(a, row, piece, place, key, done); });
    if (a.pieces > 1) no_alternatives(a, row, piece, n, tid, kThreads);
  }
}

// ---------------------------------------------------------------------------
// the pieces of a row joined: statistics by one wave, then the k largest of the pieces'
// sorted candidates, all in LDS, by the same rule as in a piece.  The candidates go to the
// threads by rank, all pieces' first ones first: the largest lie in different threads, and
// tau is near the k-th (by piece, 63 pieces of 64 candidates: 17.5 µs, 64 of 128: 31.6;
// by rank 7.5 and 9.7).
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void k_logprobs_join(LogprobsArgs a) {
  extern __shared__ __align__(16) char join_smem[];
  __shared__ Running whole;
  constexpr int kStrict = GroupTop::kStrict;
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
    const float zy = target_logit<T>(a, row, y, kind);
    Running r = Running::none(c2);
    if (tid < a.pieces) {
      const RowStat s = a.stats[row * a.pieces + tid];
      r = Running::from(s.m, s.s, s.u, c2);
    }
    join_wave(r, c2);
    if (tid == 0) {
      whole = r;
      write_row(a, row, zy, kind, Row(r, a.scale, c2));
    }
  }
  if (a.top == 0) return;
  uint64_t* keys = (uint64_t*)join_smem;
  const int n = a.pieces * a.top;
  uint64_t mine = 0;
#pragma unroll 8
  for (int i = tid; i < n; i += kThreads) {
    const uint32_t rank = (uint32_t)i / (uint32_t)a.pieces, p = (uint32_t)i - rank * a.pieces;
    const uint64_t key = a.cand[row * n + p * a.top + rank];
    keys[i] = key;
    mine = key > mine ? key : mine;
  }
  most[tid] = mine ? key_value(mine) : -INFINITY;
  if (tid == 0) count = 0;
  __syncthreads();
  const Row done(whole, a.scale, c2);
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
// l is kept within bounds (log_p_of).  Rows that
// take no part are zeros and their logits are not read.  Memory bound: 4096 × 128000 bf16,
// a quarter of the rows ignored, 318 µs, 5.8 TB/s of what is read and written; 512 × 10007
// fp32 10 µs.  A thread takes 32 elements at most, all loads in flight, so a row of up to 2048
// words is a wave's, and a longer one is shared evenly by workgroups of at most 8192 words
// (all but the last full: 8192 × 10007 bf16 82 µs, so 66).  A unit is 16 bytes, so that
// every load and store of a wave is whole lines (fp32 units of 8 elements, two of each:
// 2048 × 128000 423 µs, so 357).  Aligned rows are read nontemporally (bf16 2048 × 128000
// 183 µs, else 195, 4096 × 32000 87 and 92; but odd rows share their lines with the next
// unit: 300 × 50257 14.8 and 13.1).
// ---------------------------------------------------------------------------
template <typename T, int G>
__global__ __launch_bounds__(kThreads) void k_logprobs_grad(LogprobsGradArgs a) {
  const int tid = G == 64 ? threadIdx.x & 63 : threadIdx.x;
  const uint32_t id = blockIdx.x * (kThreads / G) + (G == 64 ? threadIdx.x >> 6 : 0);
  const int64_t row = id / (uint32_t)a.pieces;
  const int piece = (int)(id - (uint32_t)row * a.pieces);
  if (row >= a.rows) return;
  constexpr int W = 16 / sizeof(T), N = kGradUnits * 8 / W;
  const int j0 = piece * a.units + tid;                  // this thread's units of 16 bytes: j0 + k·G
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
  const int units = (a.vocab + W - 1) / W, end = (piece + 1) * a.units < units ? (piece + 1) * a.units : units;
  const auto start = [&](int j) { return (j + 1) * W <= a.vocab ? j * W : a.vocab - W; };      // the last: the row's last W
  Unit<T, W> x[N];
  if (a.aligned) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int j = j0 + k * G;
      if (takes_part && j < end) x[k].load_once(src + start(j));
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int j = j0 + k * G;
      if (takes_part && j < end && a.vocab >= W) x[k].load(src + start(j));
    }
  }
  if (takes_part && j0 == 0 && a.vocab < W) {
    float v[W];
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = e < a.vocab ? element(src + e) : 0.f;
    x[0].set(v);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int j = j0 + k * G;
    if (j >= end) break;
    const int at = a.vocab < W ? 0 : start(j);
    float v[W];
    if (takes_part) {
      x[k].values(v);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float l = log_p_of(fmaf(v[e], a.scale, -lse), lse);
        const float p = __builtin_amdgcn_exp2f(l * kLog2e);
        const float d = -p * fmaf(h, l + entropy, g);
        v[e] = a.scale * (at + e == target ? d + g : d);
      }
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = 0.f;
    }
    if ((j + 1) * W <= a.vocab) {
      store_unit(dst + at, v);
    } else {                                             // its own elements: the others are another thread's, also in place
#pragma unroll
      for (int e = 0; e < W; ++e)
        if (at + e >= j * W && at + e < a.vocab) store_element(dst + at + e, v[e]);
    }
  }
}

// ---------------------------------------------------------------------------
// launchers
// ---------------------------------------------------------------------------
template <typename T>
static int logprobs(const LogprobsArgs& a, void* stream) {
  const unsigned work = (unsigned)(a.rows * a.pieces), waves = (unsigned)cdiv(work, kThreads / 64);
  if (a.wave_rows) {
    if (!a.top) DMUON_LAUNCH(PH_LOGPROBS, stream, k_logprobs_wave<T>, waves, kThreads, 0, a);
    if (a.piece <= kWaveTop) DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs_wave_top<T, 1>), waves, kThreads, 0, a);
    DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs_wave_top<T, 3>), waves, kThreads, 0, a);
  }
  if (!a.top) DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs<T, kNoTop>), work, kThreads, 0, a);
  if (a.piece <= kPieceLeast) DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs<T, kShort>), work, kThreads, sizeof(GroupTop), a);
  DMUON_LAUNCH(PH_LOGPROBS, stream, (k_logprobs<T, kLong>), work, kThreads, sizeof(GroupTop) + sizeof(GroupShared), a);
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
