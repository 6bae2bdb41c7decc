// Log probability of a given token, entropy and top tokens of every row of logits, in
// one pass over the row.
//
// With M = max x, S = sum e^(x - M) and T = sum e^(x - M) (x - M) <= 0:
//
//   log p(t) = (x_t - M) - log S,    H = log S - T / S.
//
// Both terms of H are non-negative, so a row that is almost certain keeps its small
// entropy to fp32's absolute precision.  Exponents are taken in base 2 with one rounding,
// y = fma(x, log2 e, -c), c = M log2 e as rounded: S, T (here sum 2^y y) and the given
// token's y all refer to the same c, so its rounding cancels.  But that rounding is the
// y of the maximum itself, up to half a step of c: 1/16 for |M| < 2^20, where it is let be,
// and 128 or more, past the range of 2^y, from |c| = 2^31 on.  So from |M| = 2^20 on (a row
// or a part of one masked with -1e9 or -1e30, say) M is taken off first, y = (x - M) log2 e,
// which costs an instruction per element there and elsewhere a test per step.  A wave keeps
// one running M; sums move to a new reference as S' = r S, T' = r (T + d S), d the
// difference of the references, r = 2^d.  Sums are fp32.
//
// Top tokens: a wave keeps its best (value, index) pairs sorted, one per lane, and
// a bound g; a vector whose maximum is at most g (all but a few, once the list has
// filled) costs one comparison, which also finds a new M and a NaN.  Before the first
// vector g comes from the K-th largest of the lanes' maxima over the first loads: K
// elements are known to lie at or above it.  Values are ordered as 32-bit keys (NaN
// above +inf, -0 equal to +0); equal values by lower index.
//
// Few long rows: a row is split over work-groups, and a second launch joins the parts in
// a fixed order.
//
// HBM-bound on long texts: 4096 x 65536 bf16 with the top token 94 to 97 us, 5.6 TB/s (a large
// read reaches 5.95); 8192 x 32000 fp16 92 to 94 us, 5.6 TB/s.  With 20 top tokens the former takes
// 149 us: some 70 elements per wave pass its bound.  1 x 128000 bf16 with 20 top tokens 13 us:
// about 7 in 63 parts, whose selection is a chain of dependent steps, 5.5 in the join.
#include "gptq_internal.h"

namespace gptq {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kUnroll = 2;              // 16-byte vectors per lane and iteration
constexpr int kMaxTop = 64;
// lanes with elements for the list from which on it is merged with all of them at once (first
// loads: 4): 4096 x 65536 bf16 with 20 top tokens 149 us, 160 with 4, 155 never after the
// first loads, 167 with a lane's elements picked by comparisons in every lane
constexpr int kMerge = 8;
constexpr int kMaxSplits = 128;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kFloor = -1e30f;        // stands for -inf in a product with 2^-inf = 0
constexpr float kFar = 0x1p20f;         // maxima of at least this magnitude are subtracted first
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

struct F32 {
  typedef float elem;
  static constexpr int E = 4;           // elements of a 16-byte vector
  static constexpr uint32_t kNone = 0xff800000u;      // a word of -inf
  static __device__ float one(elem x) { return x; }
  static __device__ uint32_t word(elem x) { return __builtin_bit_cast(uint32_t, x); }   // x, then -inf
};
struct F16 {
  typedef uint16_t elem;
  static constexpr int E = 8;
  static constexpr uint32_t kNone = 0xfc00fc00u;
  static __device__ float one(elem x) { return (float)__builtin_bit_cast(_Float16, x); }
  static __device__ uint32_t word(elem x) { return (kNone & 0xffff0000u) | x; }
};
struct BF16 {
  typedef uint16_t elem;
  static constexpr int E = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
  static __device__ float one(elem x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
  static __device__ uint32_t word(elem x) { return (kNone & 0xffff0000u) | x; }
};

template <typename T>
__device__ __forceinline__ void unpack(u32x4 v, float (&x)[T::E]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t u = v[q];    // a copy: a bit cast of the vector's element itself reads element 0
    if constexpr (std::is_same<T, F32>::value) x[q] = __builtin_bit_cast(float, u);
    else if constexpr (std::is_same<T, F16>::value) {
      const h2 p = __builtin_bit_cast(h2, u);
      x[2 * q] = (float)p[0];
      x[2 * q + 1] = (float)p[1];
    } else {
      x[2 * q] = __builtin_bit_cast(float, u << 16);
      x[2 * q + 1] = __builtin_bit_cast(float, u & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t b = __builtin_bit_cast(uint32_t, x == 0.f ? 0.f : x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
// key 0 (no value) gives a NaN, below which nothing lies
__device__ __forceinline__ float value_of(uint32_t key) {
  return __builtin_bit_cast(float, (key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ float fmaximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ float wave_maximum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaximum(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int l) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}

// the reference of a maximum: y = fma(x - base, log2 e, -c), either base or c being 0
struct Ref {
  float m, base, c;
};
__device__ __forceinline__ Ref make_ref(float m) {
#pragma clang fp contract(off)      // c as rounded, wherever it is used
  return fabsf(m) < kFar ? Ref{m, 0.f, m * kLog2e} : Ref{m, m, 0.f};
}
// the maximum's own y
__device__ __forceinline__ float own_y(const Ref& r) { return r.base == 0.f ? fmaf(r.m, kLog2e, -r.c) : 0.f; }

// moves sums from one reference to another of no smaller maximum
__device__ __forceinline__ void rescale(float& s, float& t, const Ref& a, const Ref& b) {
  if (!(a.m > -INFINITY)) return;         // nothing summed yet
  const float by = a.base == 0.f && b.base == 0.f ? a.c - b.c : fmaf(a.m - b.m, kLog2e, own_y(b) - own_y(a));
  const float d = fmaxf(by, kFloor);      // no overflow in t below
  const float r = __builtin_amdgcn_exp2f(d);
  t = r * fmaf(d, s, t);
  s *= r;
}

struct Wave {
  Ref ref;              // of the wave
  float s, t;           // per lane
  float g;              // elements at or below g change neither m nor the list
  uint32_t gkey;        // key of the list's entry top_k
  uint64_t best;        // entry `lane` of the sorted list, 0: none
};

struct Part {
  float m, s, t;
};

// the largest value below the one of a key (0: none); -0 is no value of its own
__device__ __forceinline__ float value_below(uint32_t key) {
  return value_of(key == 0u ? 0u : key == 0x80000000u ? 0x7ffffffeu : key - 1);
}

// a list entry as one number: larger is better (the key, then the lower index)
__device__ __forceinline__ uint64_t entry(uint32_t key, int idx) { return ((uint64_t)key << 32) | (uint32_t)~idx; }

// Puts the elements above g of one lane's loads into the list: a lane takes one of them.
// first: index of element 0 of this lane's vector there, negative: none
template <typename T>
__device__ __forceinline__ void insert(Wave& a, const u32x4 (&found)[kUnroll][64], int from, int first, int top_k, int lane) {
  const int u = lane / T::E, e = lane % T::E;
  const float v = T::one(((const typename T::elem*)&found[u < kUnroll ? u : 0][from])[e]);
  const uint64_t mine = entry(key_of(v), first + e);
  uint64_t todo = __ballot(u < kUnroll && first >= 0 && !(v <= a.g));
  while (todo) {
    const int l = __builtin_ctzll(todo);
    todo &= todo - 1;
    const uint64_t k = ((uint64_t)lane_value((uint32_t)(mine >> 32), l) << 32) | lane_value((uint32_t)mine, l);
    const int pos = __popcll(__ballot(a.best > k));
    if (pos >= top_k) continue;
    const auto left = [](uint32_t v) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x138, 0xf, 0xf, false); };
    const uint64_t before = ((uint64_t)left((uint32_t)(a.best >> 32)) << 32) | left((uint32_t)a.best);
    a.best = lane < pos ? a.best : lane == pos ? k : before;
  }
}

// sum over the lanes up to this one
__device__ __forceinline__ int lanes_up_to(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, true);
  return v;
}

// Puts all elements above g into the list at once, if they and it are at most 64: one
// element or entry to a lane, whose place is the number of better ones.  mask: a lane's
// elements above g, bit u E + e; first(u): index of a lane's element (u, 0); scratch: 64
// entries of the wave's own.
template <typename T, typename First>
__device__ __forceinline__ bool merge(Wave& a, const u32x4 (&found)[kUnroll][64], uint32_t mask, First&& first, int top_k,
                                      int lane, uint64_t* scratch) {
  const int c = __popc(mask), upto = lanes_up_to(c);
  const int held = __popcll(__ballot(lane < top_k && a.best != 0u)), n = held + (int)lane_value((uint32_t)upto, 63);
  if (n > 64) return false;
  int at = held + upto - c;
  while (__any(mask != 0u)) {
    if (mask != 0u) {
      const int b = __builtin_ctz(mask), u = b / T::E, e = b % T::E;
      mask &= mask - 1;
      const float v = T::one(((const typename T::elem*)&found[u][lane])[e]);
      scratch[at++] = entry(key_of(v), first(u) + e);
    }
  }
  const uint64_t mine = lane < held ? a.best : lane < n ? scratch[lane] : 0u;
  int rank = 0;
  for (int j = 0; j < n; j += 4) {       // lanes from n on hold 0
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t other = ((uint64_t)lane_value((uint32_t)(mine >> 32), j + i) << 32) | lane_value((uint32_t)mine, j + i);
      rank += other > mine;
    }
  }
  if (lane < n && rank < top_k) scratch[rank] = mine;
  a.best = lane < min(n, top_k) ? scratch[lane] : 0u;
  return true;
}

// the given token of a row and its logit (0 where there is none)
struct Given {
  int64_t token;
  float x;
};
template <typename T>
__device__ __forceinline__ Given given_token(const LogprobArgs& p, int64_t row) {
  Given g{p.tokens[row], 0.f};
  if (g.token >= 0 && g.token < p.v) g.x = T::one(((const typename T::elem*)p.logits)[row * p.ld + g.token]);
  return g;
}

// outputs of one row from its joined sums; best: the row's entry t
__device__ __forceinline__ void finish(const LogprobArgs& p, int64_t row, Part r, Given given, int t, uint64_t best) {
  const bool sound = fabsf(r.m) < INFINITY;      // neither empty nor with +inf or NaN
  const Ref ref = make_ref(r.m);
  const float log2_s = log2f(r.s);
  const auto log_p = [&](float x) {
    if (!sound) return NAN;
    const float y = fmaf(x - ref.base, kLog2e, -ref.c);
    if (y < kFloor) return (x - r.m) - kLn2 * log2_s;      // beyond y's range, or -inf
    return kLn2 * (y - log2_s);
  };
  if (t < p.top_k) {
    p.top_ids[row * p.top_k + t] = ~(int)(uint32_t)best;
    p.top_logprobs[row * p.top_k + t] = log_p(value_of((uint32_t)(best >> 32)));
  }
  if (t == 0) {
    p.logprobs[row] = given.token < 0 ? 0.f : given.token >= p.v ? NAN : log_p(given.x);
    p.entropy[row] = sound ? kLn2 * (log2_s - r.t / r.s) : NAN;
  }
}

// a part's record in the workspace: m, s, t, unused, then top_k list entries
__host__ __device__ inline int64_t record_words(int top_k) { return 4 + 2 * top_k; }

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(8))) void
logprob_kernel(LogprobArgs p, int splits, int64_t span, uint32_t* __restrict__ ws) {
  constexpr int E = T::E;
  __shared__ float ps[kWaves][3];
  __shared__ __attribute__((aligned(16))) uint64_t list[kWaves][kMaxTop];     // 0: no entry
  __shared__ uint64_t sorted[kMaxTop];
  __shared__ u32x4 found[TOP ? kWaves : 1][kUnroll][64];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t row = blockIdx.x / splits;
  const int part = (int)(blockIdx.x % splits);
  const auto* x = (const typename T::elem*)p.logits + row * p.ld;
  const int v = (int)p.v;
  // whole 16-byte vectors [head, head + E * nvec); the elements before and after go one to a lane
  const int head = min(v, (int)(((16 - ((uintptr_t)x & 15)) & 15) / sizeof(typename T::elem)));
  const int nvec = (v - head) / E, tail0 = head + nvec * E;
  const u32x4* xv = (const u32x4*)(x + head);
  Wave a{make_ref(-INFINITY), 0.f, 0.f, TOP ? NAN : -INFINITY, 0u, 0u};
  const int first = (int)min<int64_t>((int64_t)part * span, nvec), last = (int)min<int64_t>(first + span, nvec);
  const int edges = head + v - tail0;
  bool fresh = true, more = part == 0 && w == 0 && edges > 0;
  for (int b = first + w * (64 * kUnroll); b < last || more; b += kWaves * 64 * kUnroll) {
    u32x4 ld[kUnroll];          // elements that do not exist are -inf: they add nothing
    const bool edge = b >= last;
    if (!edge) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = b + 64 * u + lane;
        ld[u] = __builtin_nontemporal_load(&xv[min(i, last - 1)]);      // read once
        if (i >= last) ld[u] = u32x4{T::kNone, T::kNone, T::kNone, T::kNone};
      }
    } else {
      // what lies outside whole vectors comes last, one element to a lane; some have a
      // lower index than those before, so they pass at g too
      more = false;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) ld[u] = u32x4{T::kNone, T::kNone, T::kNone, T::kNone};
      if (lane < edges) ld[0][0] = T::word(x[lane < head ? lane : tail0 + lane - head]);
      if (TOP && !fresh) a.g = value_below(a.gkey);
    }
    float f[kUnroll][E], lm = -INFINITY;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      unpack<T>(ld[u], f[u]);
#pragma unroll
      for (int e = 0; e < E; ++e) lm = fmaximum(lm, f[u][e]);
    }
    if (__any(!(lm <= a.g))) {
      if (__any(!(lm <= a.ref.m))) {
        const Ref next = make_ref(fmaximum(a.ref.m, wave_maximum(lm)));
        rescale(a.s, a.t, a.ref, next);
        a.ref = next;
      }
      if constexpr (TOP) {
        if (fresh) {
          // a bound below which no element belongs to the top: the K-th largest lane
          // maximum, to its upper 20 bits
          const uint32_t lk = (edge ? lane < edges : b + lane < last) ? key_of(lm) : 0u;
          uint32_t bound = 0u;
#pragma unroll 1
          for (uint32_t bit = 0x80000000u; bit >= 0x1000u; bit >>= 1)
            if (__popcll(__ballot(lk >= (bound | bit))) >= p.top_k) bound |= bit;
          a.g = value_below(bound);
        }
        // through LDS, so that the rare path is one piece of code for all vectors
        // index of element 0 of vector u of a lane, negative: none
        const auto first_index = [&](int u, int l) {
          const int i = b + 64 * u + l;
          return !edge ? (i < last ? head + i * E : -1) : u > 0 || l >= edges ? -1 : l < head ? l : tail0 + l - head;
        };
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) found[w][u][lane] = ld[u];
        uint64_t lanes = __ballot(!(lm <= a.g));
        bool done = false;
        if (__popcll(lanes) >= (fresh ? 4 : kMerge)) {
          uint32_t mask = 0u;
#pragma unroll
          for (int u = 0; u < kUnroll; ++u) {
            const int n = first_index(u, lane) < 0 ? 0 : edge ? 1 : E;
#pragma unroll
            for (int e = 0; e < E; ++e) mask |= (e < n && !(f[u][e] <= a.g)) ? 1u << (u * E + e) : 0u;
          }
          done = merge<T>(a, found[w], mask, [&](int u) { return first_index(u, lane); }, p.top_k, lane, list[w]);
        }
        if (!done) {
          while (lanes) {
            const int l = __builtin_ctzll(lanes);
            lanes &= lanes - 1;
            const int at = first_index(lane / E, l);
            insert<T>(a, found[w], l, edge && lane % E != 0 ? -1 : at, p.top_k, lane);
          }
        }
        a.gkey = lane_value((uint32_t)(a.best >> 32), p.top_k - 1);
        const float kth = value_of(a.gkey);
        // the first loads' bound stays until the list has filled
        a.g = a.gkey != 0u ? kth : a.g;
      } else {
        a.g = a.ref.m;
      }
      // unpacked anew: kept over this path, the elements would cost registers and so waves
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        asm volatile("" : "+v"(ld[u]));
        unpack<T>(ld[u], f[u]);
      }
    }
    fresh = false;
    if (__any(a.ref.base != 0.f)) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) f[u][e] -= a.ref.base;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float y = fmaxf(fmaf(f[u][e], kLog2e, -a.ref.c), kFloor);
        const float q = __builtin_amdgcn_exp2f(y);
        a.s += q;
        a.t = fmaf(q, y, a.t);
      }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    a.s += __shfl_xor(a.s, o, 64);
    a.t += __shfl_xor(a.t, o, 64);
  }
  if (lane == 0) {
    ps[w][0] = a.ref.m;
    ps[w][1] = a.s;
    ps[w][2] = a.t;
  }
  const uint64_t mine = a.best;
  if (TOP) {
    list[w][lane] = lane < p.top_k ? mine : 0u;
    if (w == 0) sorted[lane] = 0u;
  }
  __syncthreads();
  Part r{ps[0][0], 0.f, 0.f};
#pragma unroll
  for (int i = 1; i < kWaves; ++i) r.m = fmaximum(r.m, ps[i][0]);
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    float s = ps[i][1], q = ps[i][2];
    rescale(s, q, make_ref(ps[i][0]), make_ref(r.m));
    r.s += s;
    r.t += q;
  }
  if (TOP) {
    // an entry's place among the waves' lists is the number of better ones
    if (lane < p.top_k && mine != 0u) {
      int rank = 0;
#pragma unroll 1
      for (int j = 0; j < p.top_k; j += 2)
#pragma unroll
        for (int i = 0; i < kWaves; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) rank += list[i][j + e] > mine;
      if (rank < p.top_k) sorted[rank] = mine;
    }
    __syncthreads();
  }
  if (splits == 1) {
    finish(p, row, r, given_token<T>(p, row), t, t < p.top_k ? sorted[t] : 0u);
    return;
  }
  uint32_t* rec = ws + (int64_t)blockIdx.x * record_words(p.top_k);
  if (t == 0) {
    rec[0] = __builtin_bit_cast(uint32_t, r.m);
    rec[1] = __builtin_bit_cast(uint32_t, r.s);
    rec[2] = __builtin_bit_cast(uint32_t, r.t);
  }
  if (t < p.top_k) {
    ((uint64_t*)rec)[2 + t] = sorted[t];
  }
}

// one row per work-group: wave 0 joins the sums.  The top: among the first `depth`
// entries of every part's list, the one with top_k - 1 better ones is a bound; the
// entries at or above it (at most top_k + top_k^2 / depth: a list with more than depth
// of them has all its first ones there) are gathered, and an entry's place is the number
// of better ones among them.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprob_join_kernel(LogprobArgs p, int splits,
                                                                const uint32_t* __restrict__ ws) {
  extern __shared__ uint64_t lists[];      // [splits][top_k], then the entries gathered from them
  __shared__ uint64_t sorted[kMaxTop];
  __shared__ uint64_t bound;
  __shared__ int count;
  const int t = threadIdx.x, lane = t & 63, K = p.top_k;
  const int64_t row = blockIdx.x, words = record_words(K);
  const uint32_t* rec = ws + row * splits * words;
  for (int i = t; i < splits * K; i += 8 * kThreads) {      // eight loads at a time
    uint64_t e[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t at = i + u * kThreads, l = at / (uint32_t)K;
      e[u] = at < (uint32_t)(splits * K) ? ((const uint64_t*)(rec + l * words))[2 + at - l * K] : 0u;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + u * kThreads < splits * K) lists[i + u * kThreads] = e[u];
  }
  Part r{-INFINITY, 0.f, 0.f};
  Given given{-1, 0.f};
  if (t < 64) {
    given = given_token<T>(p, row);
    Part own[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 64 * h;
      own[h] = Part{-INFINITY, 0.f, 0.f};
      if (i < splits) {
        const uint32_t* q = rec + i * words;
        own[h] = Part{__builtin_bit_cast(float, q[0]), __builtin_bit_cast(float, q[1]), __builtin_bit_cast(float, q[2])};
      }
      r.m = fmaximum(r.m, own[h].m);
    }
    r.m = wave_maximum(r.m);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      rescale(own[h].s, own[h].t, make_ref(own[h].m), make_ref(r.m));
      r.s += own[h].s;
      r.t += own[h].t;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      r.s += __shfl_xor(r.s, o, 64);
      r.t += __shfl_xor(r.t, o, 64);
    }
  }
  uint64_t place = 0u;
  if (K > 0) {
    const int depth = max(1, min(K, (2 * K + splits - 1) / splits)), some = splits * depth;
    uint64_t* const cand = lists + splits * K;
    if (t < kMaxTop) sorted[t] = 0u;
    if (t == 0) {
      count = 0;
      bound = 0u;
    }
    __syncthreads();
    for (int i = t; i < some; i += kThreads) {
      const uint64_t e = lists[(i % splits) * K + i / splits];
      int rank = 0;
      for (int d = 0; d < depth; ++d)
#pragma unroll 8
        for (int j = 0; j < splits; ++j) rank += lists[j * K + d] > e;
      if (rank == K - 1 && e != 0u) bound = e;        // one entry: they differ
    }
    __syncthreads();
    const uint64_t least = bound;
    for (int i = t; i < splits * K; i += kThreads) {
      const uint64_t e = lists[i];
      if (e >= least && e != 0u) cand[atomicAdd(&count, 1)] = e;
    }
    __syncthreads();
    const int n = count;
    for (int i = t; i < n; i += kThreads) {
      const uint64_t e = cand[i];
      int rank = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += cand[j] > e;
      if (rank < K) sorted[rank] = e;
    }
    __syncthreads();
    if (t < K) place = sorted[t];
  }
  if (t < 64) finish(p, row, r, given, t, place);
}

template <typename T>
hipError_t launch(const LogprobPlan& plan, const LogprobArgs& p, uint32_t* ws, hipStream_t s) {
  const int64_t span = cdiv(plan.span, T::E);     // vectors of a part
  const dim3 grid((unsigned)(p.n * plan.splits));
  if (p.top_k > 0) logprob_kernel<T, true><<<grid, kThreads, 0, s>>>(p, plan.splits, span, ws);
  else logprob_kernel<T, false><<<grid, kThreads, 0, s>>>(p, plan.splits, span, ws);
  if (plan.splits > 1)
    logprob_join_kernel<T><<<dim3((unsigned)p.n), kThreads, (size_t)plan.splits * p.top_k * 16, s>>>(p, plan.splits, ws);
  return hipGetLastError();
}

}  // namespace

// Parts of a row: at least 2048 elements, together some 2048 work-groups (1024 from 128 rows
// on), and as many lists as the join's LDS holds.  The second launch pays from rows of about
// 28 KB on: 1 x 6000 bf16 8.1 us in parts, 6.2 whole, 1 x 20000 8.4 against 8.7; 64 x 6000 fp32
// with 20 top tokens 13.6 against 12.4, 64 x 9000 14.0 against 16.0.  With more rows than CUs
// from longer ones on, 512 rows are enough by themselves: 350 x 16000 bf16 13.5 against 10.8,
// 350 x 50000 19.4 against 20.7, 350 x 128000 29 against 39, 500 x 50000 with 20 40.4 against 37.4.
LogprobPlan logprob_plan(int64_t n, int64_t v, int64_t top_k, int elem_bytes) {
  LogprobPlan p{1, v, 0};
  const int64_t least = (28 << 10) * std::max<int64_t>(1, n / 64 - 2);
  const int64_t want = n >= 512 || v * elem_bytes < least ? 1 : cdiv(n >= 128 ? 1024 : 2048, std::max<int64_t>(n, 1));
  const int64_t most = std::min<int64_t>(std::min<int64_t>(kMaxSplits, 4096 / std::max<int64_t>(top_k, 1)), cdiv(v, 2048));
  p.splits = (int)std::max<int64_t>(1, std::min(want, most));
  p.span = cdiv(v, p.splits);
  if (p.splits > 1) p.ws_bytes = (size_t)n * p.splits * record_words((int)top_k) * 4;
  return p;
}

hipError_t logprob_launch(const LogprobPlan& plan, const LogprobArgs& p, void* ws, hipStream_t s) {
  if (p.dtype == kF32) return launch<F32>(plan, p, (uint32_t*)ws, s);
  if (p.dtype == kF16) return launch<F16>(plan, p, (uint32_t*)ws, s);
  return launch<BF16>(plan, p, (uint32_t*)ws, s);
}

}  // namespace gptq
