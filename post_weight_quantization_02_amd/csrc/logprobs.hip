// Log probability of a given token, entropy and top tokens of every row of logits, in
// one pass over the row.
//
// With M = max x, S = sum e^(x - M) and T = sum e^(x - M) (x - M) <= 0:
//
//   log p(t) = (x_t - M) - log S,    H = log S - T / S.
//
// Both terms of H are non-negative, so a row that is almost certain keeps its small
// entropy to fp32's absolute precision.  A wave keeps one running M; a part's sums
// move to a new M as S' = r S, T' = r (T + d S), d = M - M', r = e^d.  x - M is
// subtracted before anything is multiplied, so a common offset of the logits costs
// nothing.  Sums are fp32, exponentials in base 2 (T in units of log 2).
//
// Top tokens: a wave keeps its best 64 (value, index) pairs sorted, one per lane, and
// a bound g; a vector whose maximum is at most g (all but a few, once the list has
// filled) costs one comparison, which also finds a new M and a NaN.  Before the first
// vector g comes from the K-th largest of the lanes' maxima over the first loads: K
// elements are known to lie at or above it.  Values are ordered as 32-bit keys (NaN
// above +inf, -0 equal to +0); equal values by lower index.
//
// Few rows: a row is split over work-groups, and a second launch joins the parts in
// a fixed order.
#include "gptq_internal.h"

namespace gptq {
namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kUnroll = 4;              // 16-byte vectors per lane and iteration
constexpr int kMaxTop = 64;
constexpr int kMaxSplits = 128;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kFloor = -1e30f;        // stands for -inf in a product with e^-inf = 0
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

struct F32 {
  typedef float elem;
  static constexpr int E = 4;           // elements of a 16-byte vector
  static __device__ float one(elem x) { return x; }
};
struct F16 {
  typedef uint16_t elem;
  static constexpr int E = 8;
  static __device__ float one(elem x) { return (float)__builtin_bit_cast(_Float16, x); }
};
struct BF16 {
  typedef uint16_t elem;
  static constexpr int E = 8;
  static __device__ float one(elem x) { return __builtin_bit_cast(float, (uint32_t)x << 16); }
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

// moves the sums from maximum m to maximum M
__device__ __forceinline__ void rescale(float& s, float& t, float m, float M) {
  if (!(m > -INFINITY)) return;         // nothing summed yet
  const float d = fmaxf((m - M) * kLog2e, kFloor);   // finite also from a mask of the type's lowest value
  const float r = __builtin_amdgcn_exp2f(d);
  t = r * fmaf(d, s, t);
  s *= r;
}

struct Wave {
  float m, s, t;        // s, t per lane; m of the wave
  float g;              // elements at or below g change neither m nor the list
  uint32_t gkey, key;   // key, idx: entry `lane` of the sorted list
  int idx;
};

template <bool TOP, int E>
__device__ __forceinline__ void take(Wave& a, const float (&x)[E], int i0, bool valid, int top_k, int lane) {
  float v = x[0];
#pragma unroll
  for (int e = 1; e < E; ++e) v = fmaximum(v, x[e]);
  if (__any(!(v <= a.g))) {
    if (__any(!(v <= a.m))) {
      const float M = fmaximum(a.m, wave_maximum(v));
      rescale(a.s, a.t, a.m, M);
      a.m = M;
    }
    if constexpr (TOP) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        uint64_t todo = __ballot(valid && !(x[e] <= a.g));
        while (todo) {
          const int l = __builtin_ctzll(todo);
          todo &= todo - 1;
          const uint32_t k = key_of(__builtin_bit_cast(float, lane_value(__builtin_bit_cast(uint32_t, x[e]), l)));
          const int i = (int)lane_value((uint32_t)i0, l) + e;
          const int pos = __popcll(__ballot(a.key > k || (a.key == k && a.idx < i)));
          if (pos >= top_k) continue;
          const uint32_t pk = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a.key, 0x138, 0xf, 0xf, false);
          const int pi = __builtin_amdgcn_update_dpp(0, a.idx, 0x138, 0xf, 0xf, false);
          a.key = lane < pos ? a.key : lane == pos ? k : pk;
          a.idx = lane < pos ? a.idx : lane == pos ? i : pi;
        }
      }
      a.gkey = max(a.gkey, lane_value(a.key, top_k - 1));
      a.g = value_of(a.gkey);
    } else {
      a.g = a.m;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float d = fmaxf((x[e] - a.m) * kLog2e, kFloor);
    const float p = __builtin_amdgcn_exp2f(d);
    a.s += p;
    a.t = fmaf(p, d, a.t);
  }
}

struct Part {
  float m, s, t;
};

// outputs of one row from its joined sums; sorted: the row's top_k entries
template <typename T>
__device__ __forceinline__ void finish(const LogprobArgs& p, int64_t row, Part r, int t, const uint32_t* key,
                                       const int* idx) {
  const float log_s = logf(r.s);
  const bool sound = fabsf(r.m) < INFINITY;      // neither empty nor with +inf or NaN
  if (t < p.top_k) {
    p.top_ids[row * p.top_k + t] = idx[t];
    p.top_logprobs[row * p.top_k + t] = sound ? (value_of(key[t]) - r.m) - log_s : NAN;
  }
  if (t == 0) {
    const int64_t tok = p.tokens[row];
    float lp = 0.f;
    if (tok >= p.v) lp = NAN;
    else if (tok >= 0)
      lp = sound ? (T::one(((const typename T::elem*)p.logits)[row * p.ld + tok]) - r.m) - log_s : NAN;
    p.logprobs[row] = lp;
    p.entropy[row] = sound ? log_s - kLn2 * (r.t / r.s) : NAN;
  }
}

// a part's record in the workspace: m, s, t, unused, then top_k keys and top_k indices
__host__ __device__ inline int64_t record_words(int top_k) { return 4 + 2 * top_k; }

template <typename T, bool TOP>
__global__ __launch_bounds__(kThreads) void logprob_kernel(LogprobArgs p, int splits, int64_t span,
                                                           uint32_t* __restrict__ ws) {
  constexpr int E = T::E;
  __shared__ float ps[kWaves][3];
  __shared__ uint32_t key[kWaves][kMaxTop];
  __shared__ int idx[kWaves][kMaxTop];
  __shared__ uint32_t skey[kMaxTop];
  __shared__ int sidx[kMaxTop];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t row = blockIdx.x / splits;
  const int part = (int)(blockIdx.x % splits);
  const auto* x = (const typename T::elem*)p.logits + row * p.ld;
  const int v = (int)p.v;
  // whole 16-byte vectors [head, head + E * nvec); the elements before and after go one to a lane
  const int head = min(v, (int)(((16 - ((uintptr_t)x & 15)) & 15) / sizeof(typename T::elem)));
  const int nvec = (v - head) / E, tail0 = head + nvec * E;
  const u32x4* xv = (const u32x4*)(x + head);
  Wave a{-INFINITY, 0.f, 0.f, NAN, 0u, 0u, 0x7fffffff};
  if constexpr (!TOP) a.g = -INFINITY;
  if (part == 0 && w == 0 && head > 0) {
    const float one[1] = {lane < head ? T::one(x[lane]) : -INFINITY};
    take<TOP>(a, one, lane, lane < head, p.top_k, lane);
  }
  const int first = (int)min<int64_t>((int64_t)part * span, nvec), last = (int)min<int64_t>(first + span, nvec);
  bool fresh = true;
  for (int b = first + w * (64 * kUnroll); b < last; b += kWaves * 64 * kUnroll) {
    u32x4 ld[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) ld[u] = xv[min(b + 64 * u + lane, last - 1)];
    if (fresh) {
      // the first loads' maximum, and a bound below which no element belongs to the top:
      // the K-th largest lane maximum (at most M, so what g lets pass needs no new M)
      fresh = false;
      float lm = -INFINITY;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        float f[E];
        unpack<T>(ld[u], f);
        if (b + 64 * u + lane < last) {     // a lane past the end holds another lane's vector again
#pragma unroll
          for (int e = 0; e < E; ++e) lm = fmaximum(lm, f[e]);
        }
      }
      const float M = fmaximum(a.m, wave_maximum(lm));
      rescale(a.s, a.t, a.m, M);
      a.m = M;
      if constexpr (TOP) {
        const uint32_t lk = b + lane < last ? key_of(lm) : 0u;
        uint32_t bound = 0u;
#pragma unroll 1
        for (uint32_t bit = 0x80000000u; bit >= 0x1000u; bit >>= 1)
          if (__popcll(__ballot(lk >= (bound | bit))) >= p.top_k) bound |= bit;
        // the largest key below the bound; -0 is no key of its own
        if (bound) bound = bound == 0x80000000u ? 0x7ffffffeu : bound - 1;
        a.gkey = max(a.gkey, bound);
        a.g = value_of(a.gkey);
      } else {
        a.g = M;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = b + 64 * u + lane;
      float f[E];
      unpack<T>(ld[u], f);
      if (i >= last) {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = -INFINITY;
      }
      take<TOP>(a, f, head + i * E, i < last, p.top_k, lane);
    }
  }
  if (part == 0 && w == 0 && tail0 < v) {
    const bool has = tail0 + lane < v;
    const float one[1] = {has ? T::one(x[tail0 + lane]) : -INFINITY};
    take<TOP>(a, one, tail0 + lane, has, p.top_k, lane);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    a.s += __shfl_xor(a.s, o, 64);
    a.t += __shfl_xor(a.t, o, 64);
  }
  if (lane == 0) {
    ps[w][0] = a.m;
    ps[w][1] = a.s;
    ps[w][2] = a.t;
  }
  if (TOP && lane < p.top_k) {
    key[w][lane] = a.key;
    idx[w][lane] = a.idx;
    if (w == 0) {
      skey[lane] = 0u;
      sidx[lane] = 0x7fffffff;
    }
  }
  __syncthreads();
  Part r{ps[0][0], 0.f, 0.f};
#pragma unroll
  for (int i = 1; i < kWaves; ++i) r.m = fmaximum(r.m, ps[i][0]);
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    float s = ps[i][1], q = ps[i][2];
    rescale(s, q, ps[i][0], r.m);
    r.s += s;
    r.t += q;
  }
  if (TOP) {
    // an entry's place among the waves' lists is the number of better ones
    if (lane < p.top_k && a.key != 0u) {
      int rank = 0;
      for (int i = 0; i < kWaves; ++i)
        for (int j = 0; j < p.top_k; ++j) {
          const uint32_t k = key[i][j];
          rank += k > a.key || (k == a.key && idx[i][j] < a.idx);
        }
      if (rank < p.top_k) {
        skey[rank] = a.key;
        sidx[rank] = a.idx;
      }
    }
    __syncthreads();
  }
  if (splits == 1) {
    finish<T>(p, row, r, t, skey, sidx);
    return;
  }
  uint32_t* rec = ws + (int64_t)blockIdx.x * record_words(p.top_k);
  if (t == 0) {
    rec[0] = __builtin_bit_cast(uint32_t, r.m);
    rec[1] = __builtin_bit_cast(uint32_t, r.s);
    rec[2] = __builtin_bit_cast(uint32_t, r.t);
  }
  if (t < p.top_k) {
    rec[4 + t] = skey[t];
    rec[4 + p.top_k + t] = (uint32_t)sidx[t];
  }
}

// one row per work-group: sums joined in the order of the parts; the top tokens by
// taking the best head of the parts' sorted lists top_k times (wave 0, two lists a lane)
template <typename T>
__global__ __launch_bounds__(kThreads) void logprob_join_kernel(LogprobArgs p, int splits,
                                                                const uint32_t* __restrict__ ws) {
  extern __shared__ uint32_t lists[];      // [splits][2 top_k]
  __shared__ uint32_t skey[kMaxTop];
  __shared__ int sidx[kMaxTop];
  const int t = threadIdx.x, lane = t & 63, K = p.top_k;
  const int64_t row = blockIdx.x, words = record_words(K);
  const uint32_t* rec = ws + row * splits * words;
  for (int i = t; i < splits * 2 * K; i += kThreads) lists[i] = rec[(i / (2 * K)) * words + 4 + i % (2 * K)];
  __syncthreads();
  if (t >= 64) return;
  Part r{-INFINITY, 0.f, 0.f};
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
    rescale(own[h].s, own[h].t, own[h].m, r.m);
    r.s += own[h].s;
    r.t += own[h].t;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    r.s += __shfl_xor(r.s, o, 64);
    r.t += __shfl_xor(r.t, o, 64);
  }
  int at[2] = {0, 0};
  for (int j = 0; j < K; ++j) {
    uint64_t best = 0;
    int from = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = lane + 64 * h;
      if (i < splits && at[h] < K) {
        const uint32_t* l = lists + i * 2 * K + at[h];
        const uint64_t c = ((uint64_t)l[0] << 32) | (0xffffffffu - l[K]);
        if (c > best) {
          best = c;
          from = h;
        }
      }
    }
    uint64_t top = best;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const uint64_t c = ((uint64_t)(uint32_t)__shfl_xor((int)(top >> 32), o, 64) << 32) |
                         (uint32_t)__shfl_xor((int)(uint32_t)top, o, 64);
      top = max(top, c);
    }
    if (best == top) ++at[from];       // one lane: indices differ
    if (lane == j) {
      skey[j] = (uint32_t)(top >> 32);
      sidx[j] = (int)(0xffffffffu - (uint32_t)top);
    }
  }
  __builtin_amdgcn_wave_barrier();
  finish<T>(p, row, r, t, skey, sidx);
}

template <typename T>
hipError_t launch(const LogprobPlan& plan, const LogprobArgs& p, uint32_t* ws, hipStream_t s) {
  const int64_t span = cdiv(plan.span, T::E);     // vectors of a part
  const dim3 grid((unsigned)(p.n * plan.splits));
  if (p.top_k > 0) logprob_kernel<T, true><<<grid, kThreads, 0, s>>>(p, plan.splits, span, ws);
  else logprob_kernel<T, false><<<grid, kThreads, 0, s>>>(p, plan.splits, span, ws);
  if (plan.splits > 1)
    logprob_join_kernel<T><<<dim3((unsigned)p.n), kThreads, (size_t)plan.splits * 2 * p.top_k * 4, s>>>(p, plan.splits, ws);
  return hipGetLastError();
}

}  // namespace

LogprobPlan logprob_plan(int64_t n, int64_t v, int64_t top_k) {
  LogprobPlan p{1, v, 0};
  const int64_t want = n >= 1024 ? 1 : cdiv(2048, std::max<int64_t>(n, 1));
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
