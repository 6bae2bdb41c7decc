// Divergence of a row of logits from a teacher that gives its top tokens, and its gradient.
//
// With p = softmax(z / T) over all tokens, q over the listed tokens j (renormalised, or the
// teacher's own probabilities with q_r = 1 - sum q_j for the rest R of the tokens together):
//
//   loss = sum_j q_j (log q_j - log p_j) + q_r (log q_r - log p_r),   Q = sum_j q_j + q_r
//   dloss/dz_j = (Q p_j - q_j) / T,   dloss/dz_v = (Q p_v - q_r p_v / p_r) / T  for v in R
//
// The row's pass gives M = max and S = sum 2^((z - M) c) over R alone, c = log2 e / T: each
// listed token is left out there and has its own term, so p_r is no difference of numbers
// that nearly cancel, and the gradient over R is one multiple of 2^((z - M) c).  Differences
// z - M are taken before they are scaled, so logits far from zero lose nothing.  Elements and
// their sums are fp32; the at most 64 terms of a row's loss, which cancel where the two
// models agree, are combined in 64 bits by one wave.
//
// Which vectors of a row hold listed tokens stands in LDS: a byte for each 16-byte vector,
// the last listed token in it plus one, with a chain through the others.  All but a few
// vectors cost one LDS byte.
#include "gptq_internal.h"

namespace gptq {
namespace {

constexpr int kMaxTop = 64;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLow = -3.402823466e38f;        // the least finite number: -inf less this is -inf
constexpr int kSegment = 16384;                 // vectors whose bytes stand in LDS together
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));

struct F32 {
  typedef float elem;
  static constexpr int E = 4;           // elements of a 16-byte vector
};
struct F16 {
  typedef _Float16 elem;
  static constexpr int E = 8;
};
struct BF16 {
  typedef __bf16 elem;
  static constexpr int E = 8;
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
template <typename T>
__device__ __forceinline__ u32x4 pack(const float (&x)[T::E]) {
  u32x4 v;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (std::is_same<T, F32>::value) v[q] = __builtin_bit_cast(uint32_t, x[q]);
    else if constexpr (std::is_same<T, F16>::value) v[q] = __builtin_bit_cast(uint32_t, h2{(_Float16)x[2 * q], (_Float16)x[2 * q + 1]});
    else v[q] = __builtin_bit_cast(uint32_t, b2{(__bf16)x[2 * q], (__bf16)x[2 * q + 1]});
  }
  return v;
}

__device__ __forceinline__ float fmaximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ int lane_value(int v, int l) { return __builtin_amdgcn_readlane(v, l); }
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
__device__ __forceinline__ float wave_maximum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaximum(v, __shfl_xor(v, o, 64));
  return v;
}

// maximum and sum over a part of the rest
struct Sum {
  float m, s;
};
__device__ __forceinline__ Sum join(Sum a, Sum b, float c) {
  const float m = fmaximum(a.m, b.m);
  return Sum{m, a.s * __builtin_amdgcn_exp2f((a.m - m) * c) + b.s * __builtin_amdgcn_exp2f((b.m - m) * c)};
}

// A row as whole vectors and the elements behind them, each of which has a place of its own:
// place i < nvec is vector i, place nvec + e is element nvec E + e.
template <typename T>
struct Row {
  const typename T::elem* x;
  int v, nvec;
  __device__ __forceinline__ Row(const DistillArgs& p, int64_t row)
      : x((const typename T::elem*)p.logits + row * p.ld), v((int)p.v), nvec((int)p.v / T::E) {}
  __device__ __forceinline__ int places() const { return nvec + v - nvec * T::E; }
  __device__ __forceinline__ int place(int id) const { return id < nvec * T::E ? id / T::E : nvec + id - nvec * T::E; }
  __device__ __forceinline__ int element(int id) const { return id < nvec * T::E ? id % T::E : 0; }
  __device__ __forceinline__ u32x4 load(int i) const { return *(const u32x4_any*)(x + (int64_t)i * T::E); }
};

// The listed tokens of a row: lane j of a wave has token j.
struct Listed {
  int id;               // negative: none
  float z, t;           // its logit, and the teacher's value
  bool out;             // some token of the row is not below v
  bool any;             // some token is there
  bool first;           // no earlier one is the same token
};

// What a work-group knows of the listed tokens.
template <int PLACES>
struct Shared {
  uint8_t head[PLACES];
  int place[kMaxTop], element[kMaxTop], next[kMaxTop];      // next: the chain, 0 at its end
  float grad[kMaxTop];
  bool last[kMaxTop];   // the last one at its place
};

template <typename T, int PLACES>
__device__ __forceinline__ Listed read_listed(const DistillArgs& p, const Row<T>& r, int64_t row, int lane, Shared<PLACES>& sh) {
  Listed l{-1, 0.f, -INFINITY, false, false, true};
  if (lane < p.top) {
    l.id = p.ids[row * p.top + lane];
    l.t = p.logprobs[row * p.top + lane];
  }
  l.out = __any(l.id >= r.v);
  l.any = __any(l.id >= 0);
  if (l.id >= r.v) l.id = -1;
  if (l.id >= 0) l.z = (float)r.x[l.id];
  const int place = l.id >= 0 ? r.place(l.id) : -1;
  int next = 0;
  bool last = l.id >= 0;
  for (int i = 0; i < p.top; ++i) {
    const int other = lane_value(place, i);
    if (other == place) {
      if (i < lane) next = i + 1;
      if (i > lane) last = false;
    }
    if (lane_value(l.id, i) == l.id && i < lane) l.first = false;
  }
  sh.place[lane] = place;
  sh.element[lane] = l.id >= 0 ? r.element(l.id) : 0;
  sh.next[lane] = next;
  sh.last[lane] = last;
  return l;
}

// head[i] for the places [first, last): every thread of the work-group takes part
template <int THREADS, int PLACES>
__device__ __forceinline__ void mark(Shared<PLACES>& sh, int first, int last) {
  static_assert(PLACES % 4 == 0, "cleared in words");
  const int t = threadIdx.x;
  __syncthreads();              // the list is there, and nobody reads the places before
  for (int i = t; i < (last - first + 3) / 4; i += THREADS) ((uint32_t*)sh.head)[i] = 0u;
  __syncthreads();
  if (t < kMaxTop && sh.last[t] && sh.place[t] >= first && sh.place[t] < last) sh.head[sh.place[t] - first] = (uint8_t)(t + 1);
  __syncthreads();
}

// puts value(j) in the place of each listed token j of a vector
template <typename T, int PLACES, typename F>
__device__ __forceinline__ void replace(const Shared<PLACES>& sh, int head, float (&x)[T::E], F&& value) {
  while (head != 0) {
    const int j = head - 1, at = sh.element[j];
    const float v = value(j);
#pragma unroll
    for (int e = 0; e < T::E; ++e) x[e] = e == at ? v : x[e];
    head = sh.next[j];
  }
}

// adds up to N vectors, of which `heads` hold listed tokens, to a thread's sums
template <typename T, int N, int PLACES>
__device__ __forceinline__ void add(Sum& a, const u32x4* ld, const int* heads, const Shared<PLACES>& sh, float c) {
  float f[N][T::E], m = a.m;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    unpack<T>(ld[u], f[u]);
    if (heads[u] != 0) replace<T>(sh, heads[u], f[u], [](int) { return -INFINITY; });
#pragma unroll
    for (int e = 0; e < T::E; ++e) m = fmaximum(m, f[u][e]);
  }
  float s = a.s * __builtin_amdgcn_exp2f((a.m - m) * c);
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int e = 0; e < T::E; ++e) s += __builtin_amdgcn_exp2f((f[u][e] - m) * c);
  a = Sum{m, s};
}

// an element alone
template <int PLACES>
__device__ __forceinline__ void add_one(Sum& a, float x, int head, float c) {
  if (head == 0) a = join(a, Sum{fmaximum(x, kLow), x > -INFINITY || x != x ? 1.f : 0.f}, c);
}

template <int THREADS>
__device__ __forceinline__ Sum over_threads(Sum a, float c) {
  __shared__ Sum part[THREADS / 64];
  const int t = threadIdx.x;
  const float m = wave_maximum(a.m);
  float s = a.s * __builtin_amdgcn_exp2f((a.m - m) * c);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  if ((t & 63) == 0) part[t >> 6] = Sum{m, s};
  __syncthreads();
  Sum r{kLow, 0.f};
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) r.m = fmaximum(r.m, part[i].m);
#pragma unroll
  for (int i = 0; i < THREADS / 64; ++i) r.s += part[i].s * __builtin_amdgcn_exp2f((part[i].m - r.m) * c);
  return r;
}

// What the gradient of a row's rest is: factor * 2^((z - m) c), or the same for all
struct Rest {
  float factor, m;
  bool constant;
};

// The row's loss and gradient from its sums, by one wave.  Rows without a teacher token have
// loss and gradient 0, rows of weight 0 gradient 0, whatever their logits are.
template <int PLACES>
__device__ __forceinline__ Rest finish(const DistillArgs& p, int64_t row, const Listed& l, Sum r, bool store, Shared<PLACES>& sh) {
  const int lane = threadIdx.x & 63;
  const double inv = 1.0 / (double)p.temperature;
  const bool there = l.id >= 0;
  // the teacher
  double lq, q, rest = 0.0, mass = 1.0, sum;
  if (p.tail) {
    lq = there ? (double)l.t : -INFINITY;
    q = there ? exp(lq) : 0.0;
    sum = wave_sum(q);
    rest = sum < 1.0 ? 1.0 - sum : 0.0;
    mass = sum + rest;
  } else {
    const float top = wave_maximum(there ? l.t : -INFINITY);
    lq = there ? (double)(l.t - top) * inv : -INFINITY;
    q = there ? exp(lq) : 0.0;
    sum = wave_sum(q);
    q /= sum;
    lq -= log(sum);
  }
  // the student
  const float m = fmaximum(r.m, wave_maximum(there ? l.z : -INFINITY));
  const double dz = ((double)l.z - (double)m) * inv, dr = ((double)r.m - (double)m) * inv;
  const double u = there ? exp(dz) : 0.0, ur = exp(dr);
  const double total = (double)r.s * ur + wave_sum(there && l.first ? u : 0.0);
  const double log_total = log(total);
  double term = there && q != 0.0 ? q * (lq - (dz - log_total)) : 0.0;
  term = wave_sum(term);
  if (rest > 0.0) term += rest * (log(rest) - (dr + log((double)r.s) - log_total));
  const bool bad = l.out || !(fabsf(m) < INFINITY) || !(total > 0.0) || !(sum < INFINITY);
  if (store && lane == 0) p.loss[row] = l.out ? NAN : !l.any ? 0.f : bad ? NAN : (float)term;
  if (!p.grad) return Rest{0.f, 0.f, true};
  const double w = (p.weights ? (double)p.weights[row] : 1.0) * inv;
  if (w == 0.0 || (!l.any && !l.out) || bad) {
    const float all = w == 0.0 || (!l.any && !l.out) ? 0.f : NAN;
    sh.grad[lane] = all;
    return Rest{all, 0.f, true};
  }
  double given = 0.0;           // by all entries of this token
  for (int i = 0; i < p.top; ++i) {
    const uint64_t b = __builtin_bit_cast(uint64_t, q);
    const uint64_t o = ((uint64_t)(uint32_t)lane_value((int)(b >> 32), i) << 32) | (uint32_t)lane_value((int)(uint32_t)b, i);
    if (lane_value(l.id, i) == l.id) given += __builtin_bit_cast(double, o);
  }
  sh.grad[lane] = (float)(w * (mass * u / total - given));
  const double others = rest > 0.0 ? rest / (double)r.s : 0.0;
  return Rest{(float)(w * (mass * ur / total - others)), r.m, false};
}

// the gradient of a vector
template <typename T, int PLACES>
__device__ __forceinline__ u32x4 gradient(u32x4 ld, int head, Rest g, const Shared<PLACES>& sh, float c) {
  float f[T::E];
  unpack<T>(ld, f);
#pragma unroll
  for (int e = 0; e < T::E; ++e) f[e] = g.constant ? g.factor : g.factor * __builtin_amdgcn_exp2f((f[e] - g.m) * c);
  if (head != 0) replace<T>(sh, head, f, [&](int j) { return sh.grad[j]; });
  return pack<T>(f);
}
template <typename T>
__device__ __forceinline__ typename T::elem gradient_one(typename T::elem x, Rest g, float c) {
  return (typename T::elem)(g.constant ? g.factor : g.factor * __builtin_amdgcn_exp2f(((float)x - g.m) * c));
}

constexpr int kThreads = 256, kUnroll = 4;

// sums of the rest over the places [first, last) of a row
template <typename T>
__device__ __forceinline__ Sum stream_sums(const Row<T>& r, int first, int last, float c, Shared<kSegment>& sh) {
  const int t = threadIdx.x;
  Sum a{kLow, 0.f};
  for (int lo = first; lo < last; lo += kSegment) {
    const int hi = min(lo + kSegment, last), vec = min(hi, r.nvec);
    mark<kThreads>(sh, lo, hi);
    for (int b = lo + t; b < vec; b += kThreads * kUnroll) {
      u32x4 ld[kUnroll];
      int heads[kUnroll];
      if (b + kThreads * (kUnroll - 1) < vec) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          ld[u] = r.load(b + kThreads * u);
          heads[u] = sh.head[b + kThreads * u - lo];
        }
        add<T, kUnroll>(a, ld, heads, sh, c);
      } else {
        for (int i = b; i < vec; i += kThreads) {
          ld[0] = r.load(i);
          heads[0] = sh.head[i - lo];
          add<T, 1>(a, ld, heads, sh, c);
        }
      }
    }
    for (int i = max(lo, r.nvec) + t; i < hi; i += kThreads)
      add_one<kSegment>(a, (float)r.x[r.nvec * T::E + i - r.nvec], sh.head[i - lo], c);
  }
  return a;
}

// the gradient over the places [first, last)
template <typename T>
__device__ __forceinline__ void stream_grad(const DistillArgs& p, int64_t row, const Row<T>& r, int first, int last, Rest g,
                                            float c, Shared<kSegment>& sh) {
  const int t = threadIdx.x;
  auto* out = (typename T::elem*)p.grad + row * p.ld_grad;
  for (int lo = first; lo < last; lo += kSegment) {
    const int hi = min(lo + kSegment, last), vec = min(hi, r.nvec);
    mark<kThreads>(sh, lo, hi);
    for (int i = lo + t; i < vec; i += kThreads)
      *(u32x4_any*)(out + (int64_t)i * T::E) = gradient<T>(r.load(i), sh.head[i - lo], g, sh, c);
    for (int i = max(lo, r.nvec) + t; i < hi; i += kThreads) {
      const int e = r.nvec * T::E + i - r.nvec, h = sh.head[i - lo];
      out[e] = h != 0 ? (typename T::elem)sh.grad[h - 1] : gradient_one<T>(r.x[e], g, c);
    }
  }
}

// one work-group per row
template <typename T, bool GRAD>
__global__ __launch_bounds__(kThreads) void distill_row_kernel(DistillArgs p) {
  __shared__ Shared<kSegment> sh;
  __shared__ Rest rest;
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const float c = kLog2e / p.temperature;
  const Row<T> r(p, row);
  Listed l{};
  if (t < 64) l = read_listed<T>(p, r, row, t, sh);
  const Sum a = over_threads<kThreads>(stream_sums<T>(r, 0, r.places(), c, sh), c);
  if (t < 64) {
    const Rest g = finish(p, row, l, a, true, sh);
    if (t == 0) rest = g;
  }
  if constexpr (GRAD) {
    __syncthreads();
    stream_grad<T>(p, row, r, 0, r.places(), rest, c, sh);
  }
}

// a part of a row per work-group: its sums ...
template <typename T>
__global__ __launch_bounds__(kThreads) void distill_part_kernel(DistillArgs p, int splits, int span, Sum* __restrict__ parts) {
  __shared__ Shared<kSegment> sh;
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x / splits;
  const float c = kLog2e / p.temperature;
  const Row<T> r(p, row);
  if (t < 64) read_listed<T>(p, r, row, t, sh);
  const int part = (int)(blockIdx.x % splits), first = part * span, last = part == splits - 1 ? r.places() : first + span;
  const Sum a = over_threads<kThreads>(stream_sums<T>(r, first, last, c, sh), c);
  if (t == 0) parts[blockIdx.x] = a;
}

// ... and, when all are there, its gradient; the first one writes the loss
template <typename T, bool GRAD>
__global__ __launch_bounds__(kThreads) void distill_join_kernel(DistillArgs p, int splits, int span, const Sum* __restrict__ parts) {
  __shared__ Shared<kSegment> sh;
  __shared__ Rest rest;
  const int t = threadIdx.x;
  const int64_t row = GRAD ? blockIdx.x / splits : blockIdx.x;
  const int part = GRAD ? (int)(blockIdx.x % splits) : 0;
  const float c = kLog2e / p.temperature;
  const Row<T> r(p, row);
  if (t < 64) {
    const Listed l = read_listed<T>(p, r, row, t, sh);
    Sum a{kLow, 0.f};
    for (int i = t; i < splits; i += 64) a = join(a, parts[row * splits + i], c);
    const float m = wave_maximum(a.m);
    a.s *= __builtin_amdgcn_exp2f((a.m - m) * c);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) a.s += __shfl_xor(a.s, o, 64);
    const Rest g = finish(p, row, l, Sum{m, a.s}, part == 0, sh);
    if (t == 0) rest = g;
  }
  if constexpr (GRAD) {
    __syncthreads();
    const int first = part * span, last = part == splits - 1 ? r.places() : first + span;
    stream_grad<T>(p, row, r, first, last, rest, c, sh);
  }
}

template <typename T>
hipError_t launch(const DistillPlan& plan, const DistillArgs& p, void* ws, hipStream_t s) {
  const unsigned n = (unsigned)p.n;
  if (plan.splits == 1) {
    if (p.grad) distill_row_kernel<T, true><<<n, kThreads, 0, s>>>(p);
    else distill_row_kernel<T, false><<<n, kThreads, 0, s>>>(p);
    return hipGetLastError();
  }
  const int span = (int)(plan.span / T::E);
  Sum* parts = (Sum*)ws;
  distill_part_kernel<T><<<n * plan.splits, kThreads, 0, s>>>(p, plan.splits, span, parts);
  if (p.grad) distill_join_kernel<T, true><<<n * plan.splits, kThreads, 0, s>>>(p, plan.splits, span, parts);
  else distill_join_kernel<T, false><<<n, kThreads, 0, s>>>(p, plan.splits, span, parts);
  return hipGetLastError();
}

}  // namespace

// Parts of a row: at least 2048 elements each, together some 1024 work-groups.
DistillPlan distill_plan(int64_t n, int64_t v, int elem_bytes, bool grad) {
  DistillPlan p{1, v, 0};
  const int64_t want = n >= 512 ? 1 : cdiv(1024, std::max<int64_t>(n, 1));
  p.splits = (int)std::max<int64_t>(1, std::min(want, cdiv(v, 2048)));
  if (p.splits > 1) {
    p.span = cdiv(cdiv(v, p.splits), 8) * 8;
    p.splits = (int)cdiv(v, p.span);
    p.ws_bytes = (size_t)n * p.splits * 8;
  }
  return p;
}

hipError_t distill_launch(const DistillPlan& plan, const DistillArgs& p, void* ws, hipStream_t s) {
  if (p.dtype == kF32) return launch<F32>(plan, p, ws, s);
  if (p.dtype == kF16) return launch<F16>(plan, p, ws, s);
  return launch<BF16>(plan, p, ws, s);
}

}  // namespace gptq
