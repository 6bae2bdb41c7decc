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
// models agree, and the teacher's shares are worked out in 64 bits by one wave.
//
// Which vectors of a row hold listed tokens stands in LDS: a byte for each 16-byte vector,
// the last listed token in it plus one, with a chain through the others.  All but a few
// vectors cost one LDS byte.  What of the listed tokens does not depend on the others is
// worked out while the row is on its way; after its sums no step crosses lanes any more.
//
// HBM-bound on long texts: the gradient's row stays in registers between its two passes (1024
// threads hold 256 KB; of a longer row the rest is read again), so 4096 x 65536 bf16 takes 220
// us, 4.9 TB/s of the 5.15 that a large copy reaches (read twice: 259), 8192 x 32000 209, 1000 x
// 128000 fp32 209 (298); the loss alone of 4096 x 65536 106 us, 5.0 TB/s.  The forms of 16 vectors a
// thread are held to 128 registers, four waves a SIMD, and spill a few: fp32 4 to 8 (20 bytes of
// scratch a thread), 16-bit types 16 (36 bytes) with 256 and 512 threads, 4 or 5 (20 to 24) with 1024;
// those of 4 and 8 vectors spill none.  517 x 50001 fp32
// with 32 tokens 58 us: two rows per CU, and five rows more that cost 11 of them.  Few
// short rows: a launch, and the chain of loads (ids, their logits), sums and logarithms: 5 us
// for the loss, 8 with the gradient.
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
  static constexpr uint32_t kNone = 0xff800000u;      // a word of -inf
};
struct F16 {
  typedef _Float16 elem;
  static constexpr int E = 8;
  static constexpr uint32_t kNone = 0xfc00fc00u;
};
struct BF16 {
  typedef __bf16 elem;
  static constexpr int E = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;
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
// a lane's v from a lane of its 16, `CTRL` lanes further (0x121: one, 0x122: two, ...)
template <int CTRL>
__device__ __forceinline__ float rotated(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ double rotated(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ float lane_value(float v, int l) {
  return __builtin_bit_cast(float, lane_value(__builtin_bit_cast(int, v), l));
}
__device__ __forceinline__ double lane_value(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, ((uint64_t)(uint32_t)lane_value((int)(b >> 32), l) << 32) | (uint32_t)lane_value((int)(uint32_t)b, l));
}
// over the 64 lanes, the same in all of them, in one order whatever the values
template <typename V, typename F>
__device__ __forceinline__ V over_wave(V v, F&& f) {
  v = f(v, rotated<0x128>(v));
  v = f(v, rotated<0x124>(v));
  v = f(v, rotated<0x122>(v));
  v = f(v, rotated<0x121>(v));
  return f(f(lane_value(v, 0), lane_value(v, 16)), f(lane_value(v, 32), lane_value(v, 48)));
}
template <typename V>
__device__ __forceinline__ V wave_sum(V v) {
  return over_wave(v, [](V a, V b) { return a + b; });
}
__device__ __forceinline__ float wave_maximum(float v) { return over_wave(v, [](float a, float b) { return fmaximum(a, b); }); }

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

// What is known of a row's listed tokens before its sums are.
struct Listed {
  bool out, any;        // some token is not below v, is there
  bool sound;           // the teacher's values are
  float m;              // the maximum of their logits
  double sum_u;         // e^((z - m) / T) over the tokens
  double sum_q, terms;  // over the entries: q, and q (log q - (z - m) / T)
  double rest, mass;    // q_r, Q
};

// What a work-group knows of them: in LDS, as the sums need the registers.
template <int PLACES>
struct Shared {
  uint8_t head[PLACES];
  int place[kMaxTop], element[kMaxTop], next[kMaxTop];      // next: the chain, 0 at its end
  float grad[kMaxTop];
  double u[kMaxTop], given[kMaxTop];    // e^((z - m) / T), and the teacher's share of the token
  bool last[kMaxTop];   // the last one at its place
  Listed listed;
};

// Reads them, by one wave: lane j has token j.  Everything that does not depend on the row's
// other tokens is taken here, while the row is on its way (ALL), or only where they are.
// Every lane gets what finish needs of it; one lane leaves it in LDS too, for the kernels that
// have a barrier before finish and would rather have the registers meanwhile.
template <bool ALL, typename T, int PLACES>
__device__ __forceinline__ Listed read_listed(const DistillArgs& p, const Row<T>& r, int64_t row, int lane, Shared<PLACES>& sh) {
  Listed l;
  int id = -1;
  float t = -INFINITY, z = -INFINITY;
  if (lane < p.top) {
    id = p.ids[row * p.top + lane];
    t = p.logprobs[row * p.top + lane];
  }
  l.out = __any(id >= r.v);
  l.any = __any(id >= 0);
  if (id >= r.v) id = -1;
  const bool there = id >= 0;
  if (there) z = (float)r.x[id];
  else t = -INFINITY;
  const int place = there ? r.place(id) : -1;
  // two at one place, as good as never: chained, and the same token's entries joined
  bool met = false;
  int other = place;
  for (int i = 1; i < p.top; ++i) {
    other = __builtin_amdgcn_update_dpp(0, other, 0x13c, 0xf, 0xf, true);      // of the lane i before
    met |= other == place;
  }
  // the teacher
  const double inv = 1.0 / (double)p.temperature;
  double lq = 0.0, q = 0.0;
  l.rest = 0.0;
  l.mass = 1.0;
  if (!ALL) {
  } else if (p.tail) {
    lq = (double)t;
    q = there ? exp(lq) : 0.0;
    l.sum_q = wave_sum(q);
    l.rest = l.sum_q < 1.0 ? 1.0 - l.sum_q : 0.0;
    l.mass = l.sum_q + l.rest;
    l.sound = l.sum_q < INFINITY;
  } else {
    const float top = wave_maximum(t);
    lq = ((double)t - (double)top) * inv;
    q = there ? exp(lq) : 0.0;
    const double sum = wave_sum(q);
    q /= sum;
    lq -= log(sum);
    l.sum_q = 1.0;
    l.sound = sum < INFINITY;
  }
  double given = q;
  int next = 0;
  bool last = there, first = there;
  if (__any(met && there)) {
    given = 0.0;
    for (int i = 0; i < p.top; ++i) {
      const bool same = lane_value(id, i) == id;
      const double o = lane_value(q, i);
      if (lane_value(place, i) == place) {
        if (i < lane) next = i + 1;
        if (i > lane) last = false;
      }
      if (same && i < lane) first = false;
      if (same) given += o;
    }
  }
  sh.place[lane] = place;
  sh.element[lane] = there ? r.element(id) : 0;
  sh.next[lane] = next;
  sh.last[lane] = last;
  if (!ALL) return l;
  // the student
  l.m = fmaximum(wave_maximum(z), kLow);
  const double d = ((double)z - (double)l.m) * inv;
  const double u = there ? exp(d) : 0.0;
  l.sum_u = wave_sum(first ? u : 0.0);
  l.terms = wave_sum(there && q != 0.0 ? q * (lq - d) : 0.0);
  sh.u[lane] = u;
  sh.given[lane] = given;
  if (lane == 0) sh.listed = l;
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
__device__ __forceinline__ void add_one(Sum& a, float x, int head, float c) {
  if (head == 0) a = join(a, Sum{fmaximum(x, kLow), x > -INFINITY || x != x ? 1.f : 0.f}, c);
}

template <int THREADS>
__device__ __forceinline__ Sum over_threads(Sum a, float c) {
  __shared__ Sum part[THREADS / 64];
  const int t = threadIdx.x;
  const float m = wave_maximum(a.m);
  const float s = wave_sum(a.s * __builtin_amdgcn_exp2f((a.m - m) * c));
  if constexpr (THREADS == 64) return Sum{m, s};
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

// The row's loss and gradient from its sums, by one wave.  With m the larger of the two
// maxima, log p_j = (z_j - m) / T - log total, so the terms of the listed tokens are those
// taken before, moved from their own maximum to m.  Rows without a teacher token have loss and
// gradient 0, rows of weight 0 gradient 0, whatever their logits are.
template <int PLACES>
__device__ __forceinline__ Rest finish(const DistillArgs& p, int64_t row, Listed l, Sum r, bool store, Shared<PLACES>& sh) {
  const int lane = threadIdx.x & 63;
  const double inv = 1.0 / (double)p.temperature;
  const float m = fmaximum(r.m, l.m);
  const double dl = ((double)l.m - (double)m) * inv, dr = ((double)r.m - (double)m) * inv;
  const double ul = exp(dl), ur = exp(dr);
  const double total = (double)r.s * ur + l.sum_u * ul, log_total = log(total);
  double loss = l.terms + l.sum_q * (log_total - dl);
  if (l.rest > 0.0) loss += l.rest * (log(l.rest) - (dr + log((double)r.s) - log_total));
  const bool bad = l.out || !(fabsf(m) < INFINITY) || !(total > 0.0) || !l.sound, none = !l.any;
  if (store && lane == 0) p.loss[row] = none ? 0.f : bad ? NAN : (float)loss;
  if (!p.grad) return Rest{0.f, 0.f, true};
  const double w = (p.weights ? (double)p.weights[row] : 1.0) * inv;
  if (none || bad || w == 0.0) {
    const float all = none || w == 0.0 ? 0.f : NAN;
    sh.grad[lane] = all;
    return Rest{all, 0.f, true};
  }
  sh.grad[lane] = (float)(w * (l.mass * sh.u[lane] * ul / total - sh.given[lane]));
  const double others = l.rest > 0.0 ? l.rest / (double)r.s : 0.0;
  return Rest{(float)(w * (l.mass * ur / total - others)), r.m, false};
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

constexpr int kThreads = 256, kUnroll = 4;     // of a part; vectors under way per thread

// sums of the rest over the places [first, last) of a row
template <int THREADS, typename T>
__device__ __forceinline__ Sum stream_sums(const Row<T>& r, int first, int last, float c, Shared<kSegment>& sh) {
  const int t = threadIdx.x;
  Sum a{kLow, 0.f};
  for (int lo = first; lo < last; lo += kSegment) {
    const int hi = min(lo + kSegment, last), vec = min(hi, r.nvec);
    mark<THREADS>(sh, lo, hi);
    for (int b = lo + t; b < vec; b += THREADS * kUnroll) {
      u32x4 ld[kUnroll];
      int heads[kUnroll];
      if (b + THREADS * (kUnroll - 1) < vec) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          ld[u] = r.load(b + THREADS * u);
          heads[u] = sh.head[b + THREADS * u - lo];
        }
        add<T, kUnroll>(a, ld, heads, sh, c);
      } else {
        for (int i = b; i < vec; i += THREADS) {
          ld[0] = r.load(i);
          heads[0] = sh.head[i - lo];
          add<T, 1>(a, ld, heads, sh, c);
        }
      }
    }
    for (int i = max(lo, r.nvec) + t; i < hi; i += THREADS)
      add_one(a, (float)r.x[r.nvec * T::E + i - r.nvec], sh.head[i - lo], c);
  }
  return a;
}

// the gradient over the places [first, last)
template <int THREADS, typename T>
__device__ __forceinline__ void stream_grad(const DistillArgs& p, int64_t row, const Row<T>& r, int first, int last, Rest g,
                                            float c, Shared<kSegment>& sh) {
  const int t = threadIdx.x;
  auto* out = (typename T::elem*)p.grad + row * p.ld_grad;
  for (int lo = first; lo < last; lo += kSegment) {
    const int hi = min(lo + kSegment, last), vec = min(hi, r.nvec);
    mark<THREADS>(sh, lo, hi);
    for (int b = lo + t; b < vec; b += THREADS * kUnroll) {
      u32x4 ld[kUnroll];
      int heads[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = min(b + THREADS * u, vec - 1);
        ld[u] = r.load(i);
        heads[u] = sh.head[i - lo];
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = b + THREADS * u;
        const u32x4 o = gradient<T>(ld[u], heads[u], g, sh, c);
        if (i < vec) __builtin_nontemporal_store(o, (u32x4_any*)(out + (int64_t)i * T::E));
      }
    }
    for (int i = max(lo, r.nvec) + t; i < hi; i += THREADS) {
      const int e = r.nvec * T::E + i - r.nvec, h = sh.head[i - lo];
      out[e] = h != 0 ? (typename T::elem)sh.grad[h - 1] : gradient_one<T>(r.x[e], g, c);
    }
  }
}

// a row per work-group, read from memory for its sums and again for its gradient
template <typename T, int THREADS, bool GRAD>
__global__ __launch_bounds__(THREADS) void distill_row_kernel(DistillArgs p) {
  __shared__ Shared<kSegment> sh;
  __shared__ Rest rest;
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const float c = kLog2e / p.temperature;
  const Row<T> r(p, row);
  if (t < 64) read_listed<true>(p, r, row, t, sh);
  const Sum a = over_threads<THREADS>(stream_sums<THREADS>(r, 0, r.places(), c, sh), c);
  if (t < 64) {
    const Rest g = finish(p, row, sh.listed, a, true, sh);
    if (t == 0) rest = g;
  }
  if constexpr (GRAD) {
    __syncthreads();
    stream_grad<THREADS>(p, row, r, 0, r.places(), rest, c, sh);
  }
}

// A row per work-group, kept in its registers (but for a few spilled ones): read once, written once.  MORE > 0: a longer
// row, of which up to MORE vectors are read again, the last ones first.
template <typename T, int VPT, int THREADS, int MORE>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(VPT == 16 ? 4 : VPT == 8 ? 5 : 6))) void
distill_held_kernel(DistillArgs p) {
  constexpr int kHeld = VPT * THREADS;
  __shared__ Shared<kHeld + MORE + 16> sh;
  __shared__ Rest rest;
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const float c = kLog2e / p.temperature;
  const Row<T> r(p, row);
  u32x4 ld[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u)
    ld[u] = __builtin_nontemporal_load((const u32x4_any*)(r.x + (int64_t)min(t + u * THREADS, r.nvec - 1) * T::E));
  if (t < 64) read_listed<true>(p, r, row, t, sh);
  mark<THREADS>(sh, 0, r.places());
  Sum a{kLow, 0.f};
  constexpr int kStep = 2;
#pragma unroll
  for (int u0 = 0; u0 < VPT; u0 += kStep) {
    if (u0 * THREADS >= r.nvec) break;
    int heads[kStep];
#pragma unroll
    for (int u = 0; u < kStep; ++u) {
      const int i = t + (u0 + u) * THREADS;
      if (i >= r.nvec) ld[u0 + u] = u32x4{T::kNone, T::kNone, T::kNone, T::kNone};
      heads[u] = i < r.nvec ? sh.head[i] : 0;
    }
    add<T, kStep>(a, ld + u0, heads, sh, c);
  }
  const int behind = kHeld + (r.nvec - kHeld) / (2 * THREADS) * (2 * THREADS);      // no whole step from here on
  if constexpr (MORE > 0) {
    for (int i = kHeld + t; i < r.nvec; i += 2 * THREADS) {
      const u32x4 two[2] = {r.load(i), r.load(min(i + THREADS, r.nvec - 1))};
      const int heads[2] = {sh.head[i], sh.head[min(i + THREADS, r.nvec - 1)]};
      if (i + THREADS < r.nvec) add<T, 2>(a, two, heads, sh, c);
      else add<T, 1>(a, two, heads, sh, c);
    }
  }
  const int e = r.nvec * T::E + t;
  int head = 0;
  float x = 0.f;
  if (e < r.v) {
    x = (float)r.x[e];
    head = sh.head[r.nvec + t];
    add_one(a, x, head, c);
  }
  const Sum sum = over_threads<THREADS>(a, c);
  if (t < 64) {
    const Rest g = finish(p, row, sh.listed, sum, true, sh);
    if (t == 0) rest = g;
  }
  __syncthreads();
  const Rest g = rest;
  auto* out = (typename T::elem*)p.grad + row * p.ld_grad;
  if constexpr (MORE > 0) {
    for (int i = behind + t; i >= kHeld; i -= 2 * THREADS) {
      const u32x4 two[2] = {r.load(min(i, r.nvec - 1)), r.load(min(i + THREADS, r.nvec - 1))};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int at = i + u * THREADS;
        if (at < r.nvec)
          __builtin_nontemporal_store(gradient<T>(two[u], sh.head[at], g, sh, c), (u32x4_any*)(out + (int64_t)at * T::E));
      }
    }
  }
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int i = t + u * THREADS;
    if (i < r.nvec)
      __builtin_nontemporal_store(gradient<T>(ld[u], sh.head[i], g, sh, c), (u32x4_any*)(out + (int64_t)i * T::E));
  }
  if (e < r.v) out[e] = head != 0 ? (typename T::elem)sh.grad[head - 1] : (typename T::elem)(g.constant ? g.factor : g.factor * __builtin_amdgcn_exp2f((x - g.m) * c));
}

// a part of a row per work-group: its sums ...
template <typename T>
__global__ __launch_bounds__(kThreads) void distill_part_kernel(DistillArgs p, int splits, int span, Sum* __restrict__ parts) {
  __shared__ Shared<kSegment> sh;
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x / splits;
  const float c = kLog2e / p.temperature;
  const Row<T> r(p, row);
  if (t < 64) read_listed<false>(p, r, row, t, sh);
  const int part = (int)(blockIdx.x % splits), first = part * span, last = part == splits - 1 ? r.places() : first + span;
  const Sum a = over_threads<kThreads>(stream_sums<kThreads>(r, first, last, c, sh), c);
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
    const Listed l = read_listed<true>(p, r, row, t, sh);      // kept: no barrier stands between
    Sum a{kLow, 0.f};
    for (int i = t; i < splits; i += 64) a = join(a, parts[row * splits + i], c);
    const float m = wave_maximum(a.m);
    const float sum = wave_sum(a.s * __builtin_amdgcn_exp2f((a.m - m) * c));
    const Rest g = finish(p, row, l, Sum{m, sum}, part == 0, sh);
    if (t == 0) rest = g;
  }
  if constexpr (GRAD) {
    __syncthreads();
    const int first = part * span, last = part == splits - 1 ? r.places() : first + span;
    stream_grad<kThreads>(p, row, r, first, last, rest, c, sh);
  }
}

template <typename T>
hipError_t launch(const DistillPlan& plan, const DistillArgs& p, void* ws, hipStream_t s) {
  const unsigned n = (unsigned)p.n;
  const int nvec = (int)(p.v / T::E);
  // The smallest work-group and least registers that hold the row (8192 x 1500 bf16: 27 us by a
  // wave, 40 by four; 4096 x 64000 221 by 512 threads, 262 by 1024), twice the threads where each
  // row has a CU to itself (256 x 32001 bf16 17.3 us by 512, 20.8 by 256; 256 x 64000 22.1 by 1024,
  // 24.8 by 512).  A row for 1024 threads leaves its CU no other one to read while it writes:
  // beyond a row per CU it goes to 512 that read up to 5120 vectors again (300 x 50001 fp32,
  // 12500 vectors, 36 us against 41, 1030 rows 93 against 103, 4096 x 45000 315 against 322; but
  // 2000 x 56000, 14000 vectors, 188 against 182, and 256 x 50001 30 against 27.5).
  const bool alone = p.n <= 256;
  if (plan.splits == 1 && p.grad && nvec > 0 && nvec <= 65536) {
    const auto go = [&](auto vpt, auto threads, auto more) {
      distill_held_kernel<T, vpt.value, threads.value, more.value><<<n, threads.value, 0, s>>>(p);
    };
    using std::integral_constant;
    constexpr integral_constant<int, 0> none;
    if (nvec <= 256) go(integral_constant<int, 4>{}, integral_constant<int, 64>{}, none);
    else if (nvec <= 512) go(integral_constant<int, 8>{}, integral_constant<int, 64>{}, none);
    else if (nvec <= 1024) go(integral_constant<int, 4>{}, integral_constant<int, 256>{}, none);
    else if (nvec <= 2048 && alone) go(integral_constant<int, 4>{}, integral_constant<int, 512>{}, none);
    else if (nvec <= 2048) go(integral_constant<int, 8>{}, integral_constant<int, 256>{}, none);
    else if (nvec <= 4096 && alone) go(integral_constant<int, 8>{}, integral_constant<int, 512>{}, none);
    else if (nvec <= 4096) go(integral_constant<int, 16>{}, integral_constant<int, 256>{}, none);
    else if (nvec <= 8192 && alone) go(integral_constant<int, 8>{}, integral_constant<int, 1024>{}, none);
    else if (nvec <= 8192) go(integral_constant<int, 16>{}, integral_constant<int, 512>{}, none);
    else if (nvec <= 13312 && !alone) go(integral_constant<int, 16>{}, integral_constant<int, 512>{}, integral_constant<int, 5120>{});
    else if (nvec <= 16384) go(integral_constant<int, 16>{}, integral_constant<int, 1024>{}, none);
    else go(integral_constant<int, 16>{}, integral_constant<int, 1024>{}, integral_constant<int, 49152>{});
    return hipGetLastError();
  }
  if (plan.splits == 1) {
    if (p.grad) distill_row_kernel<T, 1024, true><<<n, 1024, 0, s>>>(p);
    // 200 x 128000 bf16: 14.5 us with 1024 threads, 20.2 with 256; 1 x 50001 and below the same
    else if (nvec >= 8192) distill_row_kernel<T, 1024, false><<<n, 1024, 0, s>>>(p);
    else distill_row_kernel<T, 256, false><<<n, 256, 0, s>>>(p);
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

// Parts of a row, of at least 4 KB and together at most 1024, where there are fewer long rows
// than CUs to take them.  With a gradient, parts read the row twice: 64 x 33001 bf16 11.5 us
// in parts, 14.6 whole, 1 x 40000 9.2 against 11.0, 1 x 128000 9.4 against 19.7; but 1 x 20000
// 9.3 against 9.4, 64 x 3000 10.3 against 8.8, 200 x 33001 16.9 against 15.8.  The loss alone:
// 1 x 40000 7.4 against 8.6, 64 x 128000 11.0 against 13.1; but 100 x 50001 fp32 11.6 against 9.0.
DistillPlan distill_plan(int64_t n, int64_t v, int elem_bytes, bool grad) {
  DistillPlan p{1, v, 0};
  const int64_t bytes = v * elem_bytes, least = (64 << 10) * (grad ? 1 : std::max<int64_t>(1, n / 20));
  const int64_t want = n > 128 || bytes < least
                           ? 1 : std::min(1024 / std::max<int64_t>(n, 1), bytes / ((4 << 10) * std::max<int64_t>(1, n / 16)));
  p.splits = (int)std::max<int64_t>(1, want);
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
