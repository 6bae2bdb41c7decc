// int8 codes with one scale per row: the operands of the 8-bit integer product.
//
// Per row: a = max |x|, a' = max(a, 2^-100), scale = a' / 127, code = rint(x (127 (1 / a'))),
// to nearest even.  1 / a' and 127 times it are rounded to fp32 once per row and the product
// with x once per element (a division per element would cost ten instructions where there is
// time for four), so a code is x / scale to nearest, but for quotients within 2^-15 of a
// half, and |code| <= 127 as 127 (1 + 2^-21) rounds to 127.  The floor keeps 127 / a' finite;
// rows below it, zeros among them, get small codes or none.  A row with a NaN or an infinity has
// no grid: its scale is NaN, which the product carries on, and its codes are 0.
//
// HBM-bound: one read of X, one byte written per element.  A row lives in the registers of
// one wave (short rows) or one work-group, in groups of 8 consecutive columns; magnitudes
// are compared as bit patterns without the sign (two 16-bit ones per instruction).  Rounding
// is an addition of 1.5 * 2^23, which leaves the code in the low byte.
#include "gptq_internal.h"

namespace gptq {
namespace {

constexpr int kThreads = 256;
constexpr float kFloor = 0x1p-100f;
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef uint16_t us2 __attribute__((ext_vector_type(2)));
// vectors at any element address: global loads and stores need no alignment here
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

struct F32 {
  static constexpr int kWords = 8;   // 32-bit words of 8 elements
  typedef float elem;
  static constexpr uint32_t kInf = 0x7f800000u;
};
struct F16 {
  static constexpr int kWords = 4;
  typedef uint16_t elem;
  static constexpr uint32_t kInf = 0x7c00u;
};
struct BF16 {
  static constexpr int kWords = 4;
  typedef uint16_t elem;
  static constexpr uint32_t kInf = 0x7f80u;
};

__device__ __forceinline__ int valid_from(int64_t left) { return left >= 8 ? 8 : left > 0 ? (int)left : 0; }

// `valid` elements from p on, the others zero
template <typename T>
__device__ __forceinline__ void load8(const typename T::elem* __restrict__ p, int valid, uint32_t (&w)[T::kWords]) {
  if (valid >= 8) {
#pragma unroll
    for (int q = 0; q < T::kWords / 4; ++q) {
      const u32x4_any v = *(const u32x4_any*)((const uint32_t*)p + 4 * q);
      w[4 * q] = v[0]; w[4 * q + 1] = v[1]; w[4 * q + 2] = v[2]; w[4 * q + 3] = v[3];
    }
    return;
  }
#pragma unroll
  for (int q = 0; q < T::kWords; ++q) w[q] = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < valid) {
      if constexpr (T::kWords == 8) w[e] = __builtin_bit_cast(uint32_t, p[e]);
      else w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    }
}

// largest magnitude of 8 elements and a, as its bit pattern (16-bit types: of either half)
template <typename T>
__device__ __forceinline__ uint32_t mag8(const uint32_t (&w)[T::kWords], uint32_t a) {
  if constexpr (T::kWords == 8) {
#pragma unroll
    for (int q = 0; q < 8; ++q) a = max(a, w[q] & 0x7fffffffu);
    return a;
  } else {
    us2 m = __builtin_bit_cast(us2, a);
#pragma unroll
    for (int q = 0; q < 4; ++q) m = __builtin_elementwise_max(m, __builtin_bit_cast(us2, w[q] & 0x7fff7fffu));
    return __builtin_bit_cast(uint32_t, m);
  }
}

template <typename T>
__device__ __forceinline__ float value(const uint32_t (&w)[T::kWords], int e) {
  if constexpr (std::is_same<T, F32>::value) return __builtin_bit_cast(float, w[e]);
  else if constexpr (std::is_same<T, F16>::value) return (float)__builtin_bit_cast(h2, w[e >> 1])[e & 1];
  else return __builtin_bit_cast(float, (e & 1) ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
}

template <typename T>
__device__ __forceinline__ float mag_value(uint32_t a) {
  if constexpr (std::is_same<T, F32>::value) return __builtin_bit_cast(float, a);
  else if constexpr (std::is_same<T, F16>::value) return (float)__builtin_bit_cast(_Float16, (uint16_t)a);
  else return __builtin_bit_cast(float, a << 16);
}

template <typename T>
__device__ __forceinline__ void store8(const uint32_t (&w)[T::kWords], float inv, uint8_t* __restrict__ p, int valid) {
#pragma clang fp contract(off)      // the product is rounded before it is rounded to a whole number
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = value<T>(w, 4 * h + e) * inv;
      b[e] = __builtin_bit_cast(uint32_t, t + 12582912.f);
    }
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
    c[h] = lo | hi;
  }
  if (valid >= 8) {
    *(u32x2_any*)p = u32x2_any{c[0], c[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = (uint8_t)(c[e >> 2] >> (8 * (e & 3)));
  }
}

// One row per LANES threads (a wave, or the work-group), G groups of 8 columns each at a
// time; a row of more is read again when its scale is known.
template <typename T, int LANES, int G>
__global__ __launch_bounds__(kThreads) void int8_rows_kernel(const typename T::elem* __restrict__ X, int64_t m, int64_t k,
                                                             int64_t ld_x, uint8_t* __restrict__ codes, int64_t ld_codes,
                                                             float* __restrict__ scales) {
  __shared__ uint32_t part[kThreads / 64];
  const int t = threadIdx.x, lane = t % LANES;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / LANES) + t / LANES;
  if (LANES == 64 && row >= m) return;
  const auto* x = X + row * ld_x;
  uint8_t* out = codes + row * ld_codes;
  constexpr int64_t kSpan = (int64_t)LANES * G * 8;
  uint32_t w[G][T::kWords], a = 0u;
  const auto load = [&](int64_t c0) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t col = c0 + (g * LANES + lane) * 8;
      load8<T>(x + min(col, k - 1), valid_from(k - col), w[g]);
    }
  };
  for (int64_t c0 = 0; c0 < k; c0 += kSpan) {
    load(c0);
#pragma unroll
    for (int g = 0; g < G; ++g) a = mag8<T>(w[g], a);
  }
  if constexpr (T::kWords == 4) a = max(a & 0xffffu, a >> 16);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) a = max(a, (uint32_t)__shfl_xor((int)a, o, 64));
  if constexpr (LANES == kThreads) {
    if ((t & 63) == 0) part[t >> 6] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) a = max(a, part[i]);
  }
  const bool sound = a < T::kInf;
  const float top = fmaxf(mag_value<T>(a), kFloor);
  const float inv = 127.f * (1.f / top);
  if (lane == 0) scales[row] = sound ? top / 127.f : NAN;
  for (int64_t c0 = 0; c0 < k; c0 += kSpan) {
    if (k > kSpan) load(c0);
    if (!sound) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int q = 0; q < T::kWords; ++q) w[g][q] = 0u;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int64_t col = c0 + (g * LANES + lane) * 8;
      store8<T>(w[g], sound ? inv : 0.f, out + col, valid_from(k - col));
    }
  }
}

template <typename T, int LANES, int G>
void launch_rows(const void* X, int64_t m, int64_t k, int64_t ld_x, uint8_t* codes, int64_t ld_codes, float* scales,
                 hipStream_t s) {
  int8_rows_kernel<T, LANES, G><<<dim3((unsigned)cdiv(m, kThreads / LANES)), kThreads, 0, s>>>(
      (const typename T::elem*)X, m, k, ld_x, codes, ld_codes, scales);
}

template <typename T>
void launch(const void* X, int64_t m, int64_t k, int64_t ld_x, uint8_t* codes, int64_t ld_codes, float* scales,
            hipStream_t s) {
  const auto go = [&](auto lanes, auto groups) {
    launch_rows<T, lanes.value, groups.value>(X, m, k, ld_x, codes, ld_codes, scales, s);
  };
  using std::integral_constant;
  if (k <= 512) go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (k <= 1024) go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (k <= 2048) go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (k <= 4096) go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  else if (k <= 8192) go(integral_constant<int, 256>{}, integral_constant<int, 4>{});
  else go(integral_constant<int, 256>{}, integral_constant<int, 8>{});
}

}  // namespace

hipError_t int8_quantize_launch(const void* X, int x_dtype, int64_t m, int64_t k, int64_t ld_x, int8_t* codes,
                                int64_t ld_codes, float* scales, hipStream_t s) {
  uint8_t* c = (uint8_t*)codes;
  if (x_dtype == kF32) launch<F32>(X, m, k, ld_x, c, ld_codes, scales, s);
  else if (x_dtype == kF16) launch<F16>(X, m, k, ld_x, c, ld_codes, scales, s);
  else launch<BF16>(X, m, k, ld_x, c, ld_codes, scales, s);
  return hipGetLastError();
}

}  // namespace gptq
