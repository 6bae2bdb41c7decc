// int8 codes with one scale per row: the operands of the 8-bit integer product.
//
// Per row: a = max |x|, a' = max(a, 2^-100), scale = a' / 127, code = rint(x (127 (1 / a'))),
// to nearest even.  1 / a' and 127 times it are rounded to fp32 once per row and the product
// with x once per element (a division of each element by the scale would cost ten instructions
// where there is time for four).  With u = 2^-24 and the scale's own rounding a code is x / scale
// to nearest but for quotients within 4 u 127 < 2^-15 of a half, or 7 u 127 < 2^-14 where a' passes
// 2^126: 1 / a' is subnormal there and off by up to 4 u.  |code| <= 127, as the largest element's
// product is at most 127 (1 + 6 u).  fl(127 / a') would be one rounding nearer and is not the
// definition: it gives other codes in 4 places of a million (16-bit elements, 5003 x 11007).  The
// floor keeps 127 / a' finite; rows below it, zeros among them, get small codes or none.  A row
// with a NaN or an infinity has
// no grid: its scale is NaN, which the product carries on, and its codes are 0.
//
// HBM-bound: one read of X, one byte written per element.  A row lives in the registers of
// one wave (short rows) or one work-group, in groups of 8 consecutive columns; magnitudes
// are compared as bit patterns without the sign (two 16-bit ones per instruction).  Rounding
// is an addition of 1.5 * 2^23, which leaves the code in the low byte.  5003 x 11007 fp16, half
// of its rows between words, 34.5 us, 4.8 TB/s, 93 % of what a large copy reaches (16-byte
// loads at odd elements and a last group taken element by element cost 10 us more); 8192 x
// 12288 fp16 56.5 us, 16384 x 4095 bf16 39.5; 1 x 4096 2.5 us, a launch.
#include "gptq_internal.h"

namespace gptq {
namespace {

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

// 8 elements from p on.  odd: p lies between two 32-bit words, inside a row; such 16-byte
// loads cost twice, so they start half a word before and are shifted.
template <typename T>
__device__ __forceinline__ void load8(const typename T::elem* __restrict__ p, bool odd, uint32_t (&w)[T::kWords]) {
  if (T::kWords == 4 && odd) {
    const u32x4_any v = *(const u32x4_any*)(p - 1);
    const uint32_t next = *(const uint32_t*)(p + 7);
    w[0] = __builtin_amdgcn_alignbit(v[1], v[0], 16); w[1] = __builtin_amdgcn_alignbit(v[2], v[1], 16);
    w[2] = __builtin_amdgcn_alignbit(v[3], v[2], 16); w[3] = __builtin_amdgcn_alignbit(next, v[3], 16);
    return;
  }
#pragma unroll
  for (int q = 0; q < T::kWords / 4; ++q) {
    const u32x4_any v = *(const u32x4_any*)((const uint32_t*)p + 4 * q);
    w[4 * q] = v[0]; w[4 * q + 1] = v[1]; w[4 * q + 2] = v[2]; w[4 * q + 3] = v[3];
  }
}

// the first n < 8 from p on, the others zero
template <typename T>
__device__ __forceinline__ void load_few(const typename T::elem* __restrict__ p, int n, uint32_t (&w)[T::kWords]) {
#pragma unroll
  for (int q = 0; q < T::kWords; ++q) w[q] = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) {
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

template <typename T, bool FEW>
__device__ __forceinline__ void store8(const uint32_t (&w)[T::kWords], float inv, uint8_t* __restrict__ p, int n) {
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
  if (!FEW) {
    *(u32x2_any*)p = u32x2_any{c[0], c[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = (uint8_t)(c[e >> 2] >> (8 * (e & 3)));
  }
}

// largest over the LANES lanes of a row (16 or 64), in every lane of it
template <int LANES>
__device__ __forceinline__ uint32_t over_lanes(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, true));
  if constexpr (LANES == 64) {
    const auto of = [&](int l) { return (uint32_t)__builtin_amdgcn_readlane((int)v, l); };
    v = max(max(of(0), of(16)), max(of(32), of(48)));
  }
  return v;
}

// One row per LANES threads (a quarter of a wave, a wave, or the work-group), G groups of 8
// columns each at a time; a row of more is read again when its scale is known.  A last group
// of fewer columns is the row's last 8, so some codes are written twice, alike.  FEW: rows of
// fewer than 8.
template <typename T, int LANES, int G, bool FEW>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void int8_rows_kernel(
    const typename T::elem* __restrict__ X, int64_t m, int k, int64_t ld_x, uint8_t* __restrict__ codes, int64_t ld_codes,
    float* __restrict__ scales) {
  constexpr int kThreads = LANES < 256 ? 256 : LANES, kSpan = LANES * G * 8;
  __shared__ uint32_t part[kThreads / 64];
  const int t = threadIdx.x, lane = t % LANES;
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kThreads / LANES) + t / LANES;
  const bool there = row < m;
  if (LANES >= 256 && !there) return;
  const auto* x = X + (there ? row : 0) * ld_x;
  uint8_t* out = codes + row * ld_codes;
  const bool odd = T::kWords == 4 && ((uintptr_t)x & 2) != 0;
  uint32_t w[G][T::kWords], a = 0u;
  const auto column = [&](int c0, int g) { return c0 + (g * LANES + lane) * 8; };
  // no lane of the work-group has columns
  const auto none = [&](int c0, int g) { return g > 0 && c0 + g * LANES * 8 >= k; };
  const auto load = [&](int c0) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (FEW) {
        load_few<T>(x, k, w[g]);
      } else if (none(c0, g)) {
#pragma unroll
        for (int q = 0; q < T::kWords; ++q) w[g][q] = 0u;
      } else {
        const int c = min(column(c0, g), k - 8);
        load8<T>(x + c, odd && c > 0 && c + 8 < k, w[g]);
      }
    }
  };
  for (int c0 = 0; c0 < k; c0 += kSpan) {
    load(c0);
#pragma unroll
    for (int g = 0; g < G; ++g) a = mag8<T>(w[g], a);
  }
  if constexpr (T::kWords == 4) a = max(a & 0xffffu, a >> 16);
  a = over_lanes<LANES == 16 ? 16 : 64>(a);
  if constexpr (LANES >= 256) {
    if ((t & 63) == 0) part[t >> 6] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) a = max(a, part[i]);
  }
  const bool sound = a < T::kInf;
  const float top = fmaxf(mag_value<T>(a), kFloor);
  const float inv = sound ? 127.f * (1.f / top) : 0.f;
  if (lane == 0 && there) scales[row] = sound ? top / 127.f : NAN;
  for (int c0 = 0; c0 < k; c0 += kSpan) {
    if (k > kSpan) load(c0);
    if (!sound) {             // nothing times 0 is NaN
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int q = 0; q < T::kWords; ++q) w[g][q] = 0u;
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c = column(c0, g);
      if (there && c < k && !none(c0, g)) store8<T, FEW>(w[g], inv, out + (FEW ? 0 : min(c, k - 8)), k);
    }
  }
}

template <typename T>
void launch(const void* X, int64_t m, int64_t k, int64_t ld_x, uint8_t* codes, int64_t ld_codes, float* scales,
            hipStream_t s) {
  const auto go = [&](auto lanes, auto groups, auto few) {
    constexpr int kThreads = lanes.value < 256 ? 256 : lanes.value;
    const int64_t blocks = cdiv(m, kThreads / lanes.value), x = std::min<int64_t>(blocks, 1 << 20);
    int8_rows_kernel<T, lanes.value, groups.value, few.value><<<dim3((unsigned)x, (unsigned)cdiv(blocks, x)), kThreads, 0, s>>>(
        (const typename T::elem*)X, m, (int)k, ld_x, codes, ld_codes, scales);
  };
  using std::integral_constant;
  const std::false_type no;
  // the fewest lanes and groups that hold the row: 16384 x 128 bf16 3.7 us by quarters of
  // waves, 6.1 by waves; 16384 x 1000 10.9 by waves, 14.6 by work-groups of 256; 5003 x 11007
  // fp16 34.5 by 512 threads, 36.7 by 256, whose six groups leave room for fewer waves
  if (k < 8) return go(integral_constant<int, 16>{}, integral_constant<int, 1>{}, std::true_type{});
  if (k <= 128) return go(integral_constant<int, 16>{}, integral_constant<int, 1>{}, no);
  if (k <= 256) return go(integral_constant<int, 16>{}, integral_constant<int, 2>{}, no);
  if (k <= 512) return go(integral_constant<int, 64>{}, integral_constant<int, 1>{}, no);
  if (k <= 1024) return go(integral_constant<int, 64>{}, integral_constant<int, 2>{}, no);
  if (k <= 2048) return go(integral_constant<int, 256>{}, integral_constant<int, 1>{}, no);
  if (k <= 4096) return go(integral_constant<int, 256>{}, integral_constant<int, 2>{}, no);
  if (k <= 8192) return go(integral_constant<int, 256>{}, integral_constant<int, 4>{}, no);
  if (k <= 12288) return go(integral_constant<int, 512>{}, integral_constant<int, 3>{}, no);
  return go(integral_constant<int, 512>{}, integral_constant<int, 4>{}, no);
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
