// e4m3 codes with one scale per block of 128 columns: the operands of the 8-bit
// floating-point product.
//
// Per block (1 x 128 for activations, 128 x 128 for weights): a = max |x| over the
// finite elements, s = 2^e with e the smallest integer >= -126 such that
// a <= 448 2^e (448 = 1.75 2^8 is e4m3's largest value; s = 1 if a = 0), and
// code = e4m3(x / s), to nearest even.  A power of two makes x / s exact, so each
// code is rounded once and no code depends on how a division rounds; since codes
// are floating point, s = a / 448 would be no more precise for normal codes (it
// would gain at most one binade at the subnormal end).  Elements that are not finite
// take no part in a and become NaN (0x7F).
//
// HBM-bound: one read of X, one byte written per element.  A thread holds
// 8 consecutive columns (16- or 32-byte loads) of 4 rows (8 for tiles), 16 lanes hold
// one row of a block; the maximum goes over those lanes by row rotations, through
// LDS for tiles.  Magnitudes are compared as bit patterns without the sign (two
// 16-bit ones per instruction), so one comparison per block also finds non-finite
// elements, and only such a block takes the path that looks at each element.  8192 x 12288
// fp16 rows 59.7 us, 5.1 TB/s, 98 % of what a large copy reaches; 11001 x 4099 fp32 tiles
// 43.9 us, 5.1 TB/s; 1 x 4096 2.5 us, a launch.
#include "gptq_internal.h"

namespace gptq {
namespace {

constexpr int kThreads = 256;
constexpr int kBlk = 128;
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

// largest magnitude of 8 elements, as its bit pattern
template <typename T>
__device__ __forceinline__ uint32_t mag8(const uint32_t (&w)[T::kWords]) {
  if constexpr (T::kWords == 8) {
    uint32_t a = 0u;
#pragma unroll
    for (int q = 0; q < 8; ++q) a = max(a, w[q] & 0x7fffffffu);
    return a;
  } else {
    us2 a = {0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      a = __builtin_elementwise_max(a, __builtin_bit_cast(us2, w[q] & 0x7fff7fffu));
    return max((uint32_t)a[0], (uint32_t)a[1]);
  }
}

// the same over finite elements only
template <typename T>
__device__ __forceinline__ uint32_t mag8_finite(const uint32_t (&w)[T::kWords]) {
  uint32_t a = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = T::kWords == 8 ? w[e] & 0x7fffffffu : (w[e >> 1] >> (16 * (e & 1))) & 0x7fffu;
    a = max(a, b < T::kInf ? b : 0u);
  }
  return a;
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

// s = 2^e and 1 / s for the block maximum a (finite)
__device__ __forceinline__ float block_scale(float a, float& inv) {
  const uint32_t b = __builtin_bit_cast(uint32_t, a);
  int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -126);
  if (b == 0u) e = 0;
  inv = __builtin_bit_cast(float, (uint32_t)(127 - e) << 23);
  return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
}

template <typename T>
__device__ __forceinline__ void store8(const uint32_t (&w)[T::kWords], float inv, bool odd, uint8_t* __restrict__ p,
                                       int valid) {
  int c[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = value<T>(w, 4 * h + e) * inv;
    c[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], c[h], false);
    c[h] = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], c[h], true);
    if (odd) {   // the block has an element that is not finite
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!(fabsf(value<T>(w, 4 * h + e)) < INFINITY)) c[h] = (c[h] & ~(0xff << (8 * e))) | (0x7f << (8 * e));
    }
  }
  if (valid >= 8) {
    *(u32x2_any*)p = u32x2_any{(uint32_t)c[0], (uint32_t)c[1]};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < valid) p[e] = (uint8_t)(c[e >> 2] >> (8 * (e & 3)));
  }
}

// maximum over the 16 lanes of a row, in every lane of it
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, true));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, true));
}

constexpr int kRowIters = 4, kRowsPerWg = 16 * kRowIters;

// grid (column blocks, 64-row blocks); scales[block][row]
template <typename T>
__global__ __launch_bounds__(kThreads) void quant_rows_kernel(const typename T::elem* __restrict__ X, int64_t m,
                                                              int64_t k, int64_t ld_x, uint8_t* __restrict__ codes,
                                                              int64_t ld_codes, float* __restrict__ scales,
                                                              int64_t ld_scales) {
  const int t = threadIdx.x, g = t >> 4;
  const int64_t col = (int64_t)blockIdx.x * kBlk + (t & 15) * 8;
  const int64_t row0 = (int64_t)blockIdx.y * kRowsPerWg + g;
  const int valid = (int)min<int64_t>(max<int64_t>(k - col, 0), 8);
  uint32_t w[kRowIters][T::kWords];
#pragma unroll
  for (int i = 0; i < kRowIters; ++i) {
    const int64_t row = row0 + 16 * i;
    load8<T>(X + min<int64_t>(row, m - 1) * ld_x + min<int64_t>(col, k - 1), valid, w[i]);
  }
#pragma unroll
  for (int i = 0; i < kRowIters; ++i) {
    const int64_t row = row0 + 16 * i;
    uint32_t a = row_max(mag8<T>(w[i]));
    const bool odd = a >= T::kInf;
    if (odd) a = row_max(mag8_finite<T>(w[i]));
    float inv;
    const float s = block_scale(mag_value<T>(a), inv);
    if (row < m) {
      store8<T>(w[i], inv, odd, codes + row * ld_codes + col, valid);
      if ((t & 15) == 0) scales[(int64_t)blockIdx.x * ld_scales + row] = s;
    }
  }
}

constexpr int kTileIters = 8;

// grid (column blocks, row blocks); scales[row block][column block]
template <typename T>
__global__ __launch_bounds__(kThreads) void quant_tiles_kernel(const typename T::elem* __restrict__ X, int64_t m,
                                                               int64_t k, int64_t ld_x, uint8_t* __restrict__ codes,
                                                               int64_t ld_codes, float* __restrict__ scales,
                                                               int64_t ld_scales) {
  __shared__ uint32_t part[2][16];
  const int t = threadIdx.x, g = t >> 4;
  const int64_t col = (int64_t)blockIdx.x * kBlk + (t & 15) * 8;
  const int64_t row0 = (int64_t)blockIdx.y * kBlk + g;
  const int valid = (int)min<int64_t>(max<int64_t>(k - col, 0), 8);
  uint32_t w[kTileIters][T::kWords];
#pragma unroll
  for (int i = 0; i < kTileIters; ++i)   // rows past the end repeat the last one, which lies in the same tile
    load8<T>(X + min<int64_t>(row0 + 16 * i, m - 1) * ld_x + min<int64_t>(col, k - 1), valid, w[i]);
  uint32_t a = 0u;
#pragma unroll
  for (int i = 0; i < kTileIters; ++i) a = max(a, mag8<T>(w[i]));
  a = row_max(a);
  if ((t & 15) == 0) part[0][g] = a;
  __syncthreads();
  a = row_max(part[0][t & 15]);
  const bool odd = a >= T::kInf;         // the same in every thread
  if (odd) {
    a = 0u;
#pragma unroll
    for (int i = 0; i < kTileIters; ++i) a = max(a, mag8_finite<T>(w[i]));
    a = row_max(a);
    if ((t & 15) == 0) part[1][g] = a;
    __syncthreads();
    a = row_max(part[1][t & 15]);
  }
  float inv;
  const float s = block_scale(mag_value<T>(a), inv);
  if (t == 0) scales[(int64_t)blockIdx.y * ld_scales + blockIdx.x] = s;
#pragma unroll
  for (int i = 0; i < kTileIters; ++i) {
    const int64_t row = row0 + 16 * i;
    if (row < m) store8<T>(w[i], inv, odd, codes + row * ld_codes + col, valid);
  }
}

template <typename T>
void launch(const void* X, int64_t m, int64_t k, int64_t ld_x, int64_t block_rows, uint8_t* codes, int64_t ld_codes,
            float* scales, int64_t ld_scales, hipStream_t s) {
  const auto x = (const typename T::elem*)X;
  if (block_rows == 1)
    quant_rows_kernel<T><<<dim3((unsigned)cdiv(k, kBlk), (unsigned)cdiv(m, kRowsPerWg)), kThreads, 0, s>>>(
        x, m, k, ld_x, codes, ld_codes, scales, ld_scales);
  else
    quant_tiles_kernel<T><<<dim3((unsigned)cdiv(k, kBlk), (unsigned)cdiv(m, kBlk)), kThreads, 0, s>>>(
        x, m, k, ld_x, codes, ld_codes, scales, ld_scales);
}

}  // namespace

hipError_t fp8_quantize_launch(const void* X, int x_dtype, int64_t m, int64_t k, int64_t ld_x, int64_t block_rows,
                               uint8_t* codes, int64_t ld_codes, float* scales, int64_t ld_scales, hipStream_t s) {
  if (x_dtype == kF32) launch<F32>(X, m, k, ld_x, block_rows, codes, ld_codes, scales, ld_scales, s);
  else if (x_dtype == kF16) launch<F16>(X, m, k, ld_x, block_rows, codes, ld_codes, scales, ld_scales, s);
  else launch<BF16>(X, m, k, ld_x, block_rows, codes, ld_codes, scales, ld_scales, s);
  return hipGetLastError();
}

}  // namespace gptq
