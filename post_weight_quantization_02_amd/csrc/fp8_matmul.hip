// Y = X W^T (+ bias) from e4m3 codes with one fp32 scale per 1 x 128 block of X and
// per 128 x 128 tile of W:
//
//   Y[i][j] = bias[j] + sum_b sx[b][i] sw[j / 128][b] sum_{c in block b} X8[i][c] W8[j][c]
//
// W is the A operand of the matrix instructions, so a lane holds one row of X (one sx)
// and four consecutive outputs.  Both operands take the columns of a block in the same
// order, so which lane holds which column does not matter.  The scaled sum over blocks
// is fp32; the sum inside a block is one of two:
//
//   Y fp16 or bf16: v_mfma_f32_16x16x128_f8f6f4 on the codes.  It adds products in
//     groups of 8, each truncated at 2^-13 of the power of two at or below the group's
//     largest exponent (measured on single products), and the groups in fp32: off by at
//     most 7 * 2^-13 sum |x w|, 1.3e-5 of the result's norm on random codes, an eighth
//     of fp16's own rounding.
//   Y fp32: codes widened to fp16 (exact) and v_mfma_f32_16x16x32_f16, whose sums are
//     fp32 throughout (9e-9 of the norm), at half the matrix rate: an fp32 result keeps
//     fp32's precision.
#include "gptq_internal.h"

namespace gptq {
namespace {

constexpr int kBlk = 128;
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef __bf16 bf16;
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

// 16 codes of a row from column c; columns from k on read as zero
__device__ __forceinline__ u32x4 load_chunk(const uint8_t* __restrict__ row, int64_t c, int64_t k) {
  if (c + 16 <= k) return *(const u32x4_any*)(row + c);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (c + e < k) v[e >> 2] |= (uint32_t)row[c + e] << (8 * (e & 3));
  return v;
}

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// a lane's 32 codes of a row and block, as the matrix instruction takes them
template <bool WIDE>
struct Frag;
template <>
struct Frag<false> {
  i32x8 c;
  __device__ __forceinline__ explicit Frag(i32x8 v) : c(v) {}
};
template <>
struct Frag<true> {
  half8 h[4];
  __device__ __forceinline__ explicit Frag(i32x8 v) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const h2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)v[2 * i + e], 1.f, false);
        const h2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)v[2 * i + e], 1.f, true);
        h[i][4 * e] = lo[0];
        h[i][4 * e + 1] = lo[1];
        h[i][4 * e + 2] = hi[0];
        h[i][4 * e + 3] = hi[1];
      }
  }
};

__device__ __forceinline__ f32x4 block_product(const Frag<false>& w, const Frag<false>& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.c, x.c, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 block_product(const Frag<true>& w, const Frag<true>& x) {
  f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.h[i], x.h[i], p, 0, 0, 0);
  return p;
}

// outputs j .. j + 3 of row i
template <typename T>
__device__ __forceinline__ void store4(T* __restrict__ Y, int64_t ld_y, const T* __restrict__ bias, int64_t i, int64_t j,
                                       int64_t m, int64_t n, f32x4 v) {
  if (i >= m) return;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (j + r < n) Y[i * ld_y + j + r] = (T)(v[r] + (bias ? (float)bias[j + r] : 0.f));
}

constexpr int kTile = 128;

// 128 x 128 outputs per work-group, 4 waves of 64 x 64, operands staged through LDS.
// A 16-byte chunk c of a tile row r lies at chunk c ^ (r & 7), so the 16 rows that a
// fragment load takes at one chunk spread over all banks.
template <typename T>
__global__ __launch_bounds__(256) void fp8_tile_kernel(const uint8_t* __restrict__ X, int64_t ld_x,
                                                       const float* __restrict__ sx, int64_t ld_sx,
                                                       const uint8_t* __restrict__ W, int64_t ld_w,
                                                       const float* __restrict__ sw, int64_t ld_sw, int64_t m, int64_t n,
                                                       int64_t k, const T* __restrict__ bias, T* __restrict__ Y,
                                                       int64_t ld_y) {
  constexpr bool WIDE = std::is_same<T, float>::value;
  __shared__ u32x4 xt[kTile * 8], wt[kTile * 8];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  const int64_t i0 = (int64_t)blockIdx.y * kTile, j0 = (int64_t)blockIdx.x * kTile;
  const int wi = (w & 1) * 64, wj = (w >> 1) * 64;
  const int lr = lane & 15, q = lane >> 4;
  f32x4 acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t nblk = (k + kBlk - 1) / kBlk;
  for (int64_t b = 0; b < nblk; ++b) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int id = t + 256 * c, r = id >> 3, ch = id & 7;
      const int at = r * 8 + (ch ^ (r & 7));
      xt[at] = load_chunk(X + min(i0 + r, m - 1) * ld_x, b * kBlk + ch * 16, k);
      wt[at] = load_chunk(W + min(j0 + r, n - 1) * ld_w, b * kBlk + ch * 16, k);
    }
    __syncthreads();
    const auto frag = [&](const u32x4* tile, int r) {
      return Frag<WIDE>(join(tile[r * 8 + (q ^ (r & 7))], tile[r * 8 + ((q + 4) ^ (r & 7))]));
    };
    const Frag<WIDE> wf[4] = {frag(wt, wj + lr), frag(wt, wj + 16 + lr), frag(wt, wj + 32 + lr), frag(wt, wj + 48 + lr)};
    const float s = sw[(j0 / kBlk) * ld_sw + b];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int r = wi + 16 * c + lr;
      const Frag<WIDE> xf = frag(xt, r);
      const float sc = s * sx[b * ld_sx + min(i0 + r, m - 1)];
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const f32x4 p = block_product(wf[a], xf);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[c][a][e] = fmaf(p[e], sc, acc[c][a][e]);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int a = 0; a < 4; ++a)
      store4<T>(Y, ld_y, bias, i0 + wi + 16 * c + lr, j0 + wj + 16 * a + 4 * q, m, n, acc[c][a]);
}

template <typename T>
hipError_t launch(const Fp8Args& p, hipStream_t s) {
  const dim3 grid((unsigned)cdiv(p.n, kTile), (unsigned)cdiv(p.m, kTile));
  fp8_tile_kernel<T><<<grid, 256, 0, s>>>(p.X, p.ld_x, p.sx, p.ld_sx, p.W, p.ld_w, p.sw, p.ld_sw, p.m, p.n, p.k,
                                          (const T*)p.bias, (T*)p.Y, p.ld_y);
  return hipGetLastError();
}

}  // namespace

Fp8Plan fp8_plan(int64_t m, int64_t n, int64_t k) { return Fp8Plan{0}; }

hipError_t fp8_matmul_launch(const Fp8Plan& plan, const Fp8Args& p, void* ws, hipStream_t s) {
  if (p.y_dtype == kF32) return launch<float>(p, s);
  if (p.y_dtype == kF16) return launch<_Float16>(p, s);
  return launch<bf16>(p, s);
}

}  // namespace gptq
