// Y = X W^T (+ bias) from int8 codes with one fp32 scale per row of X and per row of W,
// alone and by expert:
//
//   Y[i][j] = fma(fl(float(sum_c X8[r(i)][c] W8[e(i)][j][c]) sx[r(i)]), sw[e(i)][j], bias[e(i)][j])
//
// The sum is a whole number below 2^31 (k < 2^17) and exact, its conversion and the two
// scalings are rounded to fp32, Y once more to its type.  Whichever kernel computes a row,
// and whatever other rows are in the call, its bits are the same.
//
// W is the A operand of v_mfma_i32_16x16x64_i8, so a lane holds one row of X and four
// consecutive outputs.  Both operands take the columns of a block in the same order, so
// which lane holds which column does not matter.
#include "codes8.h"
#include "gptq_internal.h"

namespace gptq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 product(u32x4 w, u32x4 x, i32x4 acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), acc, 0, 0, 0);
}

// four outputs of a row from their sums; none: -0, whose addition changes nothing
__device__ __forceinline__ f32x4 outputs(i32x4 acc, float sx, f32x4 sw, f32x4 bias) {
  f32x4 v;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float t = (float)acc[e] * sx;
    v[e] = __builtin_fmaf(t, sw[e], bias[e]);
  }
  return v;
}

// the scales and biases of outputs j .. j + 3
template <typename T>
__device__ __forceinline__ void load_channels(const float* __restrict__ sw, const T* __restrict__ bias, int64_t j, int64_t n,
                                              f32x4& s, f32x4& b) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t at = min(j + e, n - 1);
    s[e] = sw[at];
    b[e] = bias ? (float)bias[at] : -0.f;
  }
}

// The positions of one expert that a work-group takes: [i0, end), at most BT of them, and
// the number of such tiles before.  Without experts, all rows are one's.
struct Rows {
  int64_t i0, end;
  int expert;
};

// Tile `slot` of the experts' tiles of BT positions, each expert starting one of its own;
// expert < 0: there are not so many.  Offsets are taken within [0, m], and an expert that
// ends before it starts has none.  Every lane of a wave takes part; the result is uniform.
template <int BT>
__device__ __forceinline__ Rows find_rows(const Int8Args& p, int slot, int& total) {
  const int lane = threadIdx.x & 63, m = (int)p.m;
  const int per = (p.experts + 63) / 64, e0 = min(lane * per, p.experts), e1 = min(e0 + per, p.experts);
  const auto at = [&](int e) { return min(max(p.offsets[e], 0), m); };
  int mine = 0, from = at(e0);
  for (int e = e0; e < e1; ++e) {
    const int to = at(e + 1);
    mine += (max(to - from, 0) + BT - 1) / BT;
    from = to;
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, o, 64);
    if (lane >= o) upto += v;
  }
  total = __builtin_amdgcn_readlane(upto, 63);
  if (slot >= total) return Rows{0, 0, -1};
  const int l = __builtin_ctzll(__ballot(upto > slot));      // the first lane that has it
  int before = __builtin_amdgcn_readlane(upto - mine, l);
  int e = __builtin_amdgcn_readlane(e0, l);
  for (; e < p.experts; ++e) {                                // within that lane's experts
    const int a = at(e), b = at(e + 1), tiles = (max(b - a, 0) + BT - 1) / BT;
    if (slot < before + tiles) {
      const int i0 = a + (slot - before) * BT;
      return Rows{i0, min(i0 + BT, b), e};
    }
    before += tiles;
  }
  return Rows{0, 0, -1};
}

// the row of X that position i takes, within X; a bad one is noted in its scale
__device__ __forceinline__ int64_t row_of(const Int8Args& p, int64_t i) {
  if (!p.rows) return i;
  const int r = p.rows[i];
  return r >= 0 && r < p.rows_x ? r : 0;
}
__device__ __forceinline__ float scale_of(const Int8Args& p, int64_t i) {
  if (!p.rows) return p.sx[i];
  const int r = p.rows[i];
  return r >= 0 && r < p.rows_x ? p.sx[r] : NAN;
}

constexpr int kTile = 128;

// ---------------------------------------------------------------- rows at any address
// 128 x 128 outputs per work-group, 4 waves of 64 x 64, LDS filled through registers by
// unaligned loads, block after block.
template <typename T, bool GROUPED>
__global__ __launch_bounds__(256) void int8_tile_kernel(Int8Args p) {
  __shared__ u32x4 xt[kTile * 8], wt[kTile * 8];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  Rows g{(int64_t)blockIdx.y * kTile, p.m, 0};
  if constexpr (GROUPED) {
    int total;
    g = find_rows<kTile>(p, blockIdx.y, total);
    if (g.expert < 0) return;
  }
  const int64_t j0 = (int64_t)blockIdx.x * kTile, last = g.end - 1;
  const uint8_t* W = p.W + g.expert * p.stride_w;
  const float* sw = p.sw + (int64_t)g.expert * p.n;
  const T* bias = p.bias ? (const T*)p.bias + (int64_t)g.expert * p.n : nullptr;
  const int wi = (w & 1) * 64, wj = (w >> 1) * 64;
  const int lr = lane & 15, q = lane >> 4;
  i32x4 acc[4][4];
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int b = 0; b < 4; ++b) acc[a][b] = i32x4{0, 0, 0, 0};
  const uint8_t *xr[4], *wr[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int r = (t + 256 * c) >> 3;
    xr[c] = p.X + row_of(p, min(g.i0 + r, last)) * p.ld_x;
    wr[c] = W + min(j0 + r, p.n - 1) * p.ld_w;
  }
  const int64_t nblk = (p.k + kBlk - 1) / kBlk;
  for (int64_t b = 0; b < nblk; ++b) {
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int id = t + 256 * c, r = id >> 3, ch = id & 7;
      const int at = r * 8 + (ch ^ (r & 7));
      xt[at] = load_chunk(xr[c], b * kBlk + ch * 16, p.k);
      wt[at] = load_chunk(wr[c], b * kBlk + ch * 16, p.k);
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const auto chunk = [&](const u32x4* tile, int r) { return tile[r * 8 + ((q + 4 * h) ^ (r & 7))]; };
      u32x4 wv[4];
#pragma unroll
      for (int a = 0; a < 4; ++a) wv[a] = chunk(wt, wj + 16 * a + lr);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const u32x4 xv = chunk(xt, wi + 16 * c + lr);
#pragma unroll
        for (int a = 0; a < 4; ++a) acc[c][a] = product(wv[a], xv, acc[c][a]);
      }
    }
  }
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const int64_t j = j0 + wj + 16 * a + 4 * q;
    f32x4 s, b;
    load_channels<T>(sw, bias, j, p.n, s, b);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int64_t i = g.i0 + wi + 16 * c + lr;
      const float sx = scale_of(p, min(i, last));
      store4<T>((T*)p.Y, p.ld_y, nullptr, i, j, g.end, p.n, outputs(acc[c][a], sx, s, b));
    }
  }
}

// tiles of `bt` positions that the experts' parts of m positions can have at most
int64_t most_tiles(int64_t m, int64_t experts, int bt) {
  const int64_t used = std::min(m, experts);
  return (m + used * (bt - 1)) / bt;
}

template <typename T>
hipError_t launch(const Int8Plan& plan, const Int8Args& p, void* ws, hipStream_t s) {
  int8_tile_kernel<T, false><<<dim3((unsigned)cdiv(p.n, kTile), (unsigned)cdiv(p.m, kTile)), 256, 0, s>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_grouped(const Int8Args& p, hipStream_t s) {
  int8_tile_kernel<T, true>
      <<<dim3((unsigned)cdiv(p.n, kTile), (unsigned)most_tiles(p.m, p.experts, kTile)), 256, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

Int8Plan int8_plan(int64_t m, int64_t n, int64_t k) { return Int8Plan{0, 1, 0}; }

hipError_t int8_matmul_launch(const Int8Plan& plan, const Int8Args& p, void* ws, hipStream_t s) {
  if (p.y_dtype == kF32) return launch<float>(plan, p, ws, s);
  if (p.y_dtype == kF16) return launch<_Float16>(plan, p, ws, s);
  return launch<bf16>(plan, p, ws, s);
}

hipError_t int8_grouped_launch(const Int8Args& p, hipStream_t s) {
  if (p.y_dtype == kF32) return launch_grouped<float>(p, s);
  if (p.y_dtype == kF16) return launch_grouped<_Float16>(p, s);
  return launch_grouped<bf16>(p, s);
}

}  // namespace gptq
