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
  Frag() = default;
  __device__ __forceinline__ explicit Frag(i32x8 v) : c(v) {}
};
template <>
struct Frag<true> {
  half8 h[4];
  Frag() = default;
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

__device__ __forceinline__ void scale_add(f32x4& acc, const f32x4& d, float s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = fmaf(d[e], s, acc[e]);
  asm volatile("" : "+v"(acc));         // here, not sunk behind the products that follow
}

__device__ __forceinline__ int64_t xcd_remap(int64_t bid, int64_t total) {
  const int64_t q = total / 8, r = total % 8;
  const int64_t x = bid % 8, i = bid / 8;
  return (x < r) ? x * (q + 1) + i : r * (q + 1) + (x - r) * q + i;
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

// sum v (+ bias) over the parts of a split product or the waves of a work-group is
// always taken in the same order, so results do not depend on timing.

// ---------------------------------------------------------------- few rows
// At most 16 TT rows of X: W is streamed once, straight into registers.  A work-group
// takes 16 rows of W, its 8 waves every eighth block of 128 columns (4 blocks' loads in
// flight each), and the waves' sums meet in LDS.  X comes from L2.  HBM-bound on W, so
// the exact (widened) block sums cost nothing.
constexpr int kFewWaves = 8, kFewUnroll = 4;

template <typename T, int TT>
__global__ __launch_bounds__(64 * kFewWaves) void fp8_few_kernel(Fp8Args p) {
  __shared__ f32x4 part[kFewWaves][TT][64];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lr = lane & 15, q = lane >> 4;
  const int64_t j0 = (int64_t)blockIdx.x * 16;
  const uint8_t* wr = p.W + min<int64_t>(j0 + lr, p.n - 1) * p.ld_w;
  const float* sw = p.sw + (j0 / kBlk) * p.ld_sw;
  const uint8_t* xr[TT];
  const float* sx[TT];
#pragma unroll
  for (int c = 0; c < TT; ++c) {
    const int64_t i = min<int64_t>(16 * c + lr, p.m - 1);
    xr[c] = p.X + i * p.ld_x;
    sx[c] = p.sx + i;
  }
  f32x4 acc[TT];
#pragma unroll
  for (int c = 0; c < TT; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const auto add = [&](i32x8 wv, const i32x8 (&xv)[TT], const float (&sc)[TT], float s) {
    const Frag<true> wf(wv);
#pragma unroll
    for (int c = 0; c < TT; ++c) {
      const f32x4 d = block_product(wf, Frag<true>(xv[c]));
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[c][e] = fmaf(d[e], s * sc[c], acc[c][e]);
    }
  };
  const auto whole = [&](const uint8_t* r, int64_t b) {
    const uint8_t* a = r + b * kBlk + 16 * q;
    return join(*(const u32x4_any*)a, *(const u32x4_any*)(a + 64));
  };
  const int64_t full = p.k / kBlk;
  int64_t b = w;
  for (; b + kFewWaves * (kFewUnroll - 1) < full; b += kFewWaves * kFewUnroll) {
    i32x8 wv[kFewUnroll], xv[kFewUnroll][TT];
    float sc[kFewUnroll][TT], s[kFewUnroll];
#pragma unroll
    for (int u = 0; u < kFewUnroll; ++u) {
      const int64_t at = b + kFewWaves * u;
      wv[u] = whole(wr, at);
      s[u] = sw[at];
#pragma unroll
      for (int c = 0; c < TT; ++c) {
        xv[u][c] = whole(xr[c], at);
        sc[u][c] = sx[c][at * p.ld_sx];
      }
    }
#pragma unroll
    for (int u = 0; u < kFewUnroll; ++u) add(wv[u], xv[u], sc[u], s[u]);
  }
  for (; b * kBlk < p.k; b += kFewWaves) {      // what is left, the last block guarded
    i32x8 xv[TT];
    float sc[TT];
    const auto any = [&](const uint8_t* r) {
      return b < full ? whole(r, b)
                      : join(load_chunk(r, b * kBlk + 16 * q, p.k), load_chunk(r, b * kBlk + 64 + 16 * q, p.k));
    };
    const i32x8 wv = any(wr);
#pragma unroll
    for (int c = 0; c < TT; ++c) {
      xv[c] = any(xr[c]);
      sc[c] = sx[c][b * p.ld_sx];
    }
    add(wv, xv, sc, sw[b]);
  }
#pragma unroll
  for (int c = 0; c < TT; ++c) part[w][c][lane] = acc[c];
  __syncthreads();
  if (w < TT) {
    f32x4 v = part[0][w][lane];
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) v += part[i][w][lane];
    store4<T>((T*)p.Y, p.ld_y, (const T*)p.bias, 16 * w + lr, j0 + 4 * q, p.m, p.n, v);
  }
}

// ---------------------------------------------------------------- tiles by LDS
// BT rows of X by BN rows of W per work-group, WT x WN waves.  Each block of 128
// columns goes to LDS without passing through registers (16-byte direct loads, a wave's
// load filling 8 rows of 128 bytes), one block ahead of the products, in two buffers
// that are variables of their own so that reading one does not wait for the other's loads.
// Row r keeps its 16-byte chunk c at place c ^ (r & 7): the 16 rows that a fragment
// load takes at one chunk then spread over all banks.  The rows' scales travel with the
// block; the tile of W has one scale, fetched a block ahead.  A last block of fewer than
// 128 columns is taken first, through registers, with zeros behind column k.  Scaling
// lags one row of tiles behind the matrix instructions, so it runs beside them.
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(4))) float uniform_float;

// `bytes` bytes from a wave-uniform address
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  const uint64_t u = ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32) |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)u, (short)0, __builtin_amdgcn_readfirstlane((int)bytes),
                                           0x00020000);
}

// 16 bytes per lane from r + voffset + soffset to LDS at `to` + 16 * lane
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t voffset, int soffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, voffset, soffset, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, float* to, uint32_t voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 4, voffset, 0, 0, 0);
}

template <int BT, int BN>
struct __attribute__((aligned(16))) Stage {
  uint8_t x[BT * kBlk];
  uint8_t w[BN * kBlk];
  float sx[BT + 64];      // each wave's load of the rows' scales writes 64 of them, the next wave's first ones too
};

template <typename T, bool WIDE, int BT, int BN, int WT, int WN, bool SPLIT>
__global__ __launch_bounds__(64 * WT * WN) void fp8_dma_kernel(Fp8Args p, int tiles_t, int tiles_n, int blocks_per_split,
                                                               float* __restrict__ parts) {
  constexpr int kWavesHere = WT * WN, TT = BT / WT / 16, TN = BN / WN / 16;
  constexpr int kXLoads = BT / 8 / kWavesHere, kWLoads = BN / 8 / kWavesHere;
  static_assert(kXLoads * 8 * kWavesHere == BT && kWLoads * 8 * kWavesHere == BN, "loads divide over the waves");
  static_assert(BN / WN <= kBlk && kBlk % (BN / WN) == 0, "one W scale per wave");
  constexpr int kScaleRows = BT / kWavesHere;
  __shared__ Stage<BT, BN> s0;
  __shared__ Stage<BT, BN> s1;
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lr = lane & 15, q = lane >> 4;
  // work-groups of one XCD take neighbouring tiles: bands of 8 tiles along X, W outermost
  const int tiles = tiles_t * tiles_n;
  const int part = blockIdx.x / tiles;
  const int id = (int)xcd_remap(blockIdx.x % tiles, tiles);
  const int band = id / (8 * tiles_n), in = id - band * 8 * tiles_n, high = min(8, tiles_t - 8 * band);
  const int64_t i0 = (int64_t)(8 * band + in % high) * BT, j0 = (int64_t)(in / high) * BN;
  const int wi = (w % WT) * (BT / WT), wj = (w / WT) * (BN / WN);
  const int nblk = (int)((p.k + kBlk - 1) / kBlk);
  const int b0 = part * blocks_per_split, b1 = min(b0 + blocks_per_split, nblk);

  const int rows_x = (int)min<int64_t>(BT, p.m - i0), rows_w = (int)min<int64_t>(BN, p.n - j0);
  const __amdgpu_buffer_rsrc_t xb = rsrc(p.X + i0 * p.ld_x, (rows_x - 1) * p.ld_x + p.k);
  const __amdgpu_buffer_rsrc_t wb = rsrc(p.W + j0 * p.ld_w, (rows_w - 1) * p.ld_w + p.k);
  // a lane's row and chunk in each of the wave's loads; rows past the end repeat the last
  const int ch = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t xo[kXLoads], wo[kWLoads];
#pragma unroll
  for (int j = 0; j < kXLoads; ++j)
    xo[j] = (uint32_t)(min((w * kXLoads + j) * 8 + (lane >> 3), rows_x - 1) * p.ld_x) + ch;
#pragma unroll
  for (int j = 0; j < kWLoads; ++j)
    wo[j] = (uint32_t)(min((w * kWLoads + j) * 8 + (lane >> 3), rows_w - 1) * p.ld_w) + ch;
  const uint32_t so = 4u * (uint32_t)min(w * kScaleRows + lane, rows_x - 1);
  uniform_float* swp = (uniform_float*)(uintptr_t)p.sw + ((j0 + wj) / kBlk < (p.n + kBlk - 1) / kBlk ? (j0 + wj) / kBlk : 0) * p.ld_sw;
  const auto fetch = [&](Stage<BT, BN>& s, int b) {
#pragma unroll
    for (int j = 0; j < kXLoads; ++j)
      load16_to_lds(xb, s.x + (w * kXLoads + j) * 8 * kBlk, xo[j], b * kBlk);
#pragma unroll
    for (int j = 0; j < kWLoads; ++j)
      load16_to_lds(wb, s.w + (w * kWLoads + j) * 8 * kBlk, wo[j], b * kBlk);
    load4_to_lds(rsrc(p.sx + (int64_t)b * p.ld_sx + i0, 4 * rows_x), s.sx + w * kScaleRows, so);
  };
  f32x4 acc[TT][TN];
#pragma unroll
  for (int c = 0; c < TT; ++c)
#pragma unroll
    for (int a = 0; a < TN; ++a) acc[c][a] = f32x4{0.f, 0.f, 0.f, 0.f};
  // a lane's chunks q and q + 4 of its row in the wave's first tile of each operand
  const uint32_t x0 = (uint32_t)((wi + lr) * kBlk + ((q ^ (lr & 7)) * 16)), x1 = x0 ^ 64;
  const uint32_t w0 = (uint32_t)((wj + lr) * kBlk + ((q ^ (lr & 7)) * 16)), w1 = w0 ^ 64;
  const uint32_t sx0 = (uint32_t)(wi + lr);
  const auto multiply = [&](const Stage<BT, BN>& s, float sw) {
    const auto frag = [&](const uint8_t* rows, uint32_t a, uint32_t b, int tile) {
      return Frag<WIDE>(join(*(const u32x4*)(rows + a + tile * 16 * kBlk), *(const u32x4*)(rows + b + tile * 16 * kBlk)));
    };
    Frag<WIDE> wf[TN];
#pragma unroll
    for (int a = 0; a < TN; ++a) wf[a] = frag(s.w, w0, w1, a);
    Frag<WIDE> xf = frag(s.x, x0, x1, 0), xn;
    float sc = sw * s.sx[sx0], sc_last = 0.f;
    f32x4 last[TN];
#pragma unroll
    for (int c = 0; c < TT; ++c) {
      f32x4 d[TN];
      float sn = 0.f;
      if (c + 1 < TT) {
        xn = frag(s.x, x0, x1, c + 1);
        sn = sw * s.sx[sx0 + 16 * (c + 1)];
      }
#pragma unroll
      for (int a = 0; a < TN; ++a) {
        d[a] = block_product(wf[a], xf);
        if (c > 0) scale_add(acc[c - 1][a], last[a], sc_last);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int a = 0; a < TN; ++a) last[a] = d[a];
      sc_last = sc;
      xf = xn;
      sc = sn;
    }
#pragma unroll
    for (int a = 0; a < TN; ++a) scale_add(acc[TT - 1][a], last[a], sc_last);
  };
  // a block of fewer than 128 columns, through registers
  const auto fetch_tail = [&](Stage<BT, BN>& s, int b) {
    for (int id = t; id < (BT + BN) * 8; id += 64 * kWavesHere) {
      const bool is_x = id < BT * 8;
      const int r = is_x ? id >> 3 : (id >> 3) - BT, c = id & 7;
      const uint8_t* row = is_x ? p.X + (i0 + min(r, rows_x - 1)) * p.ld_x : p.W + (j0 + min(r, rows_w - 1)) * p.ld_w;
      *(u32x4*)((is_x ? s.x : s.w) + r * kBlk + ((c ^ (r & 7)) * 16)) = load_chunk(row, (int64_t)b * kBlk + 16 * c, p.k);
    }
    if (t < BT) s.sx[t] = p.sx[(int64_t)b * p.ld_sx + i0 + min(t, rows_x - 1)];
  };
  const bool tail = b1 == nblk && (p.k % kBlk) != 0;
  const int steps = b1 - b0;
  const auto block_of = [&](int step) { return !tail ? b0 + step : step == 0 ? nblk - 1 : b0 + step - 1; };
  float sw_next = swp[block_of(0)];
  if (tail) fetch_tail(s0, nblk - 1);
  else fetch(s0, b0);
  for (int step = 0; step < steps; step += 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && step + 1 >= steps) break;
      Stage<BT, BN>& here = h ? s1 : s0;
      Stage<BT, BN>& there = h ? s0 : s1;
      // this block has arrived, and every wave is done with the buffer that is filled next
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      const float sw = sw_next;
      // after the last block, a block that is not used: a fetch on every path lets the
      // reads of `here` wait for nothing of `there`
      const int b = step + h + 1 < steps ? block_of(step + h + 1) : 0;
      sw_next = swp[b];
      fetch(there, b);
      multiply(here, sw);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the unused fetch writes LDS: not after this work-group's end
#pragma unroll
  for (int c = 0; c < TT; ++c)
#pragma unroll
    for (int a = 0; a < TN; ++a) {
      const int64_t i = i0 + wi + 16 * c + lr, j = j0 + wj + 16 * a + 4 * q;
      if constexpr (SPLIT) store4<float>(parts + (int64_t)part * p.m * p.n, p.n, nullptr, i, j, p.m, p.n, acc[c][a]);
      else store4<T>((T*)p.Y, p.ld_y, (const T*)p.bias, i, j, p.m, p.n, acc[c][a]);
    }
}

// Y from the parts of a product split over k
template <typename T>
__global__ __launch_bounds__(256) void fp8_sum_kernel(Fp8Args p, int splits, const float* __restrict__ parts) {
  const int64_t size = p.m * p.n;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < size; id += (int64_t)gridDim.x * 256) {
    const int64_t i = id / p.n, j = id - i * p.n;
    float v = parts[id];
    for (int s = 1; s < splits; ++s) v += parts[s * size + id];
    if (p.bias) v += (float)((const T*)p.bias)[j];
    ((T*)p.Y)[i * p.ld_y + j] = (T)v;
  }
}

constexpr int kTile = 128;

// ---------------------------------------------------------------- rows at any address
// Code rows that do not start at multiples of 16: 128 x 128 outputs per work-group,
// 4 waves of 64 x 64, the same LDS layout filled through registers by unaligned loads.
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

template <typename T, bool WIDE, int BT, int BN, int WT, int WN>
hipError_t launch_dma(const Fp8Plan& plan, const Fp8Args& p, float* ws, hipStream_t s) {
  const int tt = (int)cdiv(p.m, BT), tn = (int)cdiv(p.n, BN);
  const int per = (int)cdiv(cdiv(p.k, kBlk), plan.splits);
  if (plan.splits == 1) {
    fp8_dma_kernel<T, WIDE, BT, BN, WT, WN, false><<<tt * tn, 64 * WT * WN, 0, s>>>(p, tt, tn, per, nullptr);
  } else {
    fp8_dma_kernel<T, WIDE, BT, BN, WT, WN, true><<<tt * tn * plan.splits, 64 * WT * WN, 0, s>>>(p, tt, tn, per, ws);
    fp8_sum_kernel<T><<<(unsigned)std::min<int64_t>(cdiv(p.m * p.n, 256), 2048), 256, 0, s>>>(p, plan.splits, ws);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t launch(const Fp8Plan& plan, const Fp8Args& p, float* ws, hipStream_t s) {
  constexpr bool WIDE = std::is_same<T, float>::value;
  const unsigned few = (unsigned)cdiv(p.n, 16);
  if (plan.kind == kFp8Few) {
    if (p.m <= 16) fp8_few_kernel<T, 1><<<few, 64 * kFewWaves, 0, s>>>(p);
    else if (p.m <= 32) fp8_few_kernel<T, 2><<<few, 64 * kFewWaves, 0, s>>>(p);
    else fp8_few_kernel<T, 4><<<few, 64 * kFewWaves, 0, s>>>(p);
    return hipGetLastError();
  }
  // the direct loads need 16-byte rows, 32-bit offsets inside a tile and a whole block
  const bool dma = p.k >= kBlk && (((uintptr_t)p.X | (uintptr_t)p.W | (uint64_t)p.ld_x | (uint64_t)p.ld_w) & 15) == 0 &&
                   std::max(p.ld_x, p.ld_w) <= (int64_t(1) << 22);
  if (!dma) {
    const dim3 grid((unsigned)cdiv(p.n, kTile), (unsigned)cdiv(p.m, kTile));
    fp8_tile_kernel<T><<<grid, 256, 0, s>>>(p.X, p.ld_x, p.sx, p.ld_sx, p.W, p.ld_w, p.sw, p.ld_sw, p.m, p.n, p.k,
                                            (const T*)p.bias, (T*)p.Y, p.ld_y);
    return hipGetLastError();
  }
  if (plan.kind == kFp8Large) {
    if constexpr (WIDE) return launch_dma<T, WIDE, 128, 256, 2, 4>(plan, p, ws, s);
    else return launch_dma<T, WIDE, 256, 256, 2, 4>(plan, p, ws, s);
  }
  return launch_dma<T, WIDE, 128, 128, 2, 2>(plan, p, ws, s);
}

}  // namespace

Fp8Plan fp8_plan(int64_t m, int64_t n, int64_t k) {
  Fp8Plan p{kFp8Few, 1, 0};
  if (m <= 64) return p;
  if (cdiv(m, 256) * cdiv(n, 256) >= 192) {
    p.kind = kFp8Large;
    return p;
  }
  p.kind = kFp8Medium;
  const int64_t tiles = cdiv(m, kTile) * cdiv(n, kTile), nblk = cdiv(k, kBlk);
  const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(512 / tiles, nblk / 4));
  p.splits = (int)cdiv(nblk, cdiv(nblk, splits));     // none empty
  if (p.splits > 1) p.ws_bytes = (size_t)p.splits * m * n * sizeof(float);
  return p;
}

hipError_t fp8_matmul_launch(const Fp8Plan& plan, const Fp8Args& p, void* ws, hipStream_t s) {
  if (p.y_dtype == kF32) return launch<float>(plan, p, (float*)ws, s);
  if (p.y_dtype == kF16) return launch<_Float16>(plan, p, (float*)ws, s);
  return launch<bf16>(plan, p, (float*)ws, s);
}

}  // namespace gptq
