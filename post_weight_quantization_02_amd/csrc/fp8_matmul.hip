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
//     most 7 * 2^-13 sum |x w|; 1.3e-5 of the result's norm on codes of normal values,
//     5e-5 on random bytes, against fp16's own 3e-4.  The older v_mfma_f32_16x16x32_fp8_fp8
//     truncates in the same way at the rate of fp16, so the alternative is the sum below:
//     4096 x 12288 x 4096 366 us in place of 176, 384 x 4096 x 4096 22 in place of 16.
//   Y fp32, and few rows of any type: codes widened to fp16 (exact) and
//     v_mfma_f32_16x16x32_f16, whose sums are fp32 throughout (9e-9 of the norm), at half
//     the matrix rate: an fp32 result keeps fp32's precision.
#include "codes8.h"
#include "gptq_internal.h"

namespace gptq {
namespace {

typedef const __attribute__((address_space(4))) float uniform_float;   // read by scalar loads
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

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

// ---------------------------------------------------------------- few rows
// At most 16 TT rows of X.  A work-group takes 16 rows of W, its waves every fourth
// block of 128 columns, and the waves' sums meet in LDS at the end.  Each wave streams
// its blocks of W, and the rows of X and their scales with them, through a ring of R
// LDS slots of its own, filled by direct loads R - 1 blocks ahead: no barriers, and
// nothing in flight holds registers.  HBM-bound on W, so the exact (widened) block sums
// cost nothing.  A last block of fewer than 128 columns goes through registers, asked
// for first and multiplied last.  1 x 11008 x 4096 10.1 us, 4.5 TB/s of codes, of which
// 2.5 us are a launch's; R = 3 to 8 slots, 2 or 8 waves and streaming through registers
// were slower.
constexpr int kFewWaves = 4;

template <int TT>
struct __attribute__((aligned(16))) Slot {
  uint8_t w[16 * kBlk];
  uint8_t x[16 * TT * kBlk];
  float sx[64];
};
template <int TT, int I>
__device__ __forceinline__ Slot<TT> (&slots())[kFewWaves] {
  __shared__ Slot<TT> s[kFewWaves];
  return s;
}

template <typename T, int TT, int R, bool DMA>
__global__ __launch_bounds__(64 * kFewWaves) __attribute__((amdgpu_waves_per_eu(TT == 4 ? 1 : 2))) void
fp8_few_kernel(Fp8Args p) {
  __shared__ f32x4 part[kFewWaves][TT][64];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lr = lane & 15, q = lane >> 4;
  const int64_t j0 = (int64_t)blockIdx.x * 16;
  uniform_float* sw = (uniform_float*)(uintptr_t)p.sw + (j0 / kBlk) * p.ld_sw;
  const int rows_w = (int)min<int64_t>(16, p.n - j0), rows_x = (int)p.m;
  const int full = (int)(p.k / kBlk), nblk = (int)((p.k + kBlk - 1) / kBlk);
  f32x4 acc[TT];
#pragma unroll
  for (int c = 0; c < TT; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  // blocks through registers, where rows may start anywhere
  const auto by_registers = [&](int b) {
    const auto both = [&](const uint8_t* r) {
      return join(load_chunk(r, (int64_t)b * kBlk + 16 * q, p.k), load_chunk(r, (int64_t)b * kBlk + 64 + 16 * q, p.k));
    };
    const i32x8 wv = both(p.W + (j0 + min(lr, rows_w - 1)) * p.ld_w);
    i32x8 xv[TT];
    float sc[TT];
#pragma unroll
    for (int c = 0; c < TT; ++c) {
      const int64_t i = min(16 * c + lr, rows_x - 1);
      xv[c] = both(p.X + i * p.ld_x);
      sc[c] = p.sx[(int64_t)b * p.ld_sx + i];
    }
#pragma unroll
    for (int c = 0; c < TT; ++c) scale_add(acc[c], block_product(Frag<true>(wv), Frag<true>(xv[c])), sc[c] * sw[b]);
  };
  if constexpr (!DMA) {
    for (int b = w; b < nblk; b += kFewWaves) by_registers(b);
  } else {
    const int mine = full > w ? (full - w + kFewWaves - 1) / kFewWaves : 0;      // whole blocks w, w + 4, ...
    const __amdgpu_buffer_rsrc_t wb = rsrc(p.W + j0 * p.ld_w, (rows_w - 1) * p.ld_w + p.k);
    const __amdgpu_buffer_rsrc_t xb = rsrc(p.X, (rows_x - 1) * p.ld_x + p.k);
    const int ch = ((lane & 7) ^ (lane >> 3)) * 16;
    uint32_t wo[2], xo[2 * TT];
#pragma unroll
    for (int j = 0; j < 2; ++j) wo[j] = (uint32_t)(min(8 * j + (lane >> 3), rows_w - 1) * p.ld_w) + ch;
#pragma unroll
    for (int j = 0; j < 2 * TT; ++j) xo[j] = (uint32_t)(min(8 * j + (lane >> 3), rows_x - 1) * p.ld_x) + ch;
    const uint32_t so = 4u * (uint32_t)min(lane, rows_x - 1);
    const auto block_of = [&](int i) { return i < mine ? w + kFewWaves * i : 0; };
    const auto fetch = [&](Slot<TT>& s, int b) {
#pragma unroll
      for (int j = 0; j < 2; ++j) load16_to_lds(wb, s.w + 8 * j * kBlk, wo[j], b * kBlk);
#pragma unroll
      for (int j = 0; j < 2 * TT; ++j) load16_to_lds(xb, s.x + 8 * j * kBlk, xo[j], b * kBlk);
      load4_to_lds(rsrc(p.sx + (int64_t)b * p.ld_sx, 4 * rows_x), s.sx, so);
    };
    constexpr int kLoads = 3 + 2 * TT;
    static_assert((R - 1) * kLoads < 64, "counted by vmcnt");
    const uint32_t a0 = (uint32_t)(lr * kBlk + ((q ^ (lr & 7)) * 16)), a1 = a0 ^ 64;
    const auto use = [&](const Slot<TT>& s, float scale) {
      const Frag<true> wf(join(*(const u32x4*)(s.w + a0), *(const u32x4*)(s.w + a1)));
#pragma unroll
      for (int c = 0; c < TT; ++c) {
        const Frag<true> xf(join(*(const u32x4*)(s.x + 16 * c * kBlk + a0), *(const u32x4*)(s.x + 16 * c * kBlk + a1)));
        scale_add(acc[c], block_product(wf, xf), s.sx[16 * c + lr] * scale);
      }
    };
    // a last block of fewer columns: asked for before the others, multiplied after them
    const bool tail = full < nblk && full % kFewWaves == w;
    const int64_t c0 = (int64_t)full * kBlk + 16 * q;
    u32x4 tw[2], tx[TT][2];
    float ts[TT];
    if (tail) {
#pragma unroll
      for (int h = 0; h < 2; ++h) tw[h] = load_inside(p.W + (j0 + min(lr, rows_w - 1)) * p.ld_w, c0 + 64 * h, p.k);
#pragma unroll
      for (int c = 0; c < TT; ++c) {
        const int64_t i = min(16 * c + lr, rows_x - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) tx[c][h] = load_inside(p.X + i * p.ld_x, c0 + 64 * h, p.k);
        ts[c] = p.sx[(int64_t)full * p.ld_sx + i];
      }
    }
    if (mine > 0) {
      float sw_next = sw[w];
      static_for<0, R - 1>([&](auto i) { fetch(slots<TT, i.value>()[w], block_of(i.value)); });
      int i = 0;
      const auto one = [&](auto h) {
        // the reads of the slot that is refilled next are done; so is this slot's block once it alone is left out
        const float scale = sw_next;
        sw_next = sw[block_of(i + 1)];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        fetch(slots<TT, (h.value + R - 1) % R>()[w], block_of(i + R - 1));
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((R - 1) * kLoads) : "memory");
        use(slots<TT, h.value>()[w], scale);
        ++i;
      };
      while (i + R <= mine) static_for<0, R>(one);
      static_for<0, R - 1>([&](auto h) {
        if (i < mine) one(h);
      });
    }
    if (tail) {
      const auto both = [&](const u32x4 (&v)[2]) {
        return Frag<true>(join(align_chunk(v[0], c0, p.k), align_chunk(v[1], c0 + 64, p.k)));
      };
      const Frag<true> wf = both(tw);
      const float scale = sw[full];
#pragma unroll
      for (int c = 0; c < TT; ++c) scale_add(acc[c], block_product(wf, both(tx[c])), ts[c] * scale);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // unused fetches write LDS: not after this work-group's end
  }
#pragma unroll
  for (int c = 0; c < TT; ++c) part[w][c][lane] = acc[c];
  __syncthreads();
  if (w < TT) {         // TT <= 4 waves
    f32x4 v = part[0][w][lane];
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) v += part[i][w][lane];
    store4<T>((T*)p.Y, p.ld_y, (const T*)p.bias, 16 * w + lr, j0 + 4 * q, p.m, p.n, v);
  }
}

// ---------------------------------------------------------------- tiles by LDS
// BT rows of X by BN rows of W per work-group, WT x WN waves.  Each block of 128
// columns goes to LDS without passing through registers (16-byte direct loads, a wave's
// load filling 8 rows of 128 bytes), S - 1 blocks ahead of the products, in S buffers
// that are variables of their own so that reading one does not wait for the others' loads.
// Row r keeps its 16-byte chunk c at place c ^ (r & 7): the 16 rows that a fragment
// load takes at one chunk then spread over all banks.  The rows' scales travel with the
// block; the tile of W has one scale, fetched a block ahead.  A last block of fewer than
// 128 columns is taken first, through registers, with zeros behind column k.  Scaling
// lags one row of tiles behind the matrix instructions, so it runs beside them.
// 4096 x 12288 x 4096, fp16 outputs: 174 us, 2.37 PF, of which the loop takes 160 and the
// outputs 14 (without loads and scaling 124 to 137, the card's own limit); what the waves
// wait for is a block's arrival and its barrier.  1000 x 50001 x 1536, fp32 outputs: 167 us,
// 0.92 PF, of which 28 are 200 MB of outputs (widening the codes costs nothing).
// 384 x 4096 x 4096: 14.1 to 16.3 us; its work-groups fetch 655 KB each, 60 to 80 bytes per ns
// and CU of the 114 that L2 gives at most; 17 % of its L2 reads are misses, the first ones of
// each XCD, and its waves wait 45 % of their time.  Not kept, no gain: a second barrier with W
// two blocks ahead, the next block's fragments carried over the barrier, work-groups that
// go on from tile to tile; slower: higher wave priority around the products.
// stage I of a kernel's buffers, variables of their own: one for each group of waves
template <int BT>
struct __attribute__((aligned(16))) StageX {
  uint8_t x[BT * kBlk];
  float sx[BT + 64];      // each wave's load of the rows' scales writes 64 of them, the next wave's first ones too
};
template <int BT, int WK, int I>
__device__ __forceinline__ StageX<BT> (&stage_x())[WK] {
  __shared__ StageX<BT> s[WK];
  return s;
}
template <int BN>
struct __attribute__((aligned(16))) StageW {
  uint8_t w[BN * kBlk];
};
template <int BN, int WK, int I>
__device__ __forceinline__ StageW<BN> (&stage_w())[WK] {
  __shared__ StageW<BN> s[WK];
  return s;
}

// how a work-group keeps its buffers full
enum Flow {
  kBlocks,      // S buffers; one barrier per block
  kAhead        // S buffers; a block's codes are read into registers while the one before is multiplied
};

template <typename T, bool WIDE, int BT, int BN, int WT, int WN, int WK, int S, Flow FLOW, bool SPLIT>
__global__ __launch_bounds__(64 * WT * WN * WK) __attribute__((amdgpu_waves_per_eu(2))) void
fp8_dma_kernel(Fp8Args p, int tiles_t, int tiles_n, int blocks_per_split, float* __restrict__ parts) {
  constexpr int kWavesHere = WT * WN, TT = BT / WT / 16, TN = BN / WN / 16;
  constexpr int kXLoads = BT / 8 / kWavesHere, kWLoads = BN / 8 / kWavesHere;
  static_assert(kXLoads * 8 * kWavesHere == BT && kWLoads * 8 * kWavesHere == BN, "loads divide over the waves");
  static_assert(BN / WN <= kBlk && kBlk % (BN / WN) == 0, "one W scale per wave");
  constexpr int kScaleRows = BT / kWavesHere;
  constexpr int kLoads = kXLoads + kWLoads + 1;        // of a wave, per block
  static_assert((S - 2) * kLoads < 64, "counted by vmcnt");
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane((t >> 6) % kWavesHere);
  const int g = __builtin_amdgcn_readfirstlane((t >> 6) / kWavesHere);      // the wave's group
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
  const int64_t tile_w = (j0 + wj) / kBlk;
  uniform_float* swp = (uniform_float*)(uintptr_t)p.sw + (tile_w < (p.n + kBlk - 1) / kBlk ? tile_w : 0) * p.ld_sw;
  // the rows' scales are X's last load
  const auto fetch_x = [&](StageX<BT>& s, int b, int l) {
    if (l < kXLoads) load16_to_lds(xb, s.x + (w * kXLoads + l) * 8 * kBlk, xo[l], b * kBlk);
    else load4_to_lds(rsrc(p.sx + (int64_t)b * p.ld_sx + i0, 4 * rows_x), s.sx + w * kScaleRows, so);
  };
  const auto fetch_w = [&](StageW<BN>& s, int b, int l) {
    load16_to_lds(wb, s.w + (w * kWLoads + l) * 8 * kBlk, wo[l], b * kBlk);
  };
  const auto fetch = [&](auto i, int b) {
#pragma unroll
    for (int l = 0; l <= kXLoads; ++l) fetch_x(stage_x<BT, WK, i.value>()[g], b, l);
#pragma unroll
    for (int l = 0; l < kWLoads; ++l) fetch_w(stage_w<BN, WK, i.value>()[g], b, l);
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
  const auto pick = [&](const uint8_t* rows, uint32_t a, uint32_t b, int tile) {
    return join(*(const u32x4*)(rows + a + tile * 16 * kBlk), *(const u32x4*)(rows + b + tile * 16 * kBlk));
  };
  // acc += scale * (W tiles * X tiles): x(c) and sx(c) give tile c of X and its rows' scales,
  // asked for one tile ahead; meanwhile(c) issues loads while tile c is multiplied (issued
  // together they would hold the wave up before its first product)
  const auto multiply = [&](const i32x8 (&wv)[TN], auto&& x, auto&& sx, float sw, auto&& meanwhile) {
    Frag<WIDE> wf[TN];
#pragma unroll
    for (int a = 0; a < TN; ++a) wf[a] = Frag<WIDE>(wv[a]);
    i32x8 xv = x(0);
    // a row scale is read two tiles before its use: multiplied by sw where it was read, it
    // would hold the products up for an LDS read each tile
    float sc = sx(0), sc_last = 0.f;
    f32x4 last[TN];
#pragma unroll
    for (int c = 0; c < TT; ++c) {
      f32x4 d[TN];
      float sn = 0.f;
      const Frag<WIDE> xf(xv);
      if (c + 1 < TT) {
        xv = x(c + 1);
        sn = sx(c + 1);
      }
#pragma unroll
      for (int a = 0; a < TN; ++a) {
        d[a] = block_product(wf[a], xf);
        if (c > 0) scale_add(acc[c - 1][a], last[a], sc_last);
        __builtin_amdgcn_sched_barrier(0);
      }
      meanwhile(c);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int a = 0; a < TN; ++a) last[a] = d[a];
      sc_last = sw * sc;
      sc = sn;
    }
#pragma unroll
    for (int a = 0; a < TN; ++a) scale_add(acc[TT - 1][a], last[a], sc_last);
  };
  // a last block of fewer than 128 columns, through registers: all loads first, and LDS
  // written once the next blocks' loads are under way
  const bool tail = b1 == nblk && (p.k % kBlk) != 0;
  constexpr int kAll = 64 * kWavesHere * WK, kTail = ((BT + BN) * 8 + kAll - 1) / kAll;
  static_assert(BT <= kAll, "a scale per thread");
  u32x4 tail_v[kTail];
  float tail_s = 0.f;
  if (tail) {
#pragma unroll
    for (int i = 0; i < kTail; ++i) {
      const int id = t + i * kAll, r = min(id >> 3, BT + BN - 1);
      const uint8_t* row = r < BT ? p.X + (i0 + min(r, rows_x - 1)) * p.ld_x : p.W + (j0 + min(r - BT, rows_w - 1)) * p.ld_w;
      tail_v[i] = load_inside(row, (int64_t)(nblk - 1) * kBlk + 16 * (id & 7), p.k);
    }
    tail_s = p.sx[(int64_t)(nblk - 1) * p.ld_sx + i0 + min(t, rows_x - 1)];
  }
  const auto put_tail = [&]() {
    if (!tail) return;
    StageX<BT>& sx = stage_x<BT, WK, 0>()[0];
#pragma unroll
    for (int i = 0; i < kTail; ++i) {
      const int id = t + i * kAll, r = id >> 3, c = id & 7;
      const u32x4 v = align_chunk(tail_v[i], (int64_t)(nblk - 1) * kBlk + 16 * c, p.k);
      if (r < BT) *(u32x4*)(sx.x + r * kBlk + ((c ^ (r & 7)) * 16)) = v;
      else if (r < BT + BN) *(u32x4*)(stage_w<BN, WK, 0>()[0].w + (r - BT) * kBlk + ((c ^ (r & 7)) * 16)) = v;
    }
    if (t < BT) sx.sx[t] = tail_s;
  };
  // the groups take the blocks in turn
  const int count = b1 - b0, steps = (count + WK - 1) / WK;
  const auto block_of = [&](int at) { return !tail ? b0 + at : at == 0 ? nblk - 1 : b0 + at - 1; };
  // behind the last block, block 0, which is not used: with a fetch on every path the
  // counts of outstanding loads are known, and no read waits for a later block
  const auto next = [&](int step) { return step * WK + g < count ? block_of(step * WK + g) : 0; };
  float sw_next = swp[next(0)];
  if (!tail || g > 0) fetch(std::integral_constant<int, 0>{}, next(0));
  int step = 0;
  // one(stage, whether the group has a block): only in the last step may it have none
  const auto run = [&](auto&& one) {
    while (step + S < steps) static_for<0, S>([&](auto i) { one(i, true); });
    static_for<0, S>([&](auto i) {
      if (step < steps) one(i, WK == 1 || step * WK + g < count);
    });
  };
  if constexpr (FLOW == kBlocks) {
    static_for<1, S - 1>([&](auto i) { fetch(i, next(i.value)); });
    put_tail();
    run([&](auto i, bool has) {
      constexpr int h = i.value, to = (h + S - 1) % S;
      const StageX<BT>& s = stage_x<BT, WK, h>()[g];
      // this block has arrived, and every wave is done with the buffer that is filled next
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * kLoads) : "memory");
      const float sw = sw_next;
      sw_next = swp[next(step + 1)];
      const int b = next(step + S - 1);
      ++step;
      if (!has) return;           // nothing follows: nothing to fetch
      // the largest tiles issue their loads beside the first half of the products (prompt
      // case 181 -> 178 us); for the others that is too late (1024 x 4096 x 4096: 24.2 -> 25.8)
      constexpr int kSpread = TT == 8 ? TT / 2 : 0;
      if constexpr (kSpread == 0) fetch(std::integral_constant<int, to>{}, b);
      i32x8 wv[TN];
#pragma unroll
      for (int a = 0; a < TN; ++a) wv[a] = pick(stage_w<BN, WK, h>()[g].w, w0, w1, a);
      multiply(wv, [&](int c) { return pick(s.x, x0, x1, c); }, [&](int c) { return s.sx[sx0 + 16 * c]; }, sw,
               [&](int c) {
#pragma unroll
                 for (int l = 0; l < kLoads; ++l)
                   if (kSpread > 0 && l * kSpread / kLoads == c) {
                     if (l <= kXLoads) fetch_x(stage_x<BT, WK, to>()[g], b, l);
                     else fetch_w(stage_w<BN, WK, to>()[g], b, l - kXLoads - 1);
                   }
               });
    });
  } else {
    static_assert(S % 2 == 0, "two sets of registers in turn");
    static_for<1, S>([&](auto i) { fetch(i, next(i.value)); });
    put_tail();
    i32x8 wv[2][TN], xv[2][TT];
    float sxv[2][TT];
    constexpr int kReads = TN + TT;
    const auto read_one = [&](int set, const StageX<BT>& x, const StageW<BN>& w, int l) {
      if (l < TN) wv[set][l] = pick(w.w, w0, w1, l);
      else {
        xv[set][l - TN] = pick(x.x, x0, x1, l - TN);
        sxv[set][l - TN] = x.sx[sx0 + 16 * (l - TN)];
      }
    };
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 1) * kLoads) : "memory");
#pragma unroll
    for (int l = 0; l < kReads; ++l) read_one(0, stage_x<BT, WK, 0>()[g], stage_w<BN, WK, 0>()[g], l);
    run([&](auto i, bool has) {
      constexpr int h = i.value, set = h & 1, nx = (h + 1) % S;
      // the next block has arrived, and every wave has read this one
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * kLoads) : "memory");
      const float sw = sw_next;
      sw_next = swp[next(step + 1)];
      const int b = next(step + S);
      ++step;
      if (!has) return;
      multiply(wv[set], [&](int c) { return xv[set][c]; }, [&](int c) { return sxv[set][c]; }, sw, [&](int c) {
#pragma unroll
        for (int l = 0; l < kReads; ++l)
          if (l * TT / kReads == c) read_one(set ^ 1, stage_x<BT, WK, nx>()[g], stage_w<BN, WK, nx>()[g], l);
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
          if (l * TT / kLoads == c) {
            if (l <= kXLoads) fetch_x(stage_x<BT, WK, h>()[g], b, l);
            else fetch_w(stage_w<BN, WK, h>()[g], b, l - kXLoads - 1);
          }
      });
    });
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // unused fetches write LDS: not after this work-group's end
  if constexpr (WK > 1) {
    // group 1's sums are added to group 0's through stage 0's rows of X, as many tiles of
    // each wave at a time as fit
    constexpr int kFit = (int)sizeof(StageX<BT>::x) / (16 * 64 * kWavesHere);
    static_assert(WK == 2 && kFit >= 1, "two groups");
    f32x4* const sums = (f32x4*)stage_x<BT, WK, 0>()[0].x + w * kFit * 64 + lane;
#pragma unroll
    for (int e0 = 0; e0 < TT * TN; e0 += kFit) {
      // every wave's reads are done: of the last block, then of the sums before
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (g == 1) {
#pragma unroll
        for (int e = e0; e < e0 + kFit && e < TT * TN; ++e) sums[(e - e0) * 64] = acc[e / TN][e % TN];
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (g == 0) {
#pragma unroll
        for (int e = e0; e < e0 + kFit && e < TT * TN; ++e) acc[e / TN][e % TN] += sums[(e - e0) * 64];
      }
    }
    if (g == 1) return;
  }
  // Outputs of more than 80 MiB go past the caches' keeping: 4096 x 12288 x 4096 fp16 173 us
  // against 184, 1000 x 50001 x 1536 fp32 166 against 179 (with the call that reads them
  // next, 1 to 2 % slower); 4096 x 8192 x 1024 fp16, 64 MiB, 48 against 42.
  const bool stream = (uint64_t)p.m * (uint64_t)p.n * sizeof(T) > (uint64_t)80 << 20;
#pragma unroll
  for (int c = 0; c < TT; ++c) {
    const int64_t i = i0 + wi + 16 * c + lr, j = j0 + wj;
    if constexpr (TN == 4) {
      static_assert(!SPLIT, "split products take narrower tiles");
      store_rows64<T>((T*)p.Y, p.ld_y, (const T*)p.bias, i - lr, j, lr, q, p.m, p.n, stream, acc[c]);
    } else {
#pragma unroll
      for (int a = 0; a < TN; ++a) {
        if constexpr (SPLIT)
          store4<float>(parts + (int64_t)part * p.m * p.n, p.n, nullptr, i, j + 16 * a + 4 * q, p.m, p.n, acc[c][a]);
        else store4<T>((T*)p.Y, p.ld_y, (const T*)p.bias, i, j + 16 * a + 4 * q, p.m, p.n, acc[c][a]);
      }
    }
  }
}

// Y from the parts of a product split over k, added in one order whatever the timing, as the
// sums of a work-group's waves are: results repeat bitwise
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
// 4 waves of 64 x 64, the same LDS layout filled through registers by unaligned loads, block
// after block.  1024 x 4096 x 4096 with rows 4097 bytes apart 115 us, 4096 bytes apart 25: the
// quantizer's own codes always have aligned rows, and so has whoever wants the speed.
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

template <typename T, bool WIDE, int BT, int BN, int WT, int WN, int WK, int S, Flow FLOW>
hipError_t launch_dma(const Fp8Plan& plan, const Fp8Args& p, float* ws, hipStream_t s) {
  const int tt = (int)cdiv(p.m, BT), tn = (int)cdiv(p.n, BN);
  const int per = (int)cdiv(cdiv(p.k, kBlk), plan.splits);
  if constexpr (BT == 64 && BN == 32) {       // the only tiles of products that are split
    if (plan.splits > 1) {
      fp8_dma_kernel<T, WIDE, BT, BN, WT, WN, WK, S, FLOW, true>
          <<<tt * tn * plan.splits, 64 * WT * WN * WK, 0, s>>>(p, tt, tn, per, ws);
      fp8_sum_kernel<T><<<(unsigned)std::min<int64_t>(cdiv(p.m * p.n, 256), 2048), 256, 0, s>>>(p, plan.splits, ws);
      return hipGetLastError();
    }
  }
  fp8_dma_kernel<T, WIDE, BT, BN, WT, WN, WK, S, FLOW, false><<<tt * tn, 64 * WT * WN * WK, 0, s>>>(p, tt, tn, per, nullptr);
  return hipGetLastError();
}

template <typename T>
hipError_t launch(const Fp8Plan& plan, const Fp8Args& p, float* ws, hipStream_t s) {
  constexpr bool WIDE = std::is_same<T, float>::value;
  // the direct loads need 16-byte rows, 32-bit offsets inside a tile and a whole block
  const uint64_t ld_x = p.m > 1 ? (uint64_t)p.ld_x : 0, ld_w = p.n > 1 ? (uint64_t)p.ld_w : 0;
  const bool dma = p.k >= kBlk && (((uintptr_t)p.X | (uintptr_t)p.W | ld_x | ld_w) & 15) == 0 &&
                   std::max(ld_x, ld_w) <= (uint64_t(1) << 22);
  const unsigned few = (unsigned)cdiv(p.n, 16);
  if (plan.kind == kFp8Few) {
    if (!dma) {
      if (p.m <= 16) fp8_few_kernel<T, 1, 1, false><<<few, 64 * kFewWaves, 0, s>>>(p);
      else if (p.m <= 32) fp8_few_kernel<T, 2, 1, false><<<few, 64 * kFewWaves, 0, s>>>(p);
      else fp8_few_kernel<T, 4, 1, false><<<few, 64 * kFewWaves, 0, s>>>(p);
    } else {
      if (p.m <= 16) fp8_few_kernel<T, 1, 2, true><<<few, 64 * kFewWaves, 0, s>>>(p);
      else if (p.m <= 32) fp8_few_kernel<T, 2, 2, true><<<few, 64 * kFewWaves, 0, s>>>(p);
      else fp8_few_kernel<T, 4, 2, true><<<few, 64 * kFewWaves, 0, s>>>(p);
    }
    return hipGetLastError();
  }
  if (!dma) {
    const dim3 grid((unsigned)cdiv(p.n, kTile), (unsigned)cdiv(p.m, kTile));
    fp8_tile_kernel<T><<<grid, 256, 0, s>>>(p.X, p.ld_x, p.sx, p.ld_sx, p.W, p.ld_w, p.sw, p.ld_sw, p.m, p.n, p.k,
                                            (const T*)p.bias, (T*)p.Y, p.ld_y);
    return hipGetLastError();
  }
  switch (plan.kind) {
    case kFp8T64x32: return launch_dma<T, WIDE, 64, 32, 2, 2, 2, 4, kAhead>(plan, p, ws, s);
    case kFp8T64x64: return launch_dma<T, WIDE, 64, 64, 2, 2, 2, 4, kAhead>(plan, p, ws, s);
    case kFp8T96x64: return launch_dma<T, WIDE, 96, 64, 2, 2, 2, 3, kBlocks>(plan, p, ws, s);
    case kFp8T128x64: return launch_dma<T, WIDE, 128, 64, 2, 2, 2, 3, kBlocks>(plan, p, ws, s);
    case kFp8T128x128Two: return launch_dma<T, WIDE, 128, 128, 2, 2, 2, 2, kBlocks>(plan, p, ws, s);
    case kFp8T256x256:                // 16-bit outputs only
      if constexpr (!WIDE) return launch_dma<T, WIDE, 256, 256, 2, 4, 1, 2, kBlocks>(plan, p, ws, s);
      [[fallthrough]];
    default: return launch_dma<T, WIDE, 128, 128, 2, 2, 1, 2, kBlocks>(plan, p, ws, s);
  }
}

}  // namespace

// Which kernel (times: 16-bit outputs, k = 4096, graph replays).
//   few rows or tiles: 32 x 4096 6.8 against 8.6 us, 64 x 4096 9.2 against 10; from 17 rows
//     on X is as much of the work as W: 32 x 11008 12.7 against 11.3 (fp32 outputs, whose
//     tiles have half the matrix rate: 12.8 against 16.4).  Along k > 8192 few work-groups
//     are too slow: 1 x 512 x 16384 12.7 us, in split tiles 8.8.
//   the smallest tiles that one round of 256 CUs covers: 128 x 4096 9.1 us in 64 x 32 tiles
//     against 11.0 in the next; 256 x 4096 11.5 (64 x 64) against 16.4 and 13.6; 384 x 4096
//     14.3 (96 x 64) against 20.6 and 16.3; 512 x 4096 17.1 (128 x 64) against 26.0 and 20.9;
//     1024 x 4096 24.6 (128 x 128, two groups) against 32.3 and 26.4 (one group).
//   k in parts where one round is less than half full: 96 x 512 x 8192 9.1 us, in one 12.3.
//   beyond one round, 128 x 128 or 256 x 256, by their times in us: a 128 x 128 tile adds
//     0.0064 + 0.00216 per block of k, a round of the larger ones takes 9.1 + 1.78, one of r
//     tiles 0.38 + 0.62 r / 256 of that.  2048 x 4096 38 against 46.5 us (r = 128), 1024 x
//     12288 60 against 56 (r = 192), 4096 x 12288 230 against 185; 2048 x 12288 x 1024 36
//     against 41.
Fp8Plan fp8_plan(int64_t m, int64_t n, int64_t k, bool wide) {
  Fp8Plan p{kFp8Few, 1, 0};
  const bool few = k > 8192 && n <= 1024 ? false
                   : m <= 16             ? true
                   : m <= 32             ? wide || n <= 8192
                                         : m <= 64 && n <= 4096 && k <= 4096;
  if (few) return p;
  const struct { int kind, bt, bn; } small[] = {
      {kFp8T64x32, 64, 32}, {kFp8T64x64, 64, 64}, {kFp8T96x64, 96, 64}, {kFp8T128x64, 128, 64},
      {kFp8T128x128Two, 128, 128}};
  for (const auto& c : small) {
    const int64_t tiles = cdiv(m, c.bt) * cdiv(n, c.bn);
    if (tiles > 256) continue;
    p.kind = c.kind;
    if (c.kind == kFp8T64x32) {         // the larger ones are taken from 129 tiles on: nothing to split
      const int64_t nblk = cdiv(k, kBlk), splits = std::max<int64_t>(1, std::min<int64_t>(256 / tiles, nblk / 16));
      p.splits = (int)cdiv(nblk, cdiv(nblk, splits));     // none empty
      if (p.splits > 1) p.ws_bytes = (size_t)p.splits * m * n * sizeof(float);
    }
    return p;
  }
  const int64_t t128 = cdiv(m, 128) * cdiv(n, 128), t256 = cdiv(m, 256) * cdiv(n, 256), rest = t256 % 256;
  const double nblk = (double)cdiv(k, kBlk), rounds = (double)(t256 / 256) + (rest > 0 ? 0.38 + 0.62 * rest / 256 : 0.0);
  p.kind = !wide && rounds * (9.1 + 1.78 * nblk) < t128 * (0.0064 + 0.00216 * nblk) ? kFp8T256x256 : kFp8T128x128;
  return p;
}

hipError_t fp8_matmul_launch(const Fp8Plan& plan, const Fp8Args& p, void* ws, hipStream_t s) {
  if (p.y_dtype == kF32) return launch<float>(plan, p, (float*)ws, s);
  if (p.y_dtype == kF16) return launch<_Float16>(plan, p, (float*)ws, s);
  return launch<bf16>(plan, p, (float*)ws, s);
}

}  // namespace gptq
