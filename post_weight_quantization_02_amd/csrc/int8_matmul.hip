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
typedef int i32x16 __attribute__((ext_vector_type(16)));

// Edge of a matrix instruction's tile: 32 (v_mfma_i32_32x32x32_i8: four chunks of 32 columns a
// block) or 16 (v_mfma_i32_16x16x64_i8: two of 64).  A lane has 16 codes of row lane % M, and
// of the sums row lane % M of X and outputs 4 (lane / M) + e, for 32 in steps of 8.
template <int M>
struct Tile;
template <>
struct Tile<16> {
  typedef i32x4 Sums;
  static constexpr int kSteps = 2, kGroups = 1;
  static __device__ __forceinline__ Sums product(u32x4 w, u32x4 x, Sums acc) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), acc, 0, 0, 0);
  }
};
template <>
struct Tile<32> {
  typedef i32x16 Sums;
  static constexpr int kSteps = 4, kGroups = 4;
  static __device__ __forceinline__ Sums product(u32x4 w, u32x4 x, Sums acc) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), acc, 0, 0, 0);
  }
};
// outputs 8 g + 4 (lane / M) + e
template <int M>
__device__ __forceinline__ i32x4 group(const typename Tile<M>::Sums& s, int g) {
  return i32x4{s[4 * g], s[4 * g + 1], s[4 * g + 2], s[4 * g + 3]};
}

// an output from its sum; no bias: -0, whose addition changes nothing
__device__ __forceinline__ float output(int acc, float sx, float sw, float bias) {
  const float t = (float)acc * sx;
  float y = __builtin_fmaf(t, sw, bias);
  asm("" : "+v"(y));          // rounded to fp32 here, not only where it becomes fp16: one kernel's bits are another's
  return y;
}
__device__ __forceinline__ f32x4 outputs(i32x4 acc, float sx, f32x4 sw, f32x4 bias) {
  return f32x4{output(acc[0], sx, sw[0], bias[0]), output(acc[1], sx, sw[1], bias[1]), output(acc[2], sx, sw[2], bias[2]),
               output(acc[3], sx, sw[3], bias[3])};
}

// f(a value of Y's type)
template <typename F>
__device__ __forceinline__ void with_type(int dtype, F&& f) {
  if (dtype == kF32) f(0.f);
  else if (dtype == kF16) f((_Float16)0.f);
  else f((bf16)0.f);
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

// The positions of one expert that a work-group takes: [i0, end), at most BT of them.  Without
// experts, all rows are one's.
struct Rows {
  int64_t i0, end;
  int expert;
};
// an expert's positions, and the number of tiles of the experts before
struct Part {
  int from, to, expert, before;
};

// sum over the lanes up to this one
__device__ __forceinline__ int lanes_up_to(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, true);
  return v;
}

// The experts' tiles of BT positions, each expert starting one of its own: a lane has the
// experts [e0, e1).  Offsets are taken within [0, m], and an expert that ends before it starts
// has none.  Every lane of a wave takes part, and results are uniform.
template <int BT>
struct Experts {
  int e0, from, to;     // of the lane's first expert
  int mine, upto;       // tiles of the lane's, and of all up to them
  int total;
  static __device__ __forceinline__ int at(const Int8Args& p, int e) { return min(max(p.offsets[e], 0), (int)p.m); }
  static __device__ __forceinline__ int tiles(int a, int b) { return (max(b - a, 0) + BT - 1) / BT; }
  __device__ __forceinline__ explicit Experts(const Int8Args& p) {
    const int lane = threadIdx.x & 63, per = (p.experts + 63) / 64, e1 = min((lane + 1) * per, p.experts);
    e0 = min(lane * per, p.experts);
    from = at(p, e0);
    to = at(p, min(e0 + 1, p.experts));
    mine = e0 < e1 ? tiles(from, to) : 0;
    int a = to;
    for (int e = e0 + 1; e < e1; ++e) {
      const int b = at(p, e + 1);
      mine += tiles(a, b);
      a = b;
    }
    upto = lanes_up_to(mine);
    total = __builtin_amdgcn_readlane(upto, 63);
  }
  // the expert that has tile `slot`; expert < 0: there are not so many
  __device__ __forceinline__ Part part(const Int8Args& p, int slot) const {
    if (slot >= total) return Part{0, 0, -1, 0};
    const int l = __builtin_ctzll(__ballot(upto > slot));      // the first lane that has it
    int before = __builtin_amdgcn_readlane(upto - mine, l);
    int a = __builtin_amdgcn_readlane(from, l), b = __builtin_amdgcn_readlane(to, l);
    for (int e = __builtin_amdgcn_readlane(e0, l); e < p.experts; ++e) {      // within that lane's experts
      if (slot < before + tiles(a, b)) return Part{a, b, e, before};
      before += tiles(a, b);
      a = b;
      b = at(p, min(e + 2, p.experts));
    }
    return Part{0, 0, -1, 0};
  }
  // its tile `t`
  static __device__ __forceinline__ Rows tile(const Part& e, int t) {
    const int i0 = e.from + t * BT;
    return Rows{i0, min(i0 + BT, e.to), e.expert};
  }
  __device__ __forceinline__ Rows find(const Int8Args& p, int slot) const {
    const Part e = part(p, slot);
    return tile(e, slot - e.before);
  }
};

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
// unaligned loads, block after block: 4096 x 12288 x 4096 with rows 4101 bytes apart 707 us, 320
// x 4096 x 4096 94, bound by those loads (16-byte rows by direct loads 188 and 12.4).
template <bool GROUPED>
__global__ __launch_bounds__(256) void int8_tile_kernel(Int8Args p) {
  __shared__ u32x4 xt[kTile * 8], wt[kTile * 8];
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  Rows g{(int64_t)blockIdx.y * kTile, p.m, 0};
  if constexpr (GROUPED) {
    g = Experts<kTile>(p).find(p, blockIdx.y);
    if (g.expert < 0) return;
  }
  const int64_t j0 = (int64_t)blockIdx.x * kTile, last = g.end - 1;
  const uint8_t* W = p.W + g.expert * p.stride_w;
  const float* sw = p.sw + (int64_t)g.expert * p.n;
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
        for (int a = 0; a < 4; ++a) acc[c][a] = Tile<16>::product(wv[a], xv, acc[c][a]);
      }
    }
  }
  with_type(p.y_dtype, [&](auto zero) {
    typedef decltype(zero) T;
    const T* bias = p.bias ? (const T*)p.bias + (int64_t)g.expert * p.n : nullptr;
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
  });
}


// ---------------------------------------------------------------- few rows
// At most 16 TT positions.  A wave takes 16 TN rows of W.  The four waves of a work-group take
// every fourth block of 128 columns of the same rows, and their sums meet in LDS at the end
// (KW = 4), or rows of their own (KW = 1).  Each wave streams its blocks of W, and the rows of
// X with them, through a ring of R LDS slots of its own, filled by direct loads R - 1 blocks
// ahead: no barriers, and nothing in flight holds registers.  A last block of fewer than 128
// columns goes through registers, asked for first and multiplied last.  HBM-bound on W: 1 x
// 11008 x 4096 9.5 us, 4.7 TB/s of codes with a launch's 2.5 us in it; 29 x 5001 x 4163 7.9;
// one token's 8 of 64 experts, 1536 x 4096 each, 11.2; 303 positions of 24 experts, 1999 x
// 1111 each, 13.2.
constexpr int kFewWaves = 4;

template <int TT, int TN>
struct __attribute__((aligned(16))) Slot {
  uint8_t w[16 * TN * kBlk];
  uint8_t x[16 * TT * kBlk];
};
template <int TT, int TN, int I>
__device__ __forceinline__ Slot<TT, TN> (&slots())[kFewWaves] {
  __shared__ Slot<TT, TN> s[kFewWaves];
  return s;
}

template <int TT, int TN, int KW, int R, bool DMA, bool GROUPED>
__global__ __launch_bounds__(64 * kFewWaves) __attribute__((amdgpu_waves_per_eu(TT * TN >= 4 ? 1 : 2))) void
int8_few_kernel(Int8Args p) {
  static_assert(KW == 1 || KW == kFewWaves, "waves along the columns");
  constexpr int kOwn = KW == 1 ? TT * TN : (TT * TN + KW - 1) / KW;      // tiles that a wave stores
  __shared__ i32x4 part[KW][KW == 1 ? 1 : TT * TN][64];
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int lr = lane & 15, q = lane >> 4, wk = KW == 1 ? 0 : w;
  Rows g{0, p.m, 0};
  if constexpr (GROUPED) {
    g = Experts<16 * TT>(p).find(p, blockIdx.y);
    if (g.expert < 0) return;
  }
  const uint8_t* W = p.W + g.expert * p.stride_w;
  const int64_t j0 = ((int64_t)blockIdx.x * (kFewWaves / KW) + (KW == 1 ? w : 0)) * (16 * TN);
  if (KW == 1 && j0 >= p.n) return;
  const int rows_w = (int)min<int64_t>(16 * TN, p.n - j0), rows_x = (int)(g.end - g.i0);
  // the scales and biases of the tiles that this wave stores, asked for first
  float sx[kOwn];
  f32x4 sw[kOwn], bias[kOwn];
  const auto own = [&](int o) { return KW == 1 ? o : o * KW + w; };
  with_type(p.y_dtype, [&](auto zero) {
    typedef decltype(zero) T;
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      const int e = min(own(o), TT * TN - 1);
      load_channels<T>(p.sw + (int64_t)g.expert * p.n, p.bias ? (const T*)p.bias + (int64_t)g.expert * p.n : nullptr,
                       j0 + 16 * (e % TN) + 4 * q, p.n, sw[o], bias[o]);
      sx[o] = scale_of(p, min(g.i0 + 16 * (e / TN) + lr, g.end - 1));
    }
  });
  const int full = (int)(p.k / kBlk), nblk = (int)((p.k + kBlk - 1) / kBlk);
  i32x4 acc[TT][TN];
#pragma unroll
  for (int c = 0; c < TT; ++c)
#pragma unroll
    for (int a = 0; a < TN; ++a) acc[c][a] = i32x4{0, 0, 0, 0};
  const auto wrow = [&](int a) { return W + (j0 + min(16 * a + lr, rows_w - 1)) * p.ld_w; };
  const auto xrow = [&](int c) { return p.X + row_of(p, g.i0 + min(16 * c + lr, rows_x - 1)) * p.ld_x; };
  if constexpr (!DMA) {
    // blocks through registers, where rows may start anywhere
    for (int b = wk; b < nblk; b += KW)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = (int64_t)b * kBlk + 64 * h + 16 * q;
        u32x4 xv[TT];
#pragma unroll
        for (int c = 0; c < TT; ++c) xv[c] = load_chunk(xrow(c), at, p.k);
#pragma unroll
        for (int a = 0; a < TN; ++a) {
          const u32x4 wv = load_chunk(wrow(a), at, p.k);
#pragma unroll
          for (int c = 0; c < TT; ++c) acc[c][a] = Tile<16>::product(wv, xv[c], acc[c][a]);
        }
      }
  } else {
    const int mine = full > wk ? (full - wk + KW - 1) / KW : 0;      // whole blocks wk, wk + KW, ...
    const __amdgpu_buffer_rsrc_t wb = rsrc(W + j0 * p.ld_w, (rows_w - 1) * p.ld_w + p.k);
    // gathered rows lie anywhere in X, others are neighbours
    const __amdgpu_buffer_rsrc_t xb = p.rows ? rsrc(p.X, (p.rows_x - 1) * p.ld_x + p.k)
                                             : rsrc(p.X + g.i0 * p.ld_x, (rows_x - 1) * p.ld_x + p.k);
    const int ch = ((lane & 7) ^ (lane >> 3)) * 16;
    uint32_t wo[2 * TN], xo[2 * TT];
#pragma unroll
    for (int j = 0; j < 2 * TN; ++j) wo[j] = (uint32_t)(min(8 * j + (lane >> 3), rows_w - 1) * p.ld_w) + ch;
#pragma unroll
    for (int j = 0; j < 2 * TT; ++j) {
      const int r = min(8 * j + (lane >> 3), rows_x - 1);
      xo[j] = (uint32_t)((p.rows ? row_of(p, g.i0 + r) : r) * p.ld_x) + ch;
    }
    const auto block_of = [&](int i) { return i < mine ? wk + KW * i : 0; };
    const auto fetch = [&](Slot<TT, TN>& s, int b) {
#pragma unroll
      for (int j = 0; j < 2 * TN; ++j) load16_to_lds(wb, s.w + 8 * j * kBlk, wo[j], b * kBlk);
#pragma unroll
      for (int j = 0; j < 2 * TT; ++j) load16_to_lds(xb, s.x + 8 * j * kBlk, xo[j], b * kBlk);
    };
    constexpr int kLoads = 2 * TN + 2 * TT;
    static_assert(R > 1 && (R - 1) * kLoads < 64, "counted by vmcnt");
    const uint32_t a0 = (uint32_t)(lr * kBlk + ((q ^ (lr & 7)) * 16));
    const auto use = [&](const Slot<TT, TN>& s) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4 xv[TT];
#pragma unroll
        for (int c = 0; c < TT; ++c) xv[c] = *(const u32x4*)(s.x + 16 * c * kBlk + (a0 ^ (64 * h)));
#pragma unroll
        for (int a = 0; a < TN; ++a) {
          const u32x4 wv = *(const u32x4*)(s.w + 16 * a * kBlk + (a0 ^ (64 * h)));
#pragma unroll
          for (int c = 0; c < TT; ++c) acc[c][a] = Tile<16>::product(wv, xv[c], acc[c][a]);
        }
      }
    };
    // a last block of fewer columns: asked for before the others, multiplied after them
    const bool tail = full < nblk && full % KW == wk;
    const int64_t c0 = (int64_t)full * kBlk + 16 * q;
    u32x4 tw[TN][2], tx[TT][2];
    if (tail) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int a = 0; a < TN; ++a) tw[a][h] = load_inside(wrow(a), c0 + 64 * h, p.k);
#pragma unroll
        for (int c = 0; c < TT; ++c) tx[c][h] = load_inside(xrow(c), c0 + 64 * h, p.k);
      }
    }
    if (mine > 0) {
      static_for<0, R - 1>([&](auto i) { fetch(slots<TT, TN, i.value>()[w], block_of(i.value)); });
      int i = 0;
      const auto one = [&](auto h) {
        // the reads of the slot that is refilled next are done; so is this slot's block once it alone is left out
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        fetch(slots<TT, TN, (h.value + R - 1) % R>()[w], block_of(i + R - 1));
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((R - 1) * kLoads) : "memory");
        use(slots<TT, TN, h.value>()[w]);
        ++i;
      };
      while (i + R <= mine) static_for<0, R>(one);
      static_for<0, R - 1>([&](auto h) {
        if (i < mine) one(h);
      });
    }
    if (tail) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int a = 0; a < TN; ++a) {
          const u32x4 wv = align_chunk(tw[a][h], c0 + 64 * h, p.k);
#pragma unroll
          for (int c = 0; c < TT; ++c) acc[c][a] = Tile<16>::product(wv, align_chunk(tx[c][h], c0 + 64 * h, p.k), acc[c][a]);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // unused fetches write LDS: not after this work-group's end
  }
  if constexpr (KW > 1) {
#pragma unroll
    for (int c = 0; c < TT; ++c)
#pragma unroll
      for (int a = 0; a < TN; ++a) part[w][c * TN + a][lane] = acc[c][a];
    __syncthreads();
  }
  with_type(p.y_dtype, [&](auto zero) {
    typedef decltype(zero) T;
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      const int e = own(o);
      if (e >= TT * TN) break;
      i32x4 v;
      if constexpr (KW > 1) {
        v = part[0][e][lane];
#pragma unroll
        for (int i = 1; i < KW; ++i) v += part[i][e][lane];
      } else {
        v = acc[o / TN][o % TN];
      }
      store4<T>((T*)p.Y, p.ld_y, nullptr, g.i0 + 16 * (e / TN) + lr, j0 + 16 * (e % TN) + 4 * q, g.end, p.n,
                outputs(v, sx[o], sw[o], bias[o]));
    }
  });
}

// ---------------------------------------------------------------- tiles by LDS
// BT positions by BN rows of W per work-group, WT x WN waves (WK groups of them, which take the
// blocks in turn).  Each block of 128 columns goes to LDS without passing through registers
// (16-byte direct loads, a wave's load filling 8 rows of 128 bytes), S - 1 blocks ahead of the
// products, in S buffers that are variables of their own so that reading one does not wait for
// the others' loads.  Row r keeps its 16-byte chunk c at place c ^ turn(r).  A last block of fewer than
// 128 columns is taken first, through registers, with zeros behind column k.
// 4096 x 12288 x 4096, fp16 outputs: 164 to 197 us from card to card, 2.1 to 2.5 POPS (the
// library's int8 product 194, 2.1).  Matrix units busy 72 % of the cycles, at 1.6 of 2.4 GHz: a loop
// of this instruction alone on random codes reaches 3.3 POPS (4.7 on zeros; 16 x 16 x 64
// tiles 3.0), this kernel without loads and LDS reads 144 us where it takes 177, without loads
// 151, without stores 169.  16 experts of 512 positions, 4096 x 4096, take 170 us where one of
// 8192 takes 129: sixteen times the weights from HBM.  320 x 4096 x 4096 12.4 us: a work-group
// fetches 655 KB through L2.  Not kept, no gain or slower: half blocks read ahead in the 128
// x 128 tiles, 128 x 256 and 256 x 128 tiles, lines of later blocks touched ahead (5 to 8 %
// slower), experts' whole tiles before their last ones (4 to 12 % slower), experts' tiles
// made alike, four buffers of half a block in place of two of one (loads half a block earlier,
// twice the barriers: 4 to 6 % slower).

// LDS serves 16-byte reads of 16 lanes at a time, lanes 0 to 3, 12 to 15 and 20 to 27, then
// 4 to 11, 16 to 19 and 28 to 31, and so on from 32, from 64 banks of 4 bytes: two rows of 128.
// Lanes hold 16 rows at two chunks or 32 at one; of either, rows of one parity among those
// lanes take eight different places (with r & 7 for 32 rows they met in pairs: 19e6 cycles of
// conflicts in the CUs' 71e6 at 4096 x 12288 x 4096, now none; 175.2 us became 174.2, as what
// holds that case is the power of its products).
template <int M>
__device__ __forceinline__ int turn(int r) {
  return M == 32 ? (r >> 1) & 7 : r & 7;
}

template <int ROWS>
struct __attribute__((aligned(16))) Stage {
  uint8_t rows[ROWS * kBlk];
};
template <int BT, int WK, int I>
__device__ __forceinline__ Stage<BT> (&stage_x())[WK] {
  __shared__ Stage<BT> s[WK];
  return s;
}
template <int BN, int WK, int I>
__device__ __forceinline__ Stage<BN> (&stage_w())[WK] {
  __shared__ Stage<BN> s[WK];
  return s;
}

// A wave's 32 rows from i0 on by 128 bytes of outputs from j0 on (two tiles of 16-bit outputs,
// one of fp32): lanes of four neighbouring rows change parts (registers only), so that a store
// instruction writes 8 whole rows of 128 bytes.
template <typename T>
__device__ __forceinline__ void store_lines(T* __restrict__ Y, int64_t ld_y, int64_t i0, int64_t j0, int lane, int64_t m,
                                            bool stream, const f32x4 (&v)[sizeof(T) == 4 ? 4 : 8]) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
  const int lr = lane & 31, h = lane >> 5;
  uint32_t u[4][4];         // part s: 16 bytes from byte 16 (2 s + h) on
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = v[s][e];
        u[s][e] = __builtin_bit_cast(uint32_t, f);
      }
  } else {
    // the two lanes of a row: 8 outputs in a row for each
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const f32x4 a = v[2 * s], b = v[2 * s + 1];
      const u32x2 x = __builtin_bit_cast(u32x2, T4{(T)a[0], (T)a[1], (T)a[2], (T)a[3]});
      const u32x2 y = __builtin_bit_cast(u32x2, T4{(T)b[0], (T)b[1], (T)b[2], (T)b[3]});
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const auto r = __builtin_amdgcn_permlane32_swap(x[e], y[e], false, false);
        u[s][e] = r[0];
        u[s][2 + e] = r[1];
      }
    }
  }
  // four lanes of neighbouring rows and their four parts change places
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int a = 0; a < 4; a += 2) {
      const uint32_t r = other_lane<0>((lr & 1) ? u[a][e] : u[a + 1][e]);
      u[a][e] = (lr & 1) ? r : u[a][e];
      u[a + 1][e] = (lr & 1) ? u[a + 1][e] : r;
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const uint32_t r = other_lane<1>((lr & 2) ? u[a][e] : u[a + 2][e]);
      u[a][e] = (lr & 2) ? r : u[a][e];
      u[a + 2][e] = (lr & 2) ? u[a + 2][e] : r;
    }
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int64_t i = i0 + (lr & ~3) + t;
    if (i >= m) continue;
    u32x4_at2* y = (u32x4_at2*)((uint8_t*)(Y + i * ld_y + j0) + 16 * (2 * (lr & 3) + h));
    const u32x4_at2 o = {u[t][0], u[t][1], u[t][2], u[t][3]};
    if (stream) {
      keep_apart();
      __builtin_nontemporal_store(o, y);
      keep_apart();
    } else {
      *y = o;
    }
  }
}

// how a work-group keeps its buffers full
enum Flow {
  kBlocks,      // S buffers; one barrier per block
  kHalves,      // 2 buffers; half a block's codes are read into registers while the half before is multiplied
  kAhead        // S buffers; a block's codes are read into registers while the one before is multiplied
};

template <int BT, int BN, int WT, int WN, int WK, int S, Flow FLOW, bool SPLIT, bool GROUPED>
__global__ __launch_bounds__(64 * WT * WN * WK) __attribute__((amdgpu_waves_per_eu(2))) void
int8_dma_kernel(Int8Args p, int tiles_t, int tiles_n, int blocks_per_split, int* __restrict__ parts) {
  constexpr int kWavesHere = WT * WN, M = (BT / WT) % 32 == 0 && (BN / WN) % 32 == 0 ? 32 : 16;
  constexpr int TT = BT / WT / M, TN = BN / WN / M, KS = Tile<M>::kSteps;
  constexpr int kXLoads = BT / 8 / kWavesHere, kWLoads = BN / 8 / kWavesHere;
  static_assert(kXLoads * 8 * kWavesHere == BT && kWLoads * 8 * kWavesHere == BN, "loads divide over the waves");
  constexpr int kLoads = kXLoads + kWLoads;        // of a wave, per block
  static_assert((S - 1) * kLoads < 64, "counted by vmcnt");
  typedef typename Tile<M>::Sums Sums;
  const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane((t >> 6) % kWavesHere);
  const int grp = __builtin_amdgcn_readfirstlane((t >> 6) / kWavesHere);      // the wave's group
  const int lr = lane & (M - 1), q = lane / M;
  Rows g{0, p.m, 0};
  int part = 0;
  int64_t j0;
  if constexpr (GROUPED) {
    // work-groups of one XCD take neighbouring tiles of one expert, in bands as below (16
    // experts of 512 x 4096 x 4096 171 us, with bands across experts 179; 32 of 400 x 2048 143
    // and 157)
    const Experts<BT> experts(p);
    const int total = min(experts.total, tiles_t);      // offsets that decrease may ask for more
    if ((int)blockIdx.x >= total * tiles_n) return;
    const int id = (int)xcd_remap(blockIdx.x, (int64_t)total * tiles_n);
    const Part e = experts.part(p, id / tiles_n);
    if (e.expert < 0) return;
    const int of_e = id - e.before * tiles_n, band = of_e / (8 * tiles_n), in = of_e - band * 8 * tiles_n;
    const int high = min(8, Experts<BT>::tiles(e.from, e.to) - 8 * band);
    g = Experts<BT>::tile(e, 8 * band + in % high);
    j0 = (int64_t)(in / high) * BN;
  } else {
    // work-groups of one XCD take neighbouring tiles: bands of 8 tiles along X, W outermost
    const int tiles = tiles_t * tiles_n;
    part = blockIdx.x / tiles;
    const int id = (int)xcd_remap(blockIdx.x % tiles, tiles);
    const int band = id / (8 * tiles_n), in = id - band * 8 * tiles_n, high = min(8, tiles_t - 8 * band);
    g.i0 = (int64_t)(8 * band + in % high) * BT;
    j0 = (int64_t)(in / high) * BN;
  }
  const uint8_t* const W = p.W + g.expert * p.stride_w;
  const int wi = (w / WN) * (BT / WT), wj = (w % WN) * (BN / WN);      // waves of few rows spread over the SIMDs
  const int nblk = (int)((p.k + kBlk - 1) / kBlk);
  const int b0 = part * blocks_per_split, b1 = min(b0 + blocks_per_split, nblk);

  const int rows_x = (int)min<int64_t>(BT, g.end - g.i0), rows_w = (int)min<int64_t>(BN, p.n - j0);
  const bool gathered = GROUPED && p.rows != nullptr;       // rows anywhere in X, others are neighbours
  const __amdgpu_buffer_rsrc_t xb = gathered ? rsrc(p.X, (p.rows_x - 1) * p.ld_x + p.k)
                                             : rsrc(p.X + g.i0 * p.ld_x, (rows_x - 1) * p.ld_x + p.k);
  const __amdgpu_buffer_rsrc_t wb = rsrc(W + j0 * p.ld_w, (rows_w - 1) * p.ld_w + p.k);
  // a lane's row and chunk in each of the wave's loads; rows past the end repeat the last
  const auto chunk_of = [&](int l) { return (uint32_t)((lane & 7) ^ turn<M>(8 * l + (lane >> 3))) * 16; };
  uint32_t xo[kXLoads], wo[kWLoads];
#pragma unroll
  for (int j = 0; j < kXLoads; ++j) {
    const int r = min((w * kXLoads + j) * 8 + (lane >> 3), rows_x - 1);
    xo[j] = (uint32_t)((gathered ? row_of(p, g.i0 + r) : r) * p.ld_x) + chunk_of(w * kXLoads + j);
  }
#pragma unroll
  for (int j = 0; j < kWLoads; ++j)
    wo[j] = (uint32_t)(min((w * kWLoads + j) * 8 + (lane >> 3), rows_w - 1) * p.ld_w) + chunk_of(w * kWLoads + j);
  const auto fetch_one = [&](Stage<BT>& x, Stage<BN>& s, int b, int l) {
    if (l < kXLoads) load16_to_lds(xb, x.rows + (w * kXLoads + l) * 8 * kBlk, xo[l], b * kBlk);
    else load16_to_lds(wb, s.rows + (w * kWLoads + l - kXLoads) * 8 * kBlk, wo[l - kXLoads], b * kBlk);
  };
  const auto fetch = [&](auto i, int b) {
#pragma unroll
    for (int l = 0; l < kLoads; ++l) fetch_one(stage_x<BT, WK, i.value>()[grp], stage_w<BN, WK, i.value>()[grp], b, l);
  };
  Sums acc[TT][TN];
#pragma unroll
  for (int c = 0; c < TT; ++c)
#pragma unroll
    for (int a = 0; a < TN; ++a) acc[c][a] = Sums(0);
  // a lane's first chunk of its row in the wave's first tile of each operand; the others by xor
  const uint32_t x0 = (uint32_t)((wi + lr) * kBlk + ((q ^ turn<M>(lr)) * 16));
  const uint32_t w0 = (uint32_t)((wj + lr) * kBlk + ((q ^ turn<M>(lr)) * 16));
  const auto pick = [&](const uint8_t* rows, uint32_t a, int tile, int step) {
    return *(const u32x4*)(rows + (a ^ (step * (64 / M) * 16)) + tile * M * kBlk);
  };
  // a last block of fewer than 128 columns, through registers: all loads first, and LDS
  // written once the next blocks' loads are under way
  const bool tail = b1 == nblk && (p.k % kBlk) != 0;
  constexpr int kAll = 64 * kWavesHere * WK, kTail = ((BT + BN) * 8 + kAll - 1) / kAll;
  u32x4 tail_v[kTail];
  if (tail) {
#pragma unroll
    for (int i = 0; i < kTail; ++i) {
      const int id = t + i * kAll, r = min(id >> 3, BT + BN - 1);
      const uint8_t* row = r < BT ? p.X + (GROUPED ? row_of(p, g.i0 + min(r, rows_x - 1)) : g.i0 + min(r, rows_x - 1)) * p.ld_x
                                  : W + (j0 + min(r - BT, rows_w - 1)) * p.ld_w;
      tail_v[i] = load_inside(row, (int64_t)(nblk - 1) * kBlk + 16 * (id & 7), p.k);
    }
  }
  const auto put_tail = [&]() {
    if (!tail) return;
#pragma unroll
    for (int i = 0; i < kTail; ++i) {
      const int id = t + i * kAll, r = id >> 3, c = id & 7;
      const u32x4 v = align_chunk(tail_v[i], (int64_t)(nblk - 1) * kBlk + 16 * c, p.k);
      if (r < BT) *(u32x4*)(stage_x<BT, WK, 0>()[0].rows + r * kBlk + ((c ^ turn<M>(r)) * 16)) = v;
      else if (r < BT + BN) *(u32x4*)(stage_w<BN, WK, 0>()[0].rows + (r - BT) * kBlk + ((c ^ turn<M>(r - BT)) * 16)) = v;
    }
  };
  // the groups take the blocks in turn
  const int count = b1 - b0, steps = (count + WK - 1) / WK;
  const auto block_of = [&](int at) { return !tail ? b0 + at : at == 0 ? nblk - 1 : b0 + at - 1; };
  // behind the last block, block 0, which is not used: with a fetch on every path the
  // counts of outstanding loads are known, and no read waits for a later block
  const auto next = [&](int step) { return step * WK + grp < count ? block_of(step * WK + grp) : 0; };
  // the scales and biases go to LDS: asked for before the first block, written while it comes
  __shared__ __attribute__((aligned(16))) float sxs[SPLIT ? 1 : BT], sws[SPLIT ? 4 : BN], biases[SPLIT ? 4 : BN];
  float sx_t = 0.f, sw_t = 0.f, bias_t = -0.f;
  if constexpr (!SPLIT) {
    static_assert(BT <= kAll && BN <= kAll, "one of each per thread");
    const int64_t j = min(j0 + t, p.n - 1);
    sx_t = scale_of(p, min(g.i0 + t, g.end - 1));
    sw_t = p.sw[(int64_t)g.expert * p.n + j];
    if (p.bias) with_type(p.y_dtype, [&](auto zero) { bias_t = (float)((const decltype(zero)*)p.bias)[(int64_t)g.expert * p.n + j]; });
  }
  if (!tail || grp > 0) fetch(std::integral_constant<int, 0>{}, next(0));
  if constexpr (!SPLIT) {
    if (t < BT) sxs[t] = sx_t;
    if (t < BN) {
      sws[t] = sw_t;
      biases[t] = bias_t;
    }
  }
  int step = 0;
  // one(stage, whether the group has a block): only in the last step may it have none
  const auto run = [&](auto&& one) {
    while (step + S < steps) static_for<0, S>([&](auto i) { one(i, true); });
    static_for<0, S>([&](auto i) {
      if (step < steps) one(i, WK == 1 || step * WK + grp < count);
    });
  };
  if constexpr (FLOW == kBlocks) {
    static_for<1, S - 1>([&](auto i) { fetch(i, next(i.value)); });
    put_tail();
    run([&](auto i, bool has) {
      constexpr int h = i.value, to = (h + S - 1) % S;
      // this block has arrived, and every wave is done with the buffer that is filled next
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * kLoads) : "memory");
      const int b = next(step + S - 1);
      ++step;
      if (!has) return;           // nothing follows: nothing to fetch
      const uint8_t* xs = stage_x<BT, WK, h>()[grp].rows;
      const uint8_t* ws = stage_w<BN, WK, h>()[grp].rows;
      constexpr int kSpread = TT * TN >= 8 ? KS / 2 : 0;      // steps beside which the next loads are issued
      if constexpr (kSpread == 0) fetch(std::integral_constant<int, to>{}, b);
      u32x4 wv[2][TN], xv[2][TT];
      const auto read = [&](int set, int k) {
#pragma unroll
        for (int a = 0; a < TN; ++a) wv[set][a] = pick(ws, w0, a, k);
#pragma unroll
        for (int c = 0; c < TT; ++c) xv[set][c] = pick(xs, x0, c, k);
      };
      read(0, 0);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        if (k + 1 < KS) read((k + 1) & 1, k + 1);
        if constexpr (kSpread > 0) {
#pragma unroll
          for (int l = 0; l < kLoads; ++l)
            if (l * kSpread / kLoads == k) fetch_one(stage_x<BT, WK, to>()[grp], stage_w<BN, WK, to>()[grp], b, l);
        }
        if (!GROUPED || wi < rows_x) {         // products of rows that there are
#pragma unroll
          for (int c = 0; c < TT; ++c)
#pragma unroll
            for (int a = 0; a < TN; ++a) acc[c][a] = Tile<M>::product(wv[k & 1][a], xv[k & 1][c], acc[c][a]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    });
  } else if constexpr (FLOW == kHalves) {
    static_assert(S == 2 && WK == 1, "two buffers, one group");
    constexpr int kHalf = KS / 2, kReads = kHalf * (TN + TT), kSlots = kHalf * TN * TT;
    u32x4 wv[2][kHalf][TN], xv[2][kHalf][TT];
    // read l of the half `set` of a block
    const auto read = [&](int set, const Stage<BT>& x, const Stage<BN>& s, int l) {
      const int k = l / (TN + TT), i = l % (TN + TT);
      if (i < TN) wv[set][k][i] = pick(s.rows, w0, i, set * kHalf + k);
      else xv[set][k][i - TN] = pick(x.rows, x0, i - TN, set * kHalf + k);
    };
    put_tail();
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    fetch(std::integral_constant<int, 1>{}, next(1));
#pragma unroll
    for (int l = 0; l < kReads; ++l) read(0, stage_x<BT, WK, 0>()[grp], stage_w<BN, WK, 0>()[grp], l);
    // tiles: those of the wave's rows that there are, where it is not all
    const auto blocks = [&](auto all, int tiles) {
      const auto half = [&](int set, auto&& meanwhile) {
#pragma unroll
        for (int e = 0; e < kSlots; ++e) {
          const int k = e / (TN * TT), c = e % (TN * TT) / TN, a = e % TN;
          meanwhile(e);
          if (all || c < tiles) acc[c][a] = Tile<M>::product(wv[set][k][a], xv[set][k][c], acc[c][a]);
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      run([&](auto i, bool) {
        constexpr int h = i.value, to = h ^ 1;
        half(0, [&](int e) {
#pragma unroll
          for (int l = 0; l < kReads; ++l)
            if (l * kSlots / kReads == e) read(1, stage_x<BT, WK, h>()[grp], stage_w<BN, WK, h>()[grp], l);
        });
        // the next block has arrived, and every wave has read this one
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        const int b = next(step + 2);
        ++step;
        half(1, [&](int e) {
#pragma unroll
          for (int l = 0; l < kLoads; ++l)
            if (l * kSlots / 2 / kLoads == e) fetch_one(stage_x<BT, WK, h>()[grp], stage_w<BN, WK, h>()[grp], b, l);
#pragma unroll
          for (int l = 0; l < kReads; ++l)
            if (l * kSlots / kReads == e) read(0, stage_x<BT, WK, to>()[grp], stage_w<BN, WK, to>()[grp], l);
        });
      });
    };
    const int tiles = GROUPED ? __builtin_amdgcn_readfirstlane((rows_x - wi + M - 1) / M) : TT;
    if (!GROUPED || tiles >= TT) blocks(std::true_type{}, TT);
    else blocks(std::false_type{}, tiles);
  } else {
    static_assert(S % 2 == 0, "two sets of registers in turn");
    static_for<1, S>([&](auto i) { fetch(i, next(i.value)); });
    put_tail();
    u32x4 wv[2][KS][TN], xv[2][KS][TT];
    const auto read = [&](int set, const Stage<BT>& x, const Stage<BN>& s, int k) {
#pragma unroll
      for (int a = 0; a < TN; ++a) wv[set][k][a] = pick(s.rows, w0, a, k);
#pragma unroll
      for (int c = 0; c < TT; ++c) xv[set][k][c] = pick(x.rows, x0, c, k);
    };
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 1) * kLoads) : "memory");
#pragma unroll
    for (int k = 0; k < KS; ++k) read(0, stage_x<BT, WK, 0>()[grp], stage_w<BN, WK, 0>()[grp], k);
    run([&](auto i, bool has) {
      constexpr int h = i.value, set = h & 1, nx = (h + 1) % S;
      // the next block has arrived, and every wave has read this one
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * kLoads) : "memory");
      const int b = next(step + S);
      ++step;
      if (!has) return;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        read(set ^ 1, stage_x<BT, WK, nx>()[grp], stage_w<BN, WK, nx>()[grp], k);
#pragma unroll
        for (int l = 0; l < kLoads; ++l)
          if (l * KS / kLoads == k) fetch_one(stage_x<BT, WK, h>()[grp], stage_w<BN, WK, h>()[grp], b, l);
#pragma unroll
        for (int c = 0; c < TT; ++c)
#pragma unroll
          for (int a = 0; a < TN; ++a) acc[c][a] = Tile<M>::product(wv[set][k][a], xv[set][k][c], acc[c][a]);
        __builtin_amdgcn_sched_barrier(0);
      }
    });
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // unused fetches write LDS: not after this work-group's end
  if constexpr (WK > 1) {
    // group 1's sums are added to group 0's through stage 0's rows of X, as many fours of each
    // lane at a time as fit
    constexpr int kG = Tile<M>::kGroups, kSums = TT * TN * kG;
    constexpr int kFit = WK * (int)sizeof(Stage<BT>::rows) / (16 * 64 * kWavesHere);
    static_assert(WK == 2 && kFit >= 1, "two groups");
    i32x4* const sums = (i32x4*)stage_x<BT, WK, 0>()[0].rows + w * kFit * 64 + lane;
#pragma unroll
    for (int e0 = 0; e0 < kSums; e0 += kFit) {
      // every wave's reads are done: of the last block, then of the sums before
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (grp == 1) {
#pragma unroll
        for (int e = e0; e < e0 + kFit && e < kSums; ++e) sums[(e - e0) * 64] = group<M>(acc[e / kG / TN][e / kG % TN], e % kG);
      }
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      if (grp == 0) {
#pragma unroll
        for (int e = e0; e < e0 + kFit && e < kSums; ++e) {
          const i32x4 other = sums[(e - e0) * 64];
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[e / kG / TN][e / kG % TN][4 * (e % kG) + r] += other[r];
        }
      }
    }
    if (grp == 1) return;
  }
  if constexpr (SPLIT) {
    int* const mine = parts + (int64_t)part * p.m * p.n;
#pragma unroll
    for (int c = 0; c < TT; ++c)
#pragma unroll
      for (int a = 0; a < TN; ++a)
#pragma unroll
        for (int e = 0; e < 4 * Tile<M>::kGroups; ++e) {
          const int64_t i = g.i0 + wi + M * c + lr, j = j0 + wj + M * a + 8 * (e / 4) + 4 * q + e % 4;
          if (i < p.m && j < p.n) mine[i * p.n + j] = acc[c][a][e];
        }
  }
  if constexpr (!SPLIT) {
    float sx[TT];
#pragma unroll
    for (int c = 0; c < TT; ++c) sx[c] = sxs[wi + M * c + lr];
    with_type(p.y_dtype, [&](auto zero) {
      typedef decltype(zero) T;
      // Outputs of more than 80 MiB go past the caches' keeping where rows start at 64 bytes:
      // 4096 x 12288 x 4096 fp16 188 us against 205, 1000 x 50000 x 1536 fp32 126 against 163.
      // Other rows share lines: 1000 x 50001 x 1536 fp32 196 against 171, 4096 x 12289 x 4096
      // fp16 216 against 222.  64 MiB: 4096 x 8192 x 1024 fp16 47 against 44.
      const bool stream = (uint64_t)p.m * (uint64_t)p.n * sizeof(T) > (uint64_t)80 << 20 &&
                          ((uintptr_t)p.Y | (uintptr_t)p.ld_y * sizeof(T)) % 64 == 0;
      constexpr int kLine = 128 / (int)sizeof(T);         // outputs of a store_lines
      constexpr bool kLines = M == 32 && (BN / WN) % kLine == 0;
      const bool lines = kLines && j0 + wj + BN / WN <= p.n;       // the same for the whole wave
      constexpr int kPer = kLines ? kLine / 32 : 1, kV = kPer * Tile<M>::kGroups;      // tiles and fours at a time
#pragma unroll
      for (int a = 0; a < TN; a += kPer)
#pragma unroll
        for (int c = 0; c < TT; ++c) {
          asm volatile("" ::: "memory");        // scales and biases read anew: kept, they would cost 64 registers
          f32x4 v[kV];
#pragma unroll
          for (int e = 0; e < kV; ++e) {
            const int at = wj + M * a + 8 * e + 4 * q;
            v[e] = outputs(group<M>(acc[c][a + e / Tile<M>::kGroups], e % Tile<M>::kGroups), sx[c], *(const f32x4*)(sws + at),
                           *(const f32x4*)(biases + at));
          }
          if constexpr (kLines) {
            if (lines) {
              store_lines<T>((T*)p.Y, p.ld_y, g.i0 + wi + 32 * c, j0 + wj + 32 * a, lane, g.end, stream, v);
              continue;
            }
          }
#pragma unroll
          for (int e = 0; e < kV; ++e)
            store4<T>((T*)p.Y, p.ld_y, nullptr, g.i0 + wi + M * c + lr, j0 + wj + M * a + 8 * e + 4 * q, g.end, p.n, v[e]);
        }
    });
  }
}

// Y from the parts of a product split over k
__global__ __launch_bounds__(256) void int8_sum_kernel(Int8Args p, int splits, const int* __restrict__ parts) {
  const int64_t size = p.m * p.n;
  with_type(p.y_dtype, [&](auto zero) {
    typedef decltype(zero) T;
    for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < size; id += (int64_t)gridDim.x * 256) {
      const int64_t i = id / p.n, j = id - i * p.n;
      int v = parts[id];
      for (int s = 1; s < splits; ++s) v += parts[s * size + id];
      ((T*)p.Y)[i * p.ld_y + j] = (T)output(v, p.sx[i], p.sw[j], p.bias ? (float)((const T*)p.bias)[j] : -0.f);
    }
  });
}

// tiles of `bt` positions that the experts' parts of m positions can have at most
int64_t most_tiles(int64_t m, int64_t experts, int bt) {
  const int64_t used = std::min(m, experts);
  return (m + used * (bt - 1)) / bt;
}

// the direct loads need 16-byte rows, 32-bit offsets and a whole block
bool direct(const Int8Args& p) {
  const bool one_x = p.rows ? p.rows_x <= 1 : p.m <= 1;
  const uint64_t ld_x = one_x ? 0 : (uint64_t)p.ld_x, ld_w = p.n > 1 ? (uint64_t)p.ld_w : 0;
  const uint64_t st = p.experts > 1 ? (uint64_t)p.stride_w : 0;
  return p.k >= kBlk && (((uintptr_t)p.X | (uintptr_t)p.W | ld_x | ld_w | st) & 15) == 0 &&
         std::max(ld_x, ld_w) <= (uint64_t(1) << 22) &&
         (!p.rows || (uint64_t)p.rows_x * (uint64_t)p.ld_x <= uint64_t(1) << 31);
}

template <bool GROUPED, int BT, int BN, int WT, int WN, int WK, int S, Flow FLOW>
hipError_t launch_dma(const Int8Plan& plan, const Int8Args& p, int* ws, hipStream_t s) {
  const int tt = (int)(GROUPED ? most_tiles(p.m, p.experts, BT) : cdiv(p.m, BT)), tn = (int)cdiv(p.n, BN);
  const int per = (int)cdiv(cdiv(p.k, kBlk), plan.splits);
  if constexpr (BT == 64 && BN == 32 && !GROUPED) {       // the only tiles of products that are split
    if (plan.splits > 1) {
      int8_dma_kernel<BT, BN, WT, WN, WK, S, FLOW, true, false>
          <<<tt * tn * plan.splits, 64 * WT * WN * WK, 0, s>>>(p, tt, tn, per, ws);
      int8_sum_kernel<<<(unsigned)std::min<int64_t>(cdiv(p.m * p.n, 256), 2048), 256, 0, s>>>(p, plan.splits, ws);
      return hipGetLastError();
    }
  }
  int8_dma_kernel<BT, BN, WT, WN, WK, S, FLOW, false, GROUPED>
      <<<tt * tn, 64 * WT * WN * WK, 0, s>>>(p, tt, tn, per, nullptr);
  return hipGetLastError();
}

template <int TT, int TN, int KW, int R, bool GROUPED>
hipError_t launch_few(const Int8Args& p, bool dma, hipStream_t s) {
  const auto grid = [&](int tn, int kw) {
    return dim3((unsigned)cdiv(p.n, 16 * tn * (kFewWaves / kw)), (unsigned)(GROUPED ? most_tiles(p.m, p.experts, 16 * TT) : 1));
  };
  if (dma) int8_few_kernel<TT, TN, KW, R, true, GROUPED><<<grid(TN, KW), 64 * kFewWaves, 0, s>>>(p);
  else int8_few_kernel<TT, 1, kFewWaves, 1, false, GROUPED><<<grid(1, kFewWaves), 64 * kFewWaves, 0, s>>>(p);
  return hipGetLastError();
}

template <bool GROUPED>
hipError_t launch(const Int8Plan& plan, const Int8Args& p, void* ws, hipStream_t s) {
  const bool dma = direct(p);
  switch (plan.kind) {
    case kInt8Few16: return launch_few<1, 1, kFewWaves, 2, GROUPED>(p, dma, s);
    case kInt8Few16Own:
      if constexpr (GROUPED) return launch_few<1, 1, 1, 2, GROUPED>(p, dma, s);
    case kInt8Few16OwnDeep: return launch_few<1, 1, 1, 4, GROUPED>(p, dma, s);
    case kInt8Few32: return launch_few<2, 2, kFewWaves, 2, GROUPED>(p, dma, s);
    case kInt8Few64:
      if constexpr (!GROUPED) return launch_few<4, 1, kFewWaves, 2, GROUPED>(p, dma, s);
    default: break;
  }
  if (!dma) {
    int8_tile_kernel<GROUPED><<<dim3((unsigned)cdiv(p.n, kTile), (unsigned)(GROUPED ? most_tiles(p.m, p.experts, kTile) : cdiv(p.m, kTile))),
                                256, 0, s>>>(p);
    return hipGetLastError();
  }
  int* const parts = (int*)ws;
  if constexpr (!GROUPED) {
    switch (plan.kind) {
      case kInt8T64x32: return launch_dma<GROUPED, 64, 32, 2, 2, 2, 4, kAhead>(plan, p, parts, s);
      case kInt8T64x64: return launch_dma<GROUPED, 64, 64, 2, 2, 2, 4, kAhead>(plan, p, parts, s);
      case kInt8T96x64: return launch_dma<GROUPED, 96, 64, 2, 2, 2, 3, kBlocks>(plan, p, parts, s);
      default: break;
    }
  }
  switch (plan.kind) {
    case kInt8T128x64: return launch_dma<GROUPED, 128, 64, 2, 2, 2, 3, kBlocks>(plan, p, parts, s);
    case kInt8T128x128Two: return launch_dma<GROUPED, 128, 128, 2, 2, 2, 2, kBlocks>(plan, p, parts, s);
    case kInt8T256x256: return launch_dma<GROUPED, 256, 256, 2, 4, 1, 2, kHalves>(plan, p, parts, s);
    default: return launch_dma<GROUPED, 128, 128, 2, 2, 1, 2, kBlocks>(plan, p, parts, s);
  }
}

}  // namespace

// Which kernel (times: bf16 outputs, k = 4096 unless given, graph replays).
//   few rows: up to 16 in waves that share rows of W (1 x 1536 4.2 us, with rows of their own
//     6.0), in waves with rows of their own where those fill the card (1 x 11008 9.9 against
//     11.0); up to 32 by 32 (29 x 5001 7.7, in tiles 8.0; but 32 x 11008 12.4 against 10.9); up to
//     64 only where small tiles would not fill the card either (64 x 4096 7.8 against 8.2).
//     Along k > 8192 few work-groups are too slow: split tiles.
//   the smallest tiles that one round of 256 CUs covers: 128 x 4096 8.5 us in 64 x 32 tiles
//     against 11.5 in the next; 320 x 4096 12.4 (96 x 64) against 21.3 and 14.6; 512 x 4096
//     16.4 (128 x 64) against 21.7 and 20.7; 1024 x 4096 24.0 (128 x 128, two groups) against
//     31.8 and 26.5 (one group).
//   k in parts where one round is less than half full.
//   beyond one round, 128 x 128 or 256 x 256, by their times in us: a 128 x 128 tile adds
//     0.0064 + 0.00216 per block of k, a round of the larger ones takes 9.1 + 1.78, one of r
//     tiles 0.38 + 0.62 r / 256 of that.  2048 x 4096 40 against 47 us, 4096 x 4096 78 against
//     61, 4096 x 12288 209 against 171.
Int8Plan int8_plan(int64_t m, int64_t n, int64_t k) {
  Int8Plan p{kInt8T128x128, 1, 0};
  const bool few = k > 8192 && n <= 1024 ? false : m <= 16 ? true : m <= 32 ? n <= 8192 : m <= 64 && n <= 4096 && k <= 4096;
  if (few) {
    p.kind = m <= 16 ? (n > 8192 ? kInt8Few16OwnDeep : kInt8Few16) : m <= 32 ? kInt8Few32 : kInt8Few64;
    return p;
  }
  const struct { int kind, bt, bn; } small[] = {
      {kInt8T64x32, 64, 32}, {kInt8T64x64, 64, 64}, {kInt8T96x64, 96, 64}, {kInt8T128x64, 128, 64},
      {kInt8T128x128Two, 128, 128}};
  for (const auto& c : small) {
    const int64_t tiles = cdiv(m, c.bt) * cdiv(n, c.bn);
    if (tiles > 256) continue;
    p.kind = c.kind;
    if (c.kind == kInt8T64x32) {         // the larger ones are taken from 129 tiles on: nothing to split
      const int64_t nblk = cdiv(k, kBlk), splits = std::max<int64_t>(1, std::min<int64_t>(256 / tiles, nblk / 16));
      p.splits = (int)cdiv(nblk, cdiv(nblk, splits));     // none empty
      if (p.splits > 1) p.ws_bytes = (size_t)p.splits * m * n * sizeof(int);
    }
    return p;
  }
  const int64_t t128 = cdiv(m, 128) * cdiv(n, 128), t256 = cdiv(m, 256) * cdiv(n, 256), rest = t256 % 256;
  const double nblk = (double)cdiv(k, kBlk), rounds = (double)(t256 / 256) + (rest > 0 ? 0.38 + 0.62 * rest / 256 : 0.0);
  p.kind = rounds * (9.1 + 1.78 * nblk) < t128 * (0.0064 + 0.00216 * nblk) ? kInt8T256x256 : kInt8T128x128;
  return p;
}

// By the mean part of the experts that can have one, as the parts themselves are known on the
// device alone (times as above, experts x n; k = 4096 and 1500).
//   few rows: waves of 16 with rows of W of their own (8 x 1536, 6 each: 8.6 us with k = 1500,
//     256 x 256 tiles 24), with more blocks under way along a long k (2 of 8 x 4096, one each: 9.4
//     against 11.4); where a long k and many rows of W leave each CU many waves anyway, waves that
//     share them (64 x 1536, 4 each: 70 against 75), of 32 positions from 7 on (32 x 2048, 16
//     each: 62 against 68).  They pay up to 16 positions each (32 x 2048, 24: 27 against 24 in 128 x
//     128 tiles), up to 24 where such tiles do not fill the card (8 x 1536: 9.5 against 15.9), and
//     those of 32 up to 32 (32 x 2048, 24: 68 against 72; 40: 82 against 83).
//     Narrow stacks, used * n of some thousands and k > 2048, have too few waves of rows of their own
//     to fill the card and would do better with the ones that share them: one position each of 2 x
//     1536 9.9 against 6.8, of 8 x 512 9.7 against 7.2, of 8 x 1536 13.5 and 13.4; with k = 1500 both
//     take 5.6 at 2 x 1536.  The rule has no such border.
//   tiles: 128 x 64, 128 x 128 by two groups of waves, 128 x 128 as one, two or more rounds of
//     CUs take them (8 x 1536, 100 each: 13.6, 16.0 and 17.1; 200: 22.4, 16.4 and 17.3; 400: 32, 28
//     and 21); 256 x 256 for large parts that fill the card, whose last tiles cost less as waves
//     without rows leave out their products (16 x 4096, 512: 183 against 212; 200: 124 and 128).
Int8Plan int8_grouped_plan(int64_t m, int64_t n, int64_t k, int64_t experts) {
  const int64_t used = std::min(m, experts), each = cdiv(m, used);
  const int64_t t128 = used * cdiv(each, 128) * cdiv(n, 128), t256 = used * cdiv(each, 256) * cdiv(n, 256);
  int kind = kInt8T128x128;
  if (k > 2048 && used * n >= 49152 && each <= 32) kind = each <= 6 ? kInt8Few16 : kInt8Few32;
  else if (each <= 16 || (each <= 24 && t128 < 256)) kind = k > 2048 ? kInt8Few16OwnDeep : kInt8Few16Own;
  else if (t128 <= 128) kind = kInt8T128x64;
  else if (t128 <= 256) kind = kInt8T128x128Two;
  else if (each >= 300 && t256 >= 192) kind = kInt8T256x256;
  return Int8Plan{kind, 1, 0};
}

hipError_t int8_matmul_launch(const Int8Plan& plan, const Int8Args& p, void* ws, hipStream_t s) {
  return launch<false>(plan, p, ws, s);
}

hipError_t int8_grouped_launch(const Int8Args& p, hipStream_t s) {
  return launch<true>(int8_grouped_plan(p.m, p.n, p.k, p.experts), p, nullptr, s);
}

}  // namespace gptq
