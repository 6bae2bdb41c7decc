// What the products of 8-bit codes share: chunks of 16 codes of a row, direct loads to LDS,
// the order of tiles over the XCDs, and the stores of a wave's tiles.
#pragma once

#include "gptq_internal.h"

namespace gptq {
namespace {

constexpr int kBlk = 128;               // columns of a block
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef __bf16 bf16;

// 16 codes of a row from column c; columns from k on read as zero.  The row's last
// chunk is taken from its last 16 bytes and shifted.
__device__ __forceinline__ u32x4 load_chunk(const uint8_t* __restrict__ row, int64_t c, int64_t k) {
  if (c + 16 <= k) return *(const u32x4_any*)(row + c);
  if (c >= k) return u32x4{0u, 0u, 0u, 0u};
  if (k >= 16) {
    const auto v = __builtin_bit_cast(unsigned __int128, (u32x4)(*(const u32x4_any*)(row + k - 16)));
    return __builtin_bit_cast(u32x4, v >> (8 * (int)(c + 16 - k)));
  }
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (c + e < k) v[e >> 2] |= (uint32_t)row[c + e] << (8 * (e & 3));
  return v;
}

// The same in two steps for k >= 16, so that the loads of several chunks are under way
// together: 16 bytes that lie in the row, then the codes of column c on to the front.
__device__ __forceinline__ u32x4 load_inside(const uint8_t* __restrict__ row, int64_t c, int64_t k) {
  return *(const u32x4_any*)(row + min(c, k - 16));
}
__device__ __forceinline__ u32x4 align_chunk(u32x4 v, int64_t c, int64_t k) {
  const int past = (int)(c + 16 - k);
  if (past >= 16) return u32x4{0u, 0u, 0u, 0u};
  return past <= 0 ? v : __builtin_bit_cast(u32x4, __builtin_bit_cast(unsigned __int128, v) >> (8 * past));
}

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
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
  typedef T T4 __attribute__((ext_vector_type(4), aligned(2)));     // at any element
  if (i >= m || j >= n) return;
  T* y = Y + i * ld_y + j;
  if (j + 4 <= n) {
    if (bias) {
      const T4 b = *(const T4*)(bias + j);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += (float)b[r];
    }
    *(T4*)y = T4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (j + r < n) y[r] = (T)(v[r] + (bias ? (float)bias[j + r] : 0.f));
  }
}

// a lane's v from the lane whose number differs in bit 0 or bit 1
template <int BIT>
__device__ __forceinline__ uint32_t other_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, BIT == 0 ? 0xB1 : 0x4E, 0xf, 0xf, true);
}

// an empty statement, to keep the compiler from joining a store past the caches with the
// plain one of the other branch, which would drop the hint
__device__ __forceinline__ void keep_apart() { asm volatile(""); }

// A wave's 16 rows from i0 on x 64 outputs from j0 on, four neighbouring tiles: v[a] holds
// outputs 16 a + 4 q .. + 3 of row lr.  Lanes swap parts (registers only), so that one store
// instruction writes whole rows of 64: 4 rows of fp32, 8 of 16 bits.  stream: past the
// caches' keeping.
template <typename T>
__device__ __forceinline__ void store_rows64(T* __restrict__ Y, int64_t ld_y, const T* __restrict__ bias, int64_t i0, int64_t j0,
                                             int lr, int q, int64_t m, int64_t n, bool stream, const f32x4 (&v)[4]) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  typedef T T4_any __attribute__((ext_vector_type(4), aligned(2)));
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
  if (j0 + 64 > n) {         // the same for the whole wave
#pragma unroll
    for (int a = 0; a < 4; ++a) store4<T>(Y, ld_y, bias, i0 + lr, j0 + 16 * a + 4 * q, m, n, v[a]);
    return;
  }
  if constexpr (sizeof(T) == 4) {
    // four lanes of neighbouring rows and their four tiles change places
    uint32_t u[4][4];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float f = v[a][e];
        u[a][e] = __builtin_bit_cast(uint32_t, f);
      }
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
    const int64_t j = j0 + 16 * (lr & 3) + 4 * q;
    f32x4 b = {0.f, 0.f, 0.f, 0.f};
    if (bias) b = *(const T4_any*)(bias + j);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int64_t i = i0 + (lr & ~3) + t;
      f32x4 f;
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = __builtin_bit_cast(float, u[t][e]) + b[e];
      if (i >= m) continue;
      if (stream) {
        keep_apart();
        __builtin_nontemporal_store(T4_any(f), (T4_any*)(Y + i * ld_y + j));
        keep_apart();
      } else {
        *(T4_any*)(Y + i * ld_y + j) = f;
      }
    }
  } else {
    uint32_t u[4][2];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      f32x4 f = v[a];
      if (bias) {
        const T4_any b = *(const T4_any*)(bias + j0 + 16 * a + 4 * q);
#pragma unroll
        for (int r = 0; r < 4; ++r) f[r] += (float)b[r];
      }
      const u32x2 w = __builtin_bit_cast(u32x2, T4{(T)f[0], (T)f[1], (T)f[2], (T)f[3]});
      u[a][0] = w[0];
      u[a][1] = w[1];
    }
    // the four lanes of a row: 16 outputs in a row for each ...
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const auto r = __builtin_amdgcn_permlane32_swap(u[a][h], u[a + 2][h], false, false);
        u[a][h] = r[0];
        u[a + 2][h] = r[1];
      }
#pragma unroll
      for (int a = 0; a < 4; a += 2) {
        const auto r = __builtin_amdgcn_permlane16_swap(u[a][h], u[a + 1][h], false, false);
        u[a][h] = r[0];
        u[a + 1][h] = r[1];
      }
    }
    // ... and two neighbouring rows: the even lane takes the first 8 of both, the odd one the others
    const bool odd = lr & 1;
    u32x4_at2 even_row, odd_row;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = u[e >> 1][e & 1], hi = u[2 + (e >> 1)][e & 1];
      const uint32_t r = other_lane<0>(odd ? lo : hi);
      even_row[e] = odd ? r : lo;
      odd_row[e] = odd ? hi : r;
    }
    const int64_t i = i0 + (lr & ~1);
    T* y = Y + i * ld_y + j0 + 16 * q + 8 * (lr & 1);
    if (stream) {
      keep_apart();
      if (i < m) __builtin_nontemporal_store(even_row, (u32x4_at2*)y);
      if (i + 1 < m) __builtin_nontemporal_store(odd_row, (u32x4_at2*)(y + ld_y));
      keep_apart();
    } else {
      if (i < m) *(u32x4_at2*)y = even_row;
      if (i + 1 < m) *(u32x4_at2*)(y + ld_y) = odd_row;
    }
  }
}

typedef __attribute__((address_space(3))) void lds_void;

// `bytes` bytes from a wave-uniform address
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  const uint64_t u = ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32) |
                     (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)u, (short)0, __builtin_amdgcn_readfirstlane((int)bytes),
                                           0x00020000);
}

template <int I, int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<I + 1, N>(f);
  }
}
// 16 bytes per lane from r + voffset + soffset to LDS at `to` + 16 * lane
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t voffset, int soffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, voffset, soffset, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(__amdgpu_buffer_rsrc_t r, float* to, uint32_t voffset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 4, voffset, 0, 0, 0);
}

}  // namespace
}  // namespace gptq
