// Device code that the products of block-scaled matrices share, in 8 bits
// (fp8_matmul.hip) and in 4 (fp4_matmul.hip): their arguments, the dealing of
// tiles, the DMA into LDS, and the output from 16 x 16 accumulators.
#pragma once

#include <algorithm>
#include <type_traits>

#include "fp8_internal.h"

namespace muonh {
namespace fp8 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr;

struct Operand {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows, ld;  // ld: bytes per row of codes
  int64_t sld;       // bytes per row of scales
  int sshift;        // scale row of matrix row r: r >> sshift
};

struct MatArgs {
  Operand a, b;      // m x k, n x k
  int64_t m, n;
  int nkb;           // 128-blocks of k
  void* out;
  int64_t ldo;
  int accumulate;
  int odd;           // 2-byte results: some rows of out start off a multiple of 4 bytes
  float* part;       // partial sums [split][m][pld], or nullptr
  int64_t pld;
  int splits, per;   // k blocks per split
  int tm, tn;        // tile grid
};

// ---- output ------------------------------------------------------------------
// v: CNT consecutive results of row i from column j (16 bytes or a part of
// them). Guards the column end; the caller guards the row.
template <typename T, int CNT>
__device__ __forceinline__ void put(const MatArgs& a, int64_t i, int64_t j, const float (&v)[CNT]) {
  T* p = static_cast<T*>(a.out) + i * a.ldo + j;
  // at any multiple of T's size: gfx950 takes vector accesses at any address
  typedef T vecT __attribute__((ext_vector_type(CNT), aligned(sizeof(T))));
  if (j + CNT <= a.n) {
    vecT w;
    if (a.accumulate) {
      const vecT o = *reinterpret_cast<const vecT*>(p);
#pragma unroll
      for (int q = 0; q < CNT; ++q) w[q] = (T)((float)o[q] + v[q]);
    } else {
#pragma unroll
      for (int q = 0; q < CNT; ++q) w[q] = (T)v[q];
    }
    *reinterpret_cast<vecT*>(p) = w;
  } else {
#pragma unroll
    for (int q = 0; q < CNT; ++q)
      if (j + q < a.n) p[q] = (T)((a.accumulate ? (float)p[q] : 0.f) + v[q]);
  }
}

// Fragment row r of b's fragment f within a wave's 64 columns -> column. For
// 2-byte results (PAIR) neighbouring fragments hold 8 consecutive columns.
template <bool PAIR>
__device__ __forceinline__ int b_row(int f, int r) {
  return PAIR ? 32 * (f >> 1) + 8 * (r >> 2) + 4 * (f & 1) + (r & 3) : 16 * f + r;
}

// One row's 16 + 16 bytes of 2-byte results of a lane (columns 8 g .. +7 and
// 32 + 8 g .. +7 from p's 64; the 4 lanes l%16, g = l/16, hold the row) to an
// address that is 2 bytes off a multiple of 4 where `off`: vector stores to
// such addresses run at a third of the rate, so those rows are stored one
// element on, each lane taking the first element of its right neighbour, the
// first and the last element of the 64 by themselves.
__device__ __forceinline__ void put_odd(__bf16* p, u32x4 x, u32x4 y, int lane, bool off, bool live) {
  const int g = lane >> 4, next = ((lane + 16) & 63) << 2;
  const uint32_t nx = (uint32_t)__builtin_amdgcn_ds_bpermute(next, (int)x[0]);
  const uint32_t ny = (uint32_t)__builtin_amdgcn_ds_bpermute(next, (int)y[0]);
  if (!live) return;
  typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
  typedef uint32_t u32x3_a2 __attribute__((ext_vector_type(3), aligned(2)));
  uint16_t* q = reinterpret_cast<uint16_t*>(p) + 8 * g;
  if (!off) {
    *reinterpret_cast<u32x4_a2*>(q) = x;
    *reinterpret_cast<u32x4_a2*>(q + 32) = y;
    return;
  }
  auto shift = [](const u32x4& v, uint32_t n) {
    return u32x4{(v[0] >> 16) | (v[1] << 16), (v[1] >> 16) | (v[2] << 16), (v[2] >> 16) | (v[3] << 16),
                 (v[3] >> 16) | (n << 16)};
  };
  if (g == 0) *q = (uint16_t)x[0];
  *reinterpret_cast<u32x4_a2*>(q + 1) = shift(x, g == 3 ? ny : nx);
  const u32x4 z = shift(y, ny);
  if (g < 3) {
    *reinterpret_cast<u32x4_a2*>(q + 33) = z;
  } else {
    *reinterpret_cast<u32x3_a2*>(q + 33) = u32x3_a2{z[0], z[1], z[2]};
    q[39] = (uint16_t)(y[3] >> 16);
  }
}

// Lanes 2i and 2i + 1 hold 16 bytes x and, 64 bytes on, 16 bytes y of rows r
// and r + 1. Afterwards their x are both of row r (x of lane 2i, y of lane
// 2i + 1) and their y both of row r + 1, so that a store of x writes 8 rows of
// 128 bytes instead of 16 of 64.
template <typename V>
__device__ __forceinline__ void pair_rows(V& x, V& y, bool odd_lane) {
  i32x4 u = __builtin_bit_cast(i32x4, x), v = __builtin_bit_cast(i32x4, y);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int got = __builtin_amdgcn_mov_dpp(odd_lane ? u[e] : v[e], 0xB1, 0xF, 0xF, false);  // quad [1,0,3,2]
    u[e] = odd_lane ? got : u[e];
    v[e] = odd_lane ? v[e] : got;
  }
  x = __builtin_bit_cast(V, u);
  y = __builtin_bit_cast(V, v);
}

// Stores a wave's 16 NA rows x 64 columns from row i0, column j0: acc[q][f],
// b's fragment q, a's fragment f; lane l holds row 16 f + l%16 and columns
// b_row(q, 4 (l/16) ..+3).
template <typename T, int NA, bool ADD>
__device__ __forceinline__ void store_rows(const MatArgs& a, int64_t i0, int64_t j0, int lane,
                                           const f32x4 (&acc)[4][NA]) {
  const int r16 = lane & 15, g = lane >> 4, r2 = r16 & ~1;
  const bool odd_lane = lane & 1;
  // rows of fragments whose old values are read together
  constexpr int kGroup = NA % 3 == 0 ? 3 : sizeof(T) == 2 && NA % 4 == 0 ? 4 : 2;
  if (j0 + 64 > a.n) {  // the tile ends in these columns
#pragma unroll
    for (int f = 0; f < NA; ++f) {
      const int64_t i = i0 + 16 * f + r16;
      if (i >= a.m) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {acc[q][f][0], acc[q][f][1], acc[q][f][2], acc[q][f][3]};
        put<T, 4>(a, i, j0 + b_row<sizeof(T) == 2>(q, 4 * g), v);
      }
    }
  } else if constexpr (sizeof(T) == 4) {
    typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
    const int64_t j = j0 + 4 * g + (odd_lane ? 16 : 0);
    auto at = [&](int f, int q, int y) {
      return reinterpret_cast<f32x4_a4*>(static_cast<float*>(a.out) +
                                         min(i0 + 16 * f + r2 + y, a.m - 1) * a.ldo + j + 16 * q);
    };
#pragma unroll
    for (int f0 = 0; f0 < NA; f0 += kGroup) {
      f32x4 old[kGroup][4];
      if constexpr (ADD) {
#pragma unroll
        for (int f = 0; f < kGroup; ++f)
#pragma unroll
          for (int q = 0; q < 4; ++q) old[f][q] = *at(f0 + f, q & 2, q & 1);
      }
#pragma unroll
      for (int f = 0; f < kGroup; ++f)
#pragma unroll
        for (int q = 0; q < 4; q += 2) {
          f32x4 x = acc[q][f0 + f], y = acc[q + 1][f0 + f];
          pair_rows(x, y, odd_lane);
          if constexpr (ADD) {
            x += old[f][q];
            y += old[f][q + 1];
          }
          const int64_t i = i0 + 16 * (f0 + f) + r2;
          if (i < a.m) *at(f0 + f, q, 0) = x;
          if (i + 1 < a.m) *at(f0 + f, q, 1) = y;
        }
    }
  } else {
    typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
    typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
#pragma unroll
    for (int f0 = 0; f0 < NA; f0 += kGroup) {
      u32x4 old[kGroup][2];
      if constexpr (ADD) {
#pragma unroll
        for (int f = 0; f < kGroup; ++f)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            old[f][h] = *reinterpret_cast<const u32x4_a2*>(
                static_cast<const __bf16*>(a.out) + min(i0 + 16 * (f0 + f) + r16, a.m - 1) * a.ldo + j0 +
                32 * h + 8 * g);
      }
#pragma unroll
      for (int f = 0; f < kGroup; ++f) {
        u32x4 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4 u = acc[2 * h][f0 + f], v = acc[2 * h + 1][f0 + f];
          if constexpr (ADD) {
            const bf16x8 o = __builtin_bit_cast(bf16x8, old[f][h]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              u[e] += (float)o[e];
              v[e] += (float)o[4 + e];
            }
          }
          const bf16x8 c = {(__bf16)u[0], (__bf16)u[1], (__bf16)u[2], (__bf16)u[3],
                            (__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
          w[h] = __builtin_bit_cast(u32x4, c);
        }
        if (a.odd) {
          const int64_t i = i0 + 16 * (f0 + f) + r16;
          __bf16* p = static_cast<__bf16*>(a.out) + i * a.ldo + j0;
          put_odd(p, w[0], w[1], lane, (reinterpret_cast<uintptr_t>(p) & 2) != 0, i < a.m);
        } else {
          pair_rows(w[0], w[1], odd_lane);
          const int64_t i = i0 + 16 * (f0 + f) + r2;
          __bf16* p = static_cast<__bf16*>(a.out) + i * a.ldo + j0 + 8 * g + (odd_lane ? 32 : 0);
          if (i < a.m) *reinterpret_cast<u32x4_a4*>(p) = w[0];
          if (i + 1 < a.m) *reinterpret_cast<u32x4_a4*>(p + a.ldo) = w[1];
        }
      }
    }
  }
}

template <typename T, int NA>
__device__ __forceinline__ void store_wave(const MatArgs& a, int64_t i0, int64_t j0, int lane,
                                           const f32x4 (&acc)[4][NA]) {
  if (a.accumulate) store_rows<T, NA, true>(a, i0, j0, lane, acc);
  else store_rows<T, NA, false>(a, i0, j0, lane, acc);
}

// Block -> tile. Blocks are dealt to the 8 XCDs in turn; each XCD takes a
// contiguous eighth of the tile list, so the tiles resident on it share
// operand rows in its L2. The list runs in bands of 8 tile rows, down each
// tile column of the band. False: the block has no tile.
__device__ __forceinline__ bool map_tile(const MatArgs& a, int b, int& ti, int& tj) {
  const int64_t tot = (int64_t)a.tm * a.tn;
  const int x = b & 7, lo = (int)((x * tot) >> 3), hi = (int)(((x + 1) * tot) >> 3);
  const int t = lo + (b >> 3);
  if (t >= hi) return false;
  const int per_band = 8 * a.tn, band = t / per_band, rr = t - band * per_band;
  const int h = min(8, a.tm - 8 * band);
  ti = 8 * band + rr % h;
  tj = rr / h;
  return true;
}
int map_grid(int64_t tiles) { return (int)(8 * ceil_div(tiles, 8)); }

// Waits until at most VM of this wave's memory operations are outstanding and
// its LDS reads have retired, then the workgroup's barrier; neither memory
// accesses nor MFMAs move across.
template <int VM>
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((VM & 0xF) | ((VM >> 4) << 14) | (0x7 << 4));
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A pointer that is the same in all lanes, in scalar registers (the compiler
// may compute uniform values in vector registers, which the DMA's base cannot be).
// A memory instruction must not read a scalar register in the 5 cycles after a vector
// instruction wrote it; the compiler sees to that for its own instructions, not for
// those in inline asm. So the wait is here, between the reads of the lanes and any use of the
// pointer: without it a DMA took a stale half of its base (GPU memory fault).
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
  asm volatile("s_nop 4" : "+s"(lo), "+s"(hi));
  return reinterpret_cast<const uint8_t*>(((uint64_t)hi << 32) | lo);
}

// LDS DMA: lane l's 16 (4) bytes at base + off go to LDS bytes m0 + 16 l (4 l).
// No register results; waits and barriers are the caller's.
__device__ __forceinline__ void dma16s(const uint8_t* base, uint32_t off, uint32_t m0) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(m0) : "memory");
}
__device__ __forceinline__ void dma4s(const uint8_t* base, uint32_t off, uint32_t m0) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "{m0}"(m0) : "memory");
}

// out (+)= the partial sums, split by split in order; 4 columns per thread.
template <typename T>
__global__ __launch_bounds__(256) void k_matmul_join(MatArgs a) {
  const int64_t q4 = a.pld >> 2;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= a.m * q4) return;
  const int64_t i = e / q4, j = (e - i * q4) * 4;
  f32x4 s = {};
  for (int p = 0; p < a.splits; ++p)
    s += *reinterpret_cast<const f32x4*>(a.part + ((int64_t)p * a.m + i) * a.pld + j);
  const float v[4] = {s[0], s[1], s[2], s[3]};
  put<T, 4>(a, i, j, v);
}

constexpr int kWaves = 8;  // of the kernels whose waves share out a tile's k blocks
static_assert(kWaves == 8, "k_matmul_small deals eighths");

// Sums the waves' tiles (acc[q][f] as in store_wave) through LDS, in wave
// order, and stores the result: wave w's sums in red[w * pitch ..], NA * NB * 64
// units of 16 bytes.
template <typename T, int NA, int NB>
__device__ __forceinline__ void join_waves(const MatArgs& a, int split, int64_t i0, int64_t j0, f32x4* red,
                                           int pitch, const f32x4 (&acc)[NB][NA]) {
  constexpr bool kPair = sizeof(T) == 2 && NB >= 2;
  constexpr int kUnits = NA * NB * 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int q = 0; q < NB; ++q)
#pragma unroll
    for (int f = 0; f < NA; ++f) red[wave * pitch + (f * NB + q) * 64 + lane] = acc[q][f];
  __syncthreads();
  // a thread takes one unit (4 columns of a row), or for 2-byte results two
  // units of neighbouring fragments (8 columns)
  constexpr int kStep = kPair ? 2 : 1;
  for (int e = tid; e < kUnits / kStep; e += 64 * kWaves) {
    const int l = e & 63, fq = (e >> 6) * kStep, f = fq / NB, q = fq % NB;
    f32x4 s[kStep];
#pragma unroll
    for (int h = 0; h < kStep; ++h) {
      s[h] = red[(fq + h) * 64 + l];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s[h] += red[w * pitch + (fq + h) * 64 + l];
    }
    const int64_t i = i0 + 16 * f + (l & 15), j = j0 + b_row<kPair>(q, 4 * (l >> 4));
    if (i >= a.m) continue;
    if (a.part) {
      float* p = a.part + ((int64_t)split * a.m + i) * a.pld + j;
#pragma unroll
      for (int h = 0; h < kStep; ++h)
        if (j + 4 * h < a.pld) *reinterpret_cast<f32x4*>(p + 4 * h) = s[h];
    } else {
      float v[4 * kStep];
#pragma unroll
      for (int h = 0; h < kStep; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[4 * h + c] = s[h][c];
      put<T, 4 * kStep>(a, i, j, v);
    }
  }
}

}  // namespace
}  // namespace fp8
}  // namespace muonh
