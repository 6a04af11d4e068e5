// Products of block-scaled e4m3 matrices on gfx950 (formats and contract:
// include/muonh.h): out[i][j] = sum_k a[i][k] b[j][k], both operands read
// along their rows.
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 covers exactly one scale block of 128
// along k and applies one E8M0 scale per operand row itself, so scales cost
// no vector arithmetic on the accumulators. Lane l of a fragment holds row
// l%16 and 32 of the 128 codes: 16-byte chunks l/16 and l/16 + 4 of the row
// (any assignment of k to lanes is right as long as both operands use the
// same one; this one reads LDS without bank conflicts, see frag_off).
//
// Within one such instruction, though, the products are added in groups whose
// terms keep no bits below 2^-13 of the largest: small products beside a large
// one are lost, and where large ones cancel, nothing of the result need be
// left (fp32 sums of the same codes have a 2^-24 there). So products widen the
// codes to bf16 with their scale applied (exact) and use
// v_mfma_f32_16x16x32_bf16, whose sums are accurate to fp32 (measured 1e-7 at
// k = 8192), at half the matrix rate, for either result type. The 8-bit
// instructions serve callers that ask for them (MUONH_FP8_FAST).
#include <algorithm>
#include <type_traits>

#include "fp8_choice.h"
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

// 8 codes (two dwords) widened to bf16 times a power of two: exact for values
// that bf16 holds (multiples of 2^-133 below 2^128).
__device__ __forceinline__ bf16x8 widen8(int lo, int hi, float s) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
// 2^(byte - 127) for bytes 1 .. 254. Of a scale the conversions take the exponent
// field: 0 stands for 2^-127 and 255 for NaN, as in E8M0.
__device__ __forceinline__ float scale_of(int byte) { return __int_as_float(byte << 23); }

// acc[x][y] += X_x Y_y^T for one block of k: NX x NY products of 16 x 16.
// sx, sy: scale bytes of the fragments' rows (in the low 8 bits).
// WIDE: through bf16.
template <bool WIDE, int NX, int NY>
__device__ __forceinline__ void mma_block(const i32x8 (&x)[NX], const i32x8 (&y)[NY],
                                          const int (&sx)[NX], const int (&sy)[NY],
                                          f32x4 (&acc)[NX][NY]) {
  if constexpr (!WIDE) {
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
      for (int j = 0; j < NY; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x[i], y[j], acc[i][j], 0, 0, 0,
                                                                     sx[i], 0, sy[j]);
  } else {
    float fx[NX], fy[NY];
#pragma unroll
    for (int i = 0; i < NX; ++i) fx[i] = scale_of(sx[i] & 255);
#pragma unroll
    for (int j = 0; j < NY; ++j) fy[j] = scale_of(sy[j] & 255);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      bf16x8 wx[NX], wy[NY];
#pragma unroll
      for (int i = 0; i < NX; ++i) wx[i] = widen8(x[i][2 * q], x[i][2 * q + 1], fx[i]);
#pragma unroll
      for (int j = 0; j < NY; ++j) wy[j] = widen8(y[j][2 * q], y[j][2 * q + 1], fy[j]);
#pragma unroll
      for (int i = 0; i < NX; ++i)
#pragma unroll
        for (int j = 0; j < NY; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wx[i], wy[j], acc[i][j], 0, 0, 0);
    }
  }
}

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
__device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(u >> 32));
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

// ---------------------------------------------------------------------------
// LDS layout of the tiled kernels: an LDS row holds the 128 codes of one
// operand row; 16-byte chunk c of row r sits at position c ^ (r & 7), which
// spreads the 16 rows x 4 chunks of a fragment read over the banks (measured:
// 510 GB/s per CU against 290 with chunk pairs 2g, 2g + 1 per lane). The DMA
// writes LDS linearly, so the lane's source chunk is permuted instead. Rows
// past the matrix reload its last row; their results are not stored.
//
// The b operand is the MFMA's first one, so a lane's 4 accumulators are 4
// consecutive columns of one row of out. For 2-byte results b's rows are
// also dealt to the fragments so that a lane holds 8 consecutive columns in
// two neighbouring fragments (b_row): 16-byte stores, 64-byte runs per row,
// which lane pairs join to runs of 128 (pair_rows; on the 8-bit path 8192 x
// 6144 x 128 with bf16 results 26.8 -> 24.7 us, 8192 x 6144 x 2048 95 -> 90).
//
// 128 x 128 tiles, a ring of 4 LDS stages of one k block (32 KB each). The 8
// waves form two groups of 4 (2 x 2, wave tile 64 x 64), one wave of each per
// SIMD, that take the k blocks in turn: in phase p one group reads block p's
// fragments and sends the DMA of block p+3, into the stage that the other
// group read in phase p-1, while the other group multiplies block p-1. A
// block lands within the two phases after its own, waited for by the waves
// that sent it. Every phase ends in a barrier that retires LDS reads. At the
// end each wave hands half of its sums to its partner in the other group.
//
// With one group of 4 waves, reads, DMA and MFMAs follow one another: 0.5-0.7
// us a block however many stages were in flight; with two groups of 64 x 32
// waves that share each block, the reads and DMA of a phase outlast its 8
// MFMAs: 0.45 us.
// ---------------------------------------------------------------------------
constexpr int kOpStage = kT * kBlock;     // 16 KB
constexpr int kStageBytes = 2 * kOpStage; // A, then B
constexpr int kScaleBytes = 2 * kT * 4;   // 4 bytes of each row of both operands
constexpr int kRing = 4;

template <typename T, bool WIDE>
__global__ __launch_bounds__(512, 2) void k_matmul_tile(MatArgs a) {
  constexpr bool kPair = sizeof(T) == 2;
  __shared__ __attribute__((aligned(1024))) char lds[kRing * (kStageBytes + kScaleBytes)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int w4 = wave & 3, group = wave >> 2;
  int ti, tj;
  if (!map_tile(a, blockIdx.x, ti, tj)) return;
  const int nk = a.nkb;
  const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr)lds;
  const int64_t ra = (int64_t)ti * kT, rb = (int64_t)tj * kT;

  // DMA of a block by one group: waves 0, 1 fill a's 128 rows, waves 2, 3 b's;
  // 8 instructions of 8 rows (lane l: row l / 8, position l % 8), then the
  // scales of 64 rows. Offsets from the tile's first row.
  const bool is_a = w4 < 2;
  const Operand& op = is_a ? a.a : a.b;
  const int64_t first = is_a ? ra : rb;
  auto row = [&](int lr) {
    return min(first + (is_a ? lr : 64 * (lr >> 6) + b_row<kPair>((lr & 63) >> 4, lr & 15)), op.rows - 1);
  };
  uint32_t off[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int lr = 64 * (w4 & 1) + 8 * q + (lane >> 3);
    off[q] = (uint32_t)(row(lr) - first) * (uint32_t)op.ld + (uint32_t)(((lane & 7) ^ (lr & 7)) << 4);
  }
  const int64_t s0 = first >> op.sshift;
  const uint32_t soff = (uint32_t)((row(64 * (w4 & 1) + lane) >> op.sshift) - s0) * (uint32_t)op.sld;
  const uint8_t* codes = op.codes + first * op.ld;
  const uint8_t* scales = op.scales + s0 * op.sld;
  const uint32_t dst = base + (is_a ? 0 : kOpStage) + (w4 & 1) * 64 * kBlock;
  const uint32_t sdst = base + kRing * kStageBytes + w4 * 256;
  auto fetch_part = [&](int s, int c) {  // quarter c
    const int slot = s & (kRing - 1);
    const int64_t k = (int64_t)s * kBlock;
#pragma unroll
    for (int q = 2 * c; q < 2 * c + 2; ++q)
      dma16s(codes + k, off[q], dst + slot * kStageBytes + q * 1024);
    if (c == 3) dma4s(scales + (s & ~3), soff, sdst + slot * kScaleBytes);
  };
  auto fetch = [&](int s) {
#pragma unroll
    for (int c = 0; c < 4; ++c) fetch_part(s, c);
  };
  constexpr int kOps = 9;  // memory operations of fetch()

  const int wm = w4 >> 1, wn = w4 & 1, r16 = lane & 15, g = lane >> 4;
  const int foff = r16 * kBlock + ((g ^ (r16 & 7)) << 4);  // fragment rows start at multiples of 16
  f32x4 acc[4][4];  // [b fragment][a fragment]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
  // Phases s (read, fetch) and s + 1 (multiply) of block s. No branch between
  // the phases: the compiler moves MFMAs across barriers into later basic
  // blocks, and then keeps two sets of fragments alive.
  auto block = [&](int s, auto more) {
    constexpr bool kMore = decltype(more)::value;
    const char* st = lds + (s & (kRing - 1)) * kStageBytes;
    const char* ss = lds + kRing * kStageBytes + (s & (kRing - 1)) * kScaleBytes;
    const int sh = (s & 3) * 8;
    auto frag = [&](const char* p) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(p + foff);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(p + (foff ^ 64));
      return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    i32x8 fa[4], fb[4];
    int sa[4], sb[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      fa[f] = frag(st + (64 * wm + 16 * f) * kBlock);
      fb[f] = frag(st + kOpStage + (64 * wn + 16 * f) * kBlock);
      sa[f] = *reinterpret_cast<const int*>(ss + (64 * wm + 16 * f + r16) * 4);
      sb[f] = *reinterpret_cast<const int*>(ss + (kT + 64 * wn + 16 * f + r16) * 4);
      // between the reads: one after the other, reads and DMA outlast the
      // other group's MFMAs
      if constexpr (kMore) fetch_part(s + 3, f);
    }
    // block s + 1, sent by this group two phases ago, has landed
    stage_barrier<(kMore ? kOps : 0)>();
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      sa[f] >>= sh;
      sb[f] >>= sh;
    }
    mma_block<WIDE, 4, 4>(fb, fa, sb, sa, acc);
    stage_barrier<63>();
  };
  if (group == 0) {
    if (nk > 1) fetch(1);
    stage_barrier<63>();
  } else {
    if (nk > 0) fetch(0);
    if (nk > 2) {
      fetch(2);
      stage_barrier<kOps>();  // block 0 has landed
    } else {
      stage_barrier<0>();
    }
    stage_barrier<63>();  // phase 0
  }
  int s = group;
  for (; s + 3 < nk; s += 2) block(s, std::true_type{});
  for (; s < nk; s += 2) block(s, std::false_type{});
  if ((nk & 1) == group) stage_barrier<63>();  // the other group's last phase

  // Sums: group 0 keeps a's fragments 0, 1 of the wave tile, group 1 the
  // others; the rest goes through LDS (8 KB a wave, all DMA and reads are done).
  f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int f = 0; f < 2; ++f)
      red[((wave ^ 4) * 8 + q * 2 + f) * 64 + lane] = group == 0 ? acc[q][2 + f] : acc[q][f];
  __syncthreads();
  f32x4 sum[4][2];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int f = 0; f < 2; ++f)
      sum[q][f] = (group == 0 ? acc[q][f] : acc[q][2 + f]) + red[(wave * 8 + q * 2 + f) * 64 + lane];
  store_wave<T, 2>(a, ra + 64 * wm + 32 * group, rb + 64 * wn, lane, sum);
}

// ---------------------------------------------------------------------------
// 256 x 256 tiles, 8 waves (2 x 4, wave tile 128 x 64), two LDS stages of one
// k block (2 x 64 KB): products with enough tiles for the chip. 192 x 256
// tiles (FA = 3 instead of 4 fragments of a per half wave tile) where they
// fill the chip better: 6144 x 2048 x 8192, 192 tiles or 256 for 256 CUs, takes
// 139 instead of 154 us with fp32 results, 133 instead of 151 with bf16 ones and
// 78 instead of 80.5 on the 8-bit path (fewer active CUs clock higher). 256 x 192
// tiles gained 3-7 % there. 8192^3 takes 721 us with fp32 results (1525 TFLOP/s),
// 683 with bf16 ones (1610) and 374 on the 8-bit path (2940): power is what bounds
// all of them (about 2 GHz).
//
// The waves form two groups of 4, one wave of each per SIMD, that take turns
// phase by phase: one group's 16 MFMAs (64 widened ones) run while the other
// reads LDS and issues DMA, so the matrix cores see no gap and MFMA waves issue no memory
// instruction. A wave's block of k takes two turns, 64 of its 128 rows each
// (A0, A1), which keeps the fragments at 64 registers beside 128
// accumulators. Phases of block s, group 0 | group 1:
//   4s    read B, A0         | multiply A1 of s-1
//   4s+1  multiply A0        | read B, A0
//   4s+2  read A1            | multiply A0
//   4s+3  multiply A1        | read A1
// A stage is refilled part by part as it falls free, 24 DMA instructions in
// each of three phases, between the LDS reads, each at least three phases
// before block s+2 needs it:
//   4s+2  group 0: B rows 0-159, b's scales (B was last read in 4s+1)
//   4s+3  group 1: B rows 160-255, A rows 0-95 (group 0's, last read in 4s+2)
//   4s+4  group 0: A rows 96-255 (group 1's A1 was last read in 4s+3), a's scales
// (rows 96-191 of 192; group 0 reads the first half of A's rows, group 1 the other)
// and waited for at the end of 4s+7. Every phase ends in a barrier that
// retires the wave's LDS reads.
// ---------------------------------------------------------------------------
constexpr int kBigOp = kB * kBlock;            // 32 KB
constexpr int kBigStage = 2 * kBigOp;          // A, then B
constexpr int kBigScales = 2 * kB * 4;         // a's rows, then b's: 4 k blocks each

template <typename T, bool WIDE, int FA, int G>
__device__ __forceinline__ void big_loop(const MatArgs& a, const char* lds, uint32_t base, const uint8_t* pa,
                                         const uint8_t* pb, const uint8_t* sca, const uint8_t* scb,
                                         const uint32_t (&off)[10], uint32_t soa, uint32_t sob, int nk,
                                         int wave, int lane, f32x4 (&acc)[4][2 * FA]) {
  const int w4 = wave & 3, r16 = lane & 15, g = lane >> 4;
  const int foff = r16 * kBlock + ((g ^ (r16 & 7)) << 4);
  i32x8 fa[FA], fb[4];
  int sa[FA], sb[4];
  auto frag = [&](const char* p) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(p + foff);
    const i32x4 hi = *reinterpret_cast<const i32x4*>(p + (foff ^ 64));
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  // scale byte (in the low 8 bits) of the lane's row of a fragment; rows of b
  // follow a's 256
  auto scale = [&](int s, int row) {
    const char* q = lds + 2 * kBigStage + (s & 1) * kBigScales;
    return *reinterpret_cast<const int*>(q + (row + r16) * 4) >> ((s & 3) * 8);
  };
  // the DMA of this group for block s: `part` 0 in phase 4(s-2)+2 or +3, 1
  // (group 0) in phase 4(s-2)+4; instruction q
  constexpr int kA1 = 2 * FA - 3;         // a's rows by a wave of group 0, 8 per instruction
  constexpr int kOps[2] = {6, kA1 + 1};   // memory operations of a part
  auto fetch = [&](int s, int part, int q) {
    const uint32_t st = base + (s & 1) * kBigStage;
    const uint32_t sc = base + 2 * kBigStage + (s & 1) * kBigScales + w4 * 256;
    const int64_t k = (int64_t)s * kBlock;
    if (G == 1) {
      if (q < 3) dma16s(pb + k, off[q], st + kBigOp + (20 + 3 * w4 + q) * 1024);
      else dma16s(pa + k, off[q], st + (3 * w4 + q - 3) * 1024);
    } else if (part == 0) {
      if (q < 5) dma16s(pb + k, off[q], st + kBigOp + (5 * w4 + q) * 1024);
      else dma4s(scb + (s & ~3), sob, sc + kB * 4);
    } else {
      if (q < kA1) dma16s(pa + k, off[5 + q], st + (12 + kA1 * w4 + q) * 1024);
      else dma4s(sca + (s & ~3), soa, sc);
    }
  };
  auto fetch_all = [&](int s, int part) {
#pragma unroll
    for (int q = 0; q < kOps[part]; ++q) fetch(s, part, q);
  };
  // reads of block s with the DMA of block t (FETCH) between them
  auto load_a = [&](int s, int half, auto dma, int t) {
    const char* p = lds + (s & 1) * kBigStage + (2 * G + half) * 16 * FA * kBlock;
#pragma unroll
    for (int f = 0; f < FA; ++f) {
      fa[f] = frag(p + 16 * f * kBlock);
      sa[f] = scale(s, (2 * G + half) * 16 * FA + 16 * f);
      if constexpr (decltype(dma)::value)  // spread over the fragments
#pragma unroll
        for (int q = kOps[0] * f / FA; q < kOps[0] * (f + 1) / FA; ++q) fetch(t, 0, q);
    }
  };
  auto load_b = [&](int s, auto dma, int t) {
    const char* p = lds + (s & 1) * kBigStage + kBigOp + 64 * w4 * kBlock;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      fb[f] = frag(p + 16 * f * kBlock);
      sb[f] = scale(s, kB + 64 * w4 + 16 * f);
      if constexpr (decltype(dma)::value)
#pragma unroll
        for (int q = kOps[1] * f / 4; q < kOps[1] * (f + 1) / 4; ++q) fetch(t, 1, q);
    }
  };
  auto mul = [&](int half) {
    if constexpr (!WIDE) {
#pragma unroll
      for (int f = 0; f < FA; ++f)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[q][FA * half + f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              fb[q], fa[f], acc[q][FA * half + f], 0, 0, 0, sb[q], 0, sa[f]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bf16x8 wb[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) wb[q] = widen8(fb[q][2 * k], fb[q][2 * k + 1], scale_of(sb[q] & 255));
#pragma unroll
        for (int f = 0; f < FA; ++f) {
          const bf16x8 wa = widen8(fa[f][2 * k], fa[f][2 * k + 1], scale_of(sa[f] & 255));
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[q][FA * half + f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[q], wa, acc[q][FA * half + f], 0, 0, 0);
        }
      }
    }
  };
  fetch_all(0, 0);
  if (G == 0) fetch_all(0, 1);
  if (nk > 1) {
    fetch_all(1, 0);
    stage_barrier<kOps[0]>();
  } else {
    stage_barrier<0>();
  }
  if (G == 1) stage_barrier<63>();  // phase 0
  // One block of k; LEFT: how many more blocks follow (2: at least two). The
  // loop body has no branch: the compiler moves MFMAs across barriers into
  // later basic blocks, and then keeps two sets of fragments alive.
  auto block = [&](int s, auto left) {
    constexpr int kLeft = decltype(left)::value;
    constexpr std::false_type none{};
    load_b(s, std::bool_constant<G == 0 && kLeft >= 1>{}, s + 1);
    load_a(s, 0, none, 0);
    stage_barrier<63>();
    mul(0);
    stage_barrier<63>();
    load_a(s, 1, std::bool_constant<kLeft >= 2>{}, s + 2);
    // the end of phase 4s+3: block s+1 has landed; what was just issued for
    // block s+2 may be in flight
    constexpr int kLand = kLeft >= 2 ? kOps[0] : 0;
    stage_barrier<(G == 1 ? kLand : 63)>();
    mul(1);
    stage_barrier<(G == 0 ? kLand : 63)>();
  };
  int s = 0;
  for (; s + 2 < nk; ++s) block(s, std::integral_constant<int, 2>{});
  if (s + 1 < nk) block(s++, std::integral_constant<int, 1>{});
  block(s, std::integral_constant<int, 0>{});
  if (G == 0) stage_barrier<63>();  // group 1's last phase
}

template <typename T, bool WIDE, int FA>
__global__ __launch_bounds__(512, 2) void k_matmul_big(MatArgs a) {
  constexpr bool kPair = sizeof(T) == 2;
  __shared__ __attribute__((aligned(1024))) char lds[2 * kBigStage + 2 * kBigScales];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int ti, tj;
  if (!map_tile(a, blockIdx.x, ti, tj)) return;
  const int nk = a.nkb;
  const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr)lds;
  // Tile bases, and this lane's source offsets for each DMA instruction: LDS
  // rows 8 i .. +7 of an operand, lane l: row l / 8, position l % 8.
  const int64_t ra = (int64_t)ti * 64 * FA, rb = (int64_t)tj * kB;
  const uint8_t* pa = scalar(a.a.codes + ra * a.a.ld);
  const uint8_t* pb = scalar(a.b.codes + rb * a.b.ld);
  const int w4 = wave & 3;
  auto off_a = [&](int i) {
    const int lr = 8 * i + (lane >> 3);
    return (uint32_t)(min(ra + lr, a.m - 1) - ra) * (uint32_t)a.a.ld + (uint32_t)(((lane & 7) ^ (lr & 7)) << 4);
  };
  auto off_b = [&](int i) {
    const int lr = 8 * i + (lane >> 3);
    const int r = 64 * (lr >> 6) + b_row<kPair>((lr & 63) >> 4, lr & 15);
    return (uint32_t)(min(rb + r, a.n - 1) - rb) * (uint32_t)a.b.ld + (uint32_t)(((lane & 7) ^ (lr & 7)) << 4);
  };
  f32x4 acc[4][2 * FA];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2 * FA; ++j) acc[i][j] = f32x4{};
  uint32_t off[10];
  if (wave < 4) {
#pragma unroll
    for (int q = 0; q < 5; ++q) off[q] = off_b(5 * w4 + q);
#pragma unroll
    for (int q = 0; q < 2 * FA - 3; ++q) off[5 + q] = off_a(12 + (2 * FA - 3) * w4 + q);
    const int64_t r = min(ra + 64 * w4 + lane, a.m - 1);
    const int64_t c = min(rb + 64 * w4 + b_row<kPair>(lane >> 4, lane & 15), a.n - 1);
    const int64_t a0 = ra >> a.a.sshift, b0 = rb >> a.b.sshift;
    const uint32_t soa = (uint32_t)((r >> a.a.sshift) - a0) * (uint32_t)a.a.sld;
    const uint32_t sob = (uint32_t)((c >> a.b.sshift) - b0) * (uint32_t)a.b.sld;
    big_loop<T, WIDE, FA, 0>(a, lds, base, pa, pb, scalar(a.a.scales + a0 * a.a.sld),
                             scalar(a.b.scales + b0 * a.b.sld), off, soa, sob, nk, wave, lane, acc);
  } else {
#pragma unroll
    for (int q = 0; q < 6; ++q) off[q] = q < 3 ? off_b(20 + 3 * w4 + q) : off_a(3 * w4 + q - 3);
    big_loop<T, WIDE, FA, 1>(a, lds, base, pa, pb, nullptr, nullptr, off, 0, 0, nk, wave, lane, acc);
  }
  store_wave<T, 2 * FA>(a, ra + 32 * FA * (wave >> 2), rb + 64 * w4, lane, acc);
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

// ---------------------------------------------------------------------------
// 16 x 16 tiles: the waves of a workgroup take its k blocks in turn, with
// fragments read straight from global memory (two sets in registers: the next
// block's loads run under the current one's MFMA), and join their sums in
// wave order. Short dependent chains and every code of b read once, for
// single tokens and other products whose time is latency.
// ---------------------------------------------------------------------------
template <typename T, bool WIDE>
__global__ __launch_bounds__(64 * kWaves) void k_matmul_direct(MatArgs a) {
  __shared__ __attribute__((aligned(16))) f32x4 red[kWaves * 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  int ti, tj;
  if (!map_tile(a, blockIdx.x, ti, tj)) return;
  const int64_t i0 = (int64_t)ti * 16, j0 = (int64_t)tj * 16;
  const int kb1 = a.nkb;
  const int64_t ra = min(i0 + r16, a.m - 1), rb = min(j0 + r16, a.n - 1);
  const uint8_t *ca = a.a.codes + ra * a.a.ld + 16 * g, *cb = a.b.codes + rb * a.b.ld + 16 * g;
  const uint8_t *sa = a.a.scales + (ra >> a.a.sshift) * a.a.sld, *sb = a.b.scales + (rb >> a.b.sshift) * a.b.sld;
  struct Set {
    i32x8 a[1], b[1];
    int sa[1], sb[1];
  };
  auto frag = [](const uint8_t* p) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(p), hi = *reinterpret_cast<const i32x4*>(p + 64);
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  auto load = [&](Set& s, int kb) {
    const int64_t k = (int64_t)kb * kBlock;
    s.a[0] = frag(ca + k);
    s.b[0] = frag(cb + k);
    s.sa[0] = sa[kb];
    s.sb[0] = sb[kb];
  };
  f32x4 acc[1][1] = {{f32x4{}}};
  int kb = wave;
  Set s0, s1;
  if (kb < kb1) load(s0, kb);
  for (; kb + kWaves < kb1; kb += 2 * kWaves) {
    load(s1, kb + kWaves);
    mma_block<WIDE, 1, 1>(s0.b, s0.a, s0.sb, s0.sa, acc);
    if (kb + 2 * kWaves < kb1) load(s0, kb + 2 * kWaves);
    mma_block<WIDE, 1, 1>(s1.b, s1.a, s1.sb, s1.sa, acc);
  }
  if (kb < kb1) mma_block<WIDE, 1, 1>(s0.b, s0.a, s0.sb, s0.sa, acc);
  join_waves<T, 1, 1>(a, 0, i0, j0, red, 64, acc);
}

// ---------------------------------------------------------------------------
// 64 x 64 tiles, 8 waves that share out the tile's k blocks: for products
// with too few larger tiles for the chip. Each wave has an LDS stage of its
// own (64 rows of both operands, 16 KB, and their scales), filled by DMA in
// whole cache lines; it reads the fragments into registers, sends the DMA of
// its next block after them and multiplies. Nothing waits for another wave
// before the sums are joined (in LDS, in wave order). Reading fragments from
// global memory instead, 64 bytes of a line at a time, took 1.5 times as long.
// ---------------------------------------------------------------------------
constexpr int kSmallOp = kS * kBlock;                       // 8 KB
constexpr int kSmallStage = 2 * kSmallOp + 2 * kS * 4;      // both operands, then 4 bytes of scales per row

template <typename T, bool WIDE>
__global__ __launch_bounds__(64 * kWaves, 2) void k_matmul_small(MatArgs a) {
  constexpr bool kPair = sizeof(T) == 2;
  __shared__ __attribute__((aligned(1024))) char lds[kWaves * kSmallStage];
  static_assert(kSmallStage >= 16 * 64 * 16, "the stage also holds a wave's sums");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, g = lane >> 4, split = blockIdx.y;
  int ti, tj;
  if (!map_tile(a, blockIdx.x, ti, tj)) return;
  const int64_t i0 = (int64_t)ti * kS, j0 = (int64_t)tj * kS;
  const int kb0 = split * a.per, kb1 = min(kb0 + a.per, a.nkb);
  // DMA instruction q: LDS rows 8 q .. +7 (a's 64, then b's), lane l: row
  // l / 8, position l % 8 (chunks permuted as in the larger tiles). Offsets
  // from the tile's first rows: 64 rows of at most 2^24 bytes.
  auto row_a = [&](int r) { return min(i0 + r, a.m - 1) - i0; };
  auto row_b = [&](int r) { return min(j0 + b_row<kPair>(r >> 4, r & 15), a.n - 1) - j0; };
  uint32_t off[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int lr = 8 * (q & 7) + (lane >> 3);
    off[q] = (uint32_t)(q < 8 ? row_a(lr) : row_b(lr)) * (uint32_t)(q < 8 ? a.a.ld : a.b.ld) +
             (uint32_t)(((lane & 7) ^ (lr & 7)) << 4);
  }
  const int64_t as0 = i0 >> a.a.sshift, bs0 = j0 >> a.b.sshift;
  const uint32_t soa = (uint32_t)(((i0 + row_a(lane)) >> a.a.sshift) - as0) * (uint32_t)a.a.sld;
  const uint32_t sob = (uint32_t)(((j0 + row_b(lane)) >> a.b.sshift) - bs0) * (uint32_t)a.b.sld;
  const uint8_t *pa = a.a.codes + i0 * a.a.ld, *pb = a.b.codes + j0 * a.b.ld;
  const uint8_t *sa = a.a.scales + as0 * a.a.sld, *sb = a.b.scales + bs0 * a.b.sld;
  char* st = lds + wave * kSmallStage;
  const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr)lds + wave * kSmallStage;
  auto fetch = [&](int kb, bool first) {
    const int64_t k = (int64_t)kb * kBlock;
#pragma unroll
    for (int q = 0; q < 16; ++q) dma16s((q < 8 ? pa : pb) + k, off[q], base + q * 1024);
    if (first || (kb & 3) == 0) {
      dma4s(sa + (kb & ~3), soa, base + 2 * kSmallOp);
      dma4s(sb + (kb & ~3), sob, base + 2 * kSmallOp + kS * 4);
    }
  };
  const int foff = r16 * kBlock + ((g ^ (r16 & 7)) << 4);
  f32x4 acc[4][4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[q][f] = f32x4{};
  // An eighth of the blocks for each wave, consecutive ones: a fetch of scales
  // serves up to 4 of them (64 rows are 64 cache lines, a quarter of a
  // block's). Waves w and w + 4, which share a SIMD, take neighbouring
  // eighths, so that the SIMDs' shares differ by one block at most.
  const int order = 2 * (wave & 3) + (wave >> 2), nk = max(kb1 - kb0, 0);
  int kb = kb0 + (int)((int64_t)order * nk >> 3);
  const int end = kb0 + (int)((int64_t)(order + 1) * nk >> 3);
  if (kb < end) fetch(kb, true);
  for (; kb < end; ++kb) {
    // this wave's block has landed (memory operations retire in order, and it
    // has no others); the empty asm keeps the reads below the wait
    __builtin_amdgcn_s_waitcnt(0 | (0x7 << 4) | (0xF << 8));  // vmcnt(0)
    asm volatile("" ::: "memory");
    i32x8 fa[4], fb[4];
    int ea[4], eb[4];
    auto frag = [&](const char* p) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(p + foff);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(p + (foff ^ 64));
      return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    const char* ss = st + 2 * kSmallOp;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      fa[f] = frag(st + 16 * f * kBlock);
      fb[f] = frag(st + kSmallOp + 16 * f * kBlock);
      ea[f] = *reinterpret_cast<const int*>(ss + (16 * f + r16) * 4) >> ((kb & 3) * 8);
      eb[f] = *reinterpret_cast<const int*>(ss + (kS + 16 * f + r16) * 4) >> ((kb & 3) * 8);
    }
    if (kb + 1 < end) {
      // the reads have retired before the stage is refilled
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(0xF | (3 << 14) | (0x7 << 4) | (0 << 8));  // lgkmcnt(0)
      asm volatile("" ::: "memory");
      fetch(kb + 1, false);
    }
    mma_block<WIDE, 4, 4>(fb, fa, eb, ea, acc);
  }
  join_waves<T, 4, 4>(a, split, i0, j0, reinterpret_cast<f32x4*>(lds), kSmallStage / 16, acc);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <typename T, bool WIDE>
int launch(const MatArgs& a, const Choice& c, hipStream_t s) {
  const dim3 grid((unsigned)map_grid((int64_t)a.tm * a.tn), (unsigned)a.splits), direct(64 * kWaves);
  if (c.kind == kBig) {
    if (c.em == kB)
      hipLaunchKernelGGL((k_matmul_big<T, WIDE, 4>), grid, dim3(512), 0, s, a);
    else
      hipLaunchKernelGGL((k_matmul_big<T, WIDE, 3>), grid, dim3(512), 0, s, a);
  } else if (c.kind == kTile) {
    hipLaunchKernelGGL((k_matmul_tile<T, WIDE>), grid, dim3(512), 0, s, a);
  } else if (c.kind == kSmall) {
    hipLaunchKernelGGL((k_matmul_small<T, WIDE>), grid, direct, 0, s, a);
  } else {
    hipLaunchKernelGGL((k_matmul_direct<T, WIDE>), grid, direct, 0, s, a);
  }
  if (a.part)
    hipLaunchKernelGGL((k_matmul_join<T>), dim3((unsigned)ceil_div(a.m * (a.pld >> 2), 256)), dim3(256),
                       0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MUONH_EHIP, "fp8 matmul: %s (%d)", hipGetErrorString(e), (int)e);
  return MUONH_OK;
}

int check_operand(const char* name, const muonh_fp8_matrix* x) {
  if (!x) return fail(MUONH_EINVAL, "%s is NULL", name);
  if (bad_dim(x->rows) || bad_dim(x->cols))
    return fail(MUONH_ESHAPE, "%s: shape %lld x %lld out of [0, %d]", name, (long long)x->rows,
                (long long)x->cols, MUONH_MAX_FP8_DIM);
  if (x->block != MUONH_FP8_ROWS && x->block != MUONH_FP8_TILES)
    return fail(MUONH_EINVAL, "%s: block=%d is neither MUONH_FP8_ROWS nor MUONH_FP8_TILES", name, x->block);
  if (x->rows == 0 || x->cols == 0) return MUONH_OK;
  if (!x->codes || !x->scales) return fail(MUONH_EINVAL, "%s: codes and scales must not be NULL", name);
  if (reinterpret_cast<uintptr_t>(x->codes) & 15u || reinterpret_cast<uintptr_t>(x->scales) & 3u)
    return fail(MUONH_EINVAL, "%s: codes must be 16-byte and scales 4-byte aligned", name);
  return MUONH_OK;
}

Operand operand(const muonh_fp8_matrix* x) {
  return Operand{static_cast<const uint8_t*>(x->codes), static_cast<const uint8_t*>(x->scales), x->rows,
                 code_ld(x->cols), scale_ld(x->cols), x->block == MUONH_FP8_TILES ? 7 : 0};
}

}  // namespace
}  // namespace fp8
}  // namespace muonh

extern "C" {

size_t muonh_fp8_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t out_dtype) {
  using namespace muonh::fp8;
  if (bad_dim(m) || bad_dim(n) || bad_dim(k) || m == 0 || n == 0) return 0;
  return choose(m, n, k, !(out_dtype & MUONH_FP8_FAST)).ws_bytes;
}

int muonh_fp8_matmul(const muonh_fp8_matrix* a, const muonh_fp8_matrix* b, void* out,
                     int32_t out_dtype, int64_t out_ld, int32_t accumulate, void* workspace,
                     size_t workspace_bytes, void* stream) {
  using namespace muonh;
  using namespace muonh::fp8;
  if (const int err = check_operand("a", a)) return err;
  if (const int err = check_operand("b", b)) return err;
  if (a->cols != b->cols)
    return fail(MUONH_ESHAPE, "a has %lld columns, b %lld", (long long)a->cols, (long long)b->cols);
  const bool fast = out_dtype == (MUONH_DT_BF16 | MUONH_FP8_FAST);
  if (out_dtype != MUONH_DT_FP32 && out_dtype != MUONH_DT_BF16 && !fast)
    return fail(MUONH_EINVAL, "out_dtype=%d is none of MUONH_DT_FP32, MUONH_DT_BF16, MUONH_DT_BF16|MUONH_FP8_FAST",
                out_dtype);
  const bool bf16 = out_dtype != MUONH_DT_FP32;
  const int64_t m = a->rows, n = b->rows, k = a->cols;
  if (out_ld < n || out_ld > (1LL << 36))
    return fail(MUONH_EINVAL, "out_ld=%lld out of [n=%lld, 2^36]", (long long)out_ld, (long long)n);
  if (m == 0 || n == 0) return MUONH_OK;
  if (!out) return fail(MUONH_EINVAL, "out is NULL");
  const int esize = bf16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(out) & (uintptr_t)(esize - 1))
    return fail(MUONH_EINVAL, "out is not aligned to its type");
  if (ceil_div(m, kT) * ceil_div(n, kT) > kMaxTiles)
    return fail(MUONH_ESHAPE, "2^21 output tiles of 128 x 128 or more");
  const Choice c = choose(m, n, k, !fast);
  if (c.ws_bytes) {
    if (!workspace) return fail(MUONH_EWORKSPACE, "workspace is NULL, the product needs %zu bytes", c.ws_bytes);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
      return fail(MUONH_EWORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < c.ws_bytes)
      return fail(MUONH_EWORKSPACE, "workspace has %zu bytes, the product needs %zu", workspace_bytes, c.ws_bytes);
  }
  const Span written[2] = {span("out", out, ((m - 1) * out_ld + n) * esize),
                           span("workspace", c.ws_bytes ? workspace : nullptr, (int64_t)c.ws_bytes)};
  const Span read[4] = {span("a's codes", a->codes, m * code_ld(k)),
                        span("a's scales", a->scales, scale_rows(m, a->block) * scale_ld(k)),
                        span("b's codes", b->codes, n * code_ld(k)),
                        span("b's scales", b->scales, scale_rows(n, b->block) * scale_ld(k))};
  if (overlap(written[0], written[1])) return fail(MUONH_EALIAS, "out overlaps the workspace");
  for (const Span& w : written)
    for (const Span& r : read)
      if (overlap(w, r)) return fail(MUONH_EALIAS, "%s overlaps %s", w.name, r.name);

  MatArgs x{};
  x.a = operand(a);
  x.b = operand(b);
  x.m = m;
  x.n = n;
  x.nkb = (int)ceil_div(k, kBlock);
  x.out = out;
  x.ldo = out_ld;
  x.accumulate = accumulate != 0;
  x.odd = bf16 && ((reinterpret_cast<uintptr_t>(out) & 2) != 0 || (out_ld & 1) != 0);
  x.splits = c.splits;
  x.per = c.per;
  x.pld = ceil_div(n, 4) * 4;
  x.part = c.ws_bytes ? static_cast<float*>(workspace) : nullptr;
  x.tm = (int)ceil_div(m, c.em);
  x.tn = (int)ceil_div(n, c.en);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (fast) return launch<__bf16, false>(x, c, s);
  return bf16 ? launch<__bf16, true>(x, c, s) : launch<float, true>(x, c, s);
}

}  // extern "C"
