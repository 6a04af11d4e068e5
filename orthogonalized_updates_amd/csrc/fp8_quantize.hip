// Quantization to block-scaled e4m3 on gfx950 (formats: include/muonh.h; the
// report page, part 6/7, section 4.3 "Cost Estimation", names blockwise FP8
// linear layers, without a rounding or a scale type).
//
// One workgroup takes one 128 x 128 tile of the source, which holds whole
// blocks of every kind: 128 row groups, 128 column groups (the transposed
// form's row groups) or one tile. It reads the tile once into registers (16 x
// 16 threads, each an 8 x 8 patch), takes the maxima by lane exchanges and
// LDS, and writes one or both forms: 4 (fp32) or 2 (bf16) bytes read and 1 or
// 2 written per entry, HBM-bound.
//
// A scale is a power of two, so the conversion instruction, which divides by
// it, rounds once (to nearest, ties to even).
#include <type_traits>

#include "fp8_internal.h"

namespace muonh {
namespace fp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroups = 16;
// Blocks of one launch: a launch has fewer than 2^32 threads.
constexpr int64_t kMaxBlocks = (1 << 24) - 8;

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// 4 values over a scale 2^e (exact) to 4 codes, the first in the low byte.
typedef short s16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s) {
  s16x2 v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(s16x2{0, 0}, a, b, s, false);
  v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, c, d, s, true);
  return __builtin_bit_cast(uint32_t, v);
}

// Magnitudes order like their bits, compared as integers: a floating-point
// maximum answers a signaling NaN with a NaN and forgets what came before. A
// scale's exponent depends on the upper 16 bits of the maximum, rounded up, so
// maxima are handled in pairs of 16 bits, two in one packed instruction, and
// bf16 entries stay in pairs throughout.
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pmax(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(
      uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x05040100);
}
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302);
}
// Two magnitudes with those that are not finite as zero.
__device__ __forceinline__ uint32_t finite2(uint32_t m) {
  return ((m & 0xffffu) < 0x7f80u ? m & 0xffffu : 0u) | (m < 0x7f800000u ? m & 0xffff0000u : 0u);
}
// Upper halves of two fp32 magnitudes, rounded up.
__device__ __forceinline__ uint32_t upper2(uint32_t a, uint32_t b) {
  return high_halves(a + 0xffffu, b + 0xffffu);
}
// Maxima over the 16 lanes of a DPP row, in all of them.
template <int CTRL>
__device__ __forceinline__ uint32_t pmax_dpp(uint32_t v) {
  return pmax(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t pmax_row16(uint32_t v) {
  v = pmax_dpp<0xB1>(v);   // quad [1,0,3,2]
  v = pmax_dpp<0x4E>(v);   // quad [2,3,0,1]
  v = pmax_dpp<0x141>(v);  // mirrored halves: the other quad of 8
  return pmax_dpp<0x140>(v);  // mirrored row: the other 8
}
// Maxima over finite entries -> scale bytes e + 127, e >= -126: with a = 1.f *
// 2^E and 448 = 1.75 * 2^8, e = E - 8 where 1.f <= 1.75 (0x60 of the 7 bits),
// else E - 7.
__device__ __forceinline__ uint32_t scale_bytes2(uint32_t m) {
  const u16x2 e = (__builtin_bit_cast(u16x2, m) + u16x2{0x1f, 0x1f}) >> u16x2{7, 7};
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(e, u16x2{9, 9}) - u16x2{8, 8});
}
// The scale 2^e of a pair's byte in [1, 247], a normal number.
__device__ __forceinline__ float scale_lo(uint32_t b) { return __uint_as_float(b << 23); }
__device__ __forceinline__ float scale_hi(uint32_t b) { return __uint_as_float((b << 7) & 0x7f800000u); }
// The bytes of 8 scales from 4 pairs.
__device__ __forceinline__ uint2 bytes8(const uint32_t (&b)[4]) {
  return make_uint2(__builtin_amdgcn_perm(b[1], b[0], 0x06040200), __builtin_amdgcn_perm(b[3], b[2], 0x06040200));
}
// 8 entries (4 pairs) over a scale to 8 codes.
__device__ __forceinline__ uint2 codes8(uint32_t a, uint32_t b, uint32_t c, uint32_t d, float s) {
  auto two = [&](s16x2 v, uint32_t x, auto hi) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(v, __builtin_bit_cast(bf16x2, x), s, decltype(hi)::value);
  };
  const s16x2 x = two(two(s16x2{0, 0}, a, std::false_type{}), b, std::true_type{});
  const s16x2 y = two(two(s16x2{0, 0}, c, std::false_type{}), d, std::true_type{});
  return make_uint2(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y));
}

struct Group {
  int64_t rows, cols, src_ld;
  uint32_t first, tiles_c;  // first matrix (grouped launches); tiles per tile row
  uint32_t tiles, begin;    // tiles per matrix; first block of the group
};
struct Args {
  Group g[kMaxGroups];
  int ngroups;
  uint32_t tiles;  // of all groups
  // one matrix (ptrs == 0), or device arrays of pointers indexed by matrix
  int ptrs;
  const void* src;
  void *codes, *scales, *codes_t, *scales_t;
};

// 8 consecutive entries from i, at any multiple of the entry's size (gfx950
// takes vector accesses at any address).
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// A thread's 8 x 8 entries: zeros past the matrix.
__device__ __forceinline__ void load_patch(const float* p, int64_t ld, int64_t r0, int64_t c0, int64_t rows,
                                           int64_t cols, float (&v)[8][8]) {
  if (c0 + 8 <= cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // rows past the end reload the last one, so that no load waits in a branch
      const int64_t r = r0 + i < rows ? r0 + i : rows - 1;
      const f32x4_a4* q = reinterpret_cast<const f32x4_a4*>(p + r * ld + c0);
      const f32x4_a4 a = q[0], b = q[1];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[i][k] = a[k];
        v[i][4 + k] = b[k];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r0 + i >= rows)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = r0 + i < rows && c0 + j < cols ? p[(r0 + i) * ld + c0 + j] : 0.f;
  }
}
__device__ __forceinline__ void load_patch(const uint16_t* p, int64_t ld, int64_t r0, int64_t c0, int64_t rows,
                                           int64_t cols, u32x4_a2 (&v)[8]) {
  if (c0 + 8 <= cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + i < rows ? r0 + i : rows - 1;
      v[i] = *reinterpret_cast<const u32x4_a2*>(p + r * ld + c0);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r0 + i >= rows) v[i] = u32x4_a2{0, 0, 0, 0};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        auto at = [&](int64_t c) { return r0 + i < rows && c < cols ? (uint32_t)p[(r0 + i) * ld + c] : 0u; };
        v[i][j] = at(c0 + 2 * j) | at(c0 + 2 * j + 1) << 16;
      }
  }
}

// The scale byte of block column kb of one scale row; the block of the last
// column also writes the row's zero padding.
__device__ __forceinline__ void put_scale(uint8_t* s, int64_t row, int64_t kb, int64_t cols,
                                          uint32_t byte) {
  const int64_t ld = scale_ld(cols), nb = ceil_div(cols, kBlock);
  uint8_t* p = s + row * ld;
  p[kb] = (uint8_t)byte;
  if (kb == nb - 1)
    for (int64_t j = nb; j < ld; ++j) p[j] = 0;
}

// Thread (ty, tx) = (tid / 16, tid % 16) holds rows 8 ty .. +7, columns
// 8 tx .. +7 of the tile. PLAIN, TRANS: the forms written; TILES: one scale.
//
// Blocks are dealt to the 8 XCDs in turn; each XCD takes a contiguous eighth
// of the tiles, so that the scale bytes of neighbouring tiles, which share
// cache lines in both forms, meet in one L2. XCD x begins x eighths into its
// part: from the beginning, rows of a power of two bytes put all XCDs on the
// same memory channels (4096 x 8192 bf16 in both forms 39.1 -> 31.8 us, 8192 x
// 2048 fp32 26.7 -> 25.1, other sizes +-1 %).
//
// Measured with inputs from memory, a copy of as many bytes in parentheses:
// bf16 in both forms 8192 x 2048 17.7 us (14.6), x 4096 33.1 (27.5), x 14336
// 103 (91).
template <bool BF, bool TILES, bool PLAIN, bool TRANS>
__global__ __launch_bounds__(kThreads, 4) void k_quantize(Args a) {
  __shared__ __attribute__((aligned(16))) uint32_t red[4][kBlock / 2];  // maxima by wave
  __shared__ __attribute__((aligned(8))) uint8_t byte_of[2][kBlock];  // scale bytes of rows, columns
  __shared__ __attribute__((aligned(16))) uint8_t stage[TRANS ? kBlock * kBlock : 16];  // transposed codes
  const uint32_t x = blockIdx.x & 7;
  const uint32_t lo = (uint32_t)(((uint64_t)x * a.tiles) >> 3);
  const uint32_t count = (uint32_t)(((uint64_t)(x + 1) * a.tiles) >> 3) - lo;
  if ((blockIdx.x >> 3) >= count) return;
  uint32_t index = (blockIdx.x >> 3) + ((x * count) >> 3);
  if (index >= count) index -= count;
  index += lo;
  int gi = 0;
  for (int i = 1; i < a.ngroups; ++i)
    if (index >= a.g[i].begin) gi = i;
  const Group& g = a.g[gi];
  const uint32_t local = index - g.begin;
  const uint32_t m = local / g.tiles, t = local - m * g.tiles;
  const int64_t tr = t / g.tiles_c, tc = t - (uint32_t)tr * g.tiles_c;
  const int64_t mat = g.first + m;
  const void* src = a.ptrs ? static_cast<const void* const*>(a.src)[mat] : a.src;
  auto pick = [&](void* p) {
    return static_cast<uint8_t*>(a.ptrs ? static_cast<void* const*>(p)[mat] : p);
  };
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int tx = tid & 15, ty = tid >> 4;
  const int64_t r0 = tr * kBlock + 8 * ty, c0 = tc * kBlock + 8 * tx;
  const int64_t rows = g.rows, cols = g.cols;

  // the entries (bf16: pairs of them), and the maxima of magnitudes of rows
  // 2k, 2k + 1 and of columns 2k, 2k + 1
  constexpr bool kRows = PLAIN && !TILES, kCols = TRANS || TILES;
  float v[BF ? 1 : 8][8];
  u32x4_a2 w[BF ? 8 : 1];
  uint32_t rmax[4], cmax[4];
  if constexpr (BF) {
    load_patch(static_cast<const uint16_t*>(src), g.src_ld, r0, c0, rows, cols, w);
    auto maxima = [&](auto clean) {
      uint32_t r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t m = w[i][d] & 0x7fff7fffu;
          if constexpr (decltype(clean)::value) m = finite2(m);
          r[i] = d ? pmax(r[i], m) : m;
          cmax[d] = i ? pmax(cmax[d], m) : m;
        }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        rmax[k] = pmax(low_halves(r[2 * k], r[2 * k + 1]), high_halves(r[2 * k], r[2 * k + 1]));
    };
    maxima(std::false_type{});
    const auto& any = kCols ? cmax : rmax;
    const uint32_t all = pmax(pmax(any[0], any[1]), pmax(any[2], any[3]));
    if (finite2(all) != all) maxima(std::true_type{});
  } else {
    load_patch(static_cast<const float*>(src), g.src_ld, r0, c0, rows, cols, v);
    uint32_t r[8], c[8];
    auto maxima = [&](auto clean) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          uint32_t m = __float_as_uint(v[i][j]);
          // computed anew in the rare second pass, not kept for it in registers
          if constexpr (decltype(clean)::value) asm("" : "+v"(m));
          m &= 0x7fffffffu;
          if constexpr (decltype(clean)::value) m = m < 0x7f800000u ? m : 0u;
          r[i] = j ? umax(r[i], m) : m;
          c[j] = i ? umax(c[j], m) : m;
        }
    };
    maxima(std::false_type{});
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) all = umax(all, kCols ? c[i] : r[i]);
    if (all >= 0x7f800000u) maxima(std::true_type{});
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      rmax[k] = upper2(r[2 * k], r[2 * k + 1]);
      cmax[k] = upper2(c[2 * k], c[2 * k + 1]);
    }
  }

  float scale = 1.f;  // of the tile
  if constexpr (TILES) {
    uint32_t mx = pmax_row16(pmax(pmax(cmax[0], cmax[1]), pmax(cmax[2], cmax[3])));
    mx = pmax(mx, (uint32_t)__shfl_xor((int)mx, 16, 64));
    mx = pmax(mx, (uint32_t)__shfl_xor((int)mx, 32, 64));
    if (lane == 0) red[0][wave] = mx;
    __syncthreads();
    mx = pmax(pmax(red[0][0], red[0][1]), pmax(red[0][2], red[0][3]));
    const uint32_t byte = scale_bytes2(pmax(mx, mx >> 16)) & 0xffffu;
    scale = scale_lo(byte);
    if (tid == 0) {
      if (PLAIN) put_scale(pick(a.scales), tr, tc, cols, byte);
      if (TRANS) put_scale(pick(a.scales_t), tc, tr, rows, byte);
    }
  }

  if constexpr (PLAIN) {
    uint8_t* codes = pick(a.codes);
    const int64_t ld = code_ld(cols);
    uint32_t pair[4];  // scale bytes of rows 2k, 2k + 1
    if constexpr (kRows) {
      // the 16 threads of a row are the lanes of a DPP row
#pragma unroll
      for (int k = 0; k < 4; ++k) pair[k] = scale_bytes2(pmax_row16(rmax[k]));
      if (tx == 0) *reinterpret_cast<uint2*>(&byte_of[0][8 * ty]) = bytes8(pair);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = TILES ? scale : i & 1 ? scale_hi(pair[i >> 1]) : scale_lo(pair[i >> 1]);
      uint2 q;
      if constexpr (BF) {
        q = codes8(w[i][0], w[i][1], w[i][2], w[i][3], s);
      } else {
        q.x = codes4(v[i][0], v[i][1], v[i][2], v[i][3], s);
        q.y = codes4(v[i][4], v[i][5], v[i][6], v[i][7], s);
      }
      if (r0 + i < rows) *reinterpret_cast<uint2*>(codes + (r0 + i) * ld + c0) = q;
    }
  }

  if constexpr (TRANS) {
    float s[8];
    if constexpr (!TILES) {
      // the wave's 4 thread rows: a swap of lane halves brings both halves'
      // maxima of one pair of columns together, of pair d in the lower lanes
      // and of d + 2 in the upper ones; then the same with rows of 16 lanes
      uint32_t h[2];
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const auto p = __builtin_amdgcn_permlane32_swap(cmax[d], cmax[d + 2], false, false);
        h[d] = pmax(p[0], p[1]);
      }
      const auto p = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
      // lane 16 g + tx: pair g of the 4
      red[wave][4 * tx + (lane >> 4)] = pmax(p[0], p[1]);
      __syncthreads();
      uint32_t pair[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int c = 4 * tx + d;
        pair[d] = scale_bytes2(pmax(pmax(red[0][c], red[1][c]), pmax(red[2][c], red[3][c])));
        s[2 * d] = scale_lo(pair[d]);
        s[2 * d + 1] = scale_hi(pair[d]);
      }
      if (ty == 0) *reinterpret_cast<uint2*>(&byte_of[1][8 * tx]) = bytes8(pair);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = scale;
    }
    // Row c of the staged tile: 16 pieces of 8 codes (piece = thread row),
    // piece p at position p ^ (c / 8), so that the 16 thread columns of a
    // store fall on different banks.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint2 q;
      if constexpr (BF) {
        auto rows2 = [&](int i) {
          return j & 1 ? high_halves(w[i][j >> 1], w[i + 1][j >> 1]) : low_halves(w[i][j >> 1], w[i + 1][j >> 1]);
        };
        q = codes8(rows2(0), rows2(2), rows2(4), rows2(6), s[j]);
      } else {
        q.x = codes4(v[0][j], v[1][j], v[2][j], v[3][j], s[j]);
        q.y = codes4(v[4][j], v[5][j], v[6][j], v[7][j], s[j]);
      }
      *reinterpret_cast<uint2*>(stage + (8 * tx + j) * kBlock + ((ty ^ tx) << 3)) = q;
    }
  }
  if (TRANS || !TILES) __syncthreads();
  if (!TILES) {
    if (PLAIN && tid < kBlock && tr * kBlock + tid < rows)
      put_scale(pick(a.scales), tr * kBlock + tid, tc, cols, byte_of[0][tid]);
    const int c = tid - (kThreads - kBlock);
    if (TRANS && c >= 0 && tc * kBlock + c < cols)
      put_scale(pick(a.scales_t), tc * kBlock + c, tr, rows, byte_of[1][c]);
  }
  if (TRANS) {
    uint8_t* out = pick(a.codes_t);
    const int64_t ld = code_ld(rows);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = (tid >> 3) + 32 * k, u = tid & 7;  // 16 bytes: pieces 2u, 2u + 1
      const uint2 lo = *reinterpret_cast<const uint2*>(stage + c * kBlock + (((2 * u) ^ (c >> 3)) << 3));
      const uint2 hi = *reinterpret_cast<const uint2*>(stage + c * kBlock + (((2 * u + 1) ^ (c >> 3)) << 3));
      if (tc * kBlock + c < cols)
        *reinterpret_cast<uint4*>(out + (tc * kBlock + c) * ld + tr * kBlock + 16 * u) =
            make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

template <bool BF, bool TILES>
void launch_forms(const Args& a, bool plain, bool trans, hipStream_t s) {
  const dim3 grid((unsigned)(8 * ceil_div(a.tiles, 8))), thr(kThreads);
  if (plain && trans)
    hipLaunchKernelGGL((k_quantize<BF, TILES, true, true>), grid, thr, 0, s, a);
  else if (plain)
    hipLaunchKernelGGL((k_quantize<BF, TILES, true, false>), grid, thr, 0, s, a);
  else
    hipLaunchKernelGGL((k_quantize<BF, TILES, false, true>), grid, thr, 0, s, a);
}

int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MUONH_EHIP, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
  return MUONH_OK;
}

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

}  // namespace
}  // namespace fp8
}  // namespace muonh

extern "C" {

int64_t muonh_fp8_ld(int64_t cols) {
  return muonh::fp8::bad_dim(cols) ? 0 : muonh::fp8::code_ld(cols);
}

int64_t muonh_fp8_scale_ld(int64_t cols) {
  return muonh::fp8::bad_dim(cols) ? 0 : muonh::fp8::scale_ld(cols);
}

int64_t muonh_fp8_scale_rows(int64_t rows, int32_t block) {
  if (muonh::fp8::bad_dim(rows) || (block != MUONH_FP8_ROWS && block != MUONH_FP8_TILES)) return 0;
  return muonh::fp8::scale_rows(rows, block);
}

int muonh_fp8_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t src_ld,
                       int32_t block, void* codes, void* scales, void* codes_t, void* scales_t,
                       void* stream) {
  using namespace muonh;
  using namespace muonh::fp8;
  if (dtype != MUONH_DT_FP32 && dtype != MUONH_DT_BF16)
    return fail(MUONH_EINVAL, "dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", dtype);
  if (block != MUONH_FP8_ROWS && block != MUONH_FP8_TILES)
    return fail(MUONH_EINVAL, "block=%d is neither MUONH_FP8_ROWS nor MUONH_FP8_TILES", block);
  if (bad_dim(rows) || bad_dim(cols))
    return fail(MUONH_ESHAPE, "shape %lld x %lld out of [0, %d]", (long long)rows, (long long)cols,
                MUONH_MAX_FP8_DIM);
  if (src_ld < cols || src_ld > (1LL << 36))
    return fail(MUONH_EINVAL, "src_ld=%lld out of [cols=%lld, 2^36]", (long long)src_ld, (long long)cols);
  if (rows == 0 || cols == 0) return MUONH_OK;
  if (!src) return fail(MUONH_EINVAL, "src is NULL");
  if (!codes != !scales || !codes_t != !scales_t)
    return fail(MUONH_EINVAL, "codes and scales (codes_t and scales_t) go together");
  if (!codes && !codes_t) return fail(MUONH_EINVAL, "no output given");
  const int esize = dtype == MUONH_DT_BF16 ? 2 : 4;
  if (misaligned(src, esize)) return fail(MUONH_EINVAL, "src is not aligned to its type");
  if (misaligned(codes, 16) || misaligned(codes_t, 16) || misaligned(scales, 4) || misaligned(scales_t, 4))
    return fail(MUONH_EINVAL, "codes must be 16-byte and scales 4-byte aligned");
  const int64_t tr = ceil_div(rows, kBlock), tc = ceil_div(cols, kBlock);
  if (tr * tc > kMaxBlocks) return fail(MUONH_ESHAPE, "2^24 tiles of 128 x 128 or more");
  const Span spans[5] = {
      span("src", src, ((rows - 1) * src_ld + cols) * esize),
      span("codes", codes, rows * code_ld(cols)),
      span("scales", scales, scale_rows(rows, block) * scale_ld(cols)),
      span("codes_t", codes_t, cols * code_ld(rows)),
      span("scales_t", scales_t, scale_rows(cols, block) * scale_ld(rows))};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (overlap(spans[i], spans[j]))
        return fail(MUONH_EALIAS, "%s overlaps %s", spans[j].name, spans[i].name);

  Args a{};
  a.ngroups = 1;
  a.g[0] = Group{rows, cols, src_ld, 0, (uint32_t)tc, (uint32_t)(tr * tc), 0};
  a.tiles = (uint32_t)(tr * tc);
  a.src = src;
  a.codes = codes;
  a.scales = scales;
  a.codes_t = codes_t;
  a.scales_t = scales_t;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const bool plain = codes != nullptr, trans = codes_t != nullptr;
  if (dtype == MUONH_DT_BF16) {
    if (block == MUONH_FP8_TILES) launch_forms<true, true>(a, plain, trans, s);
    else launch_forms<true, false>(a, plain, trans, s);
  } else {
    if (block == MUONH_FP8_TILES) launch_forms<false, true>(a, plain, trans, s);
    else launch_forms<false, false>(a, plain, trans, s);
  }
  return launched("fp8 quantize");
}

int muonh_fp8_weights(const muonh_plan* plan, const float* const* W, void* const* codes,
                      void* const* scales, void* const* codes_t, void* const* scales_t,
                      void* stream) {
  using namespace muonh;
  using namespace muonh::fp8;
  if (!plan) return fail(MUONH_EINVAL, "plan is NULL");
  if (!W || !codes || !scales) return fail(MUONH_EINVAL, "W, codes and scales must be device arrays");
  if (!codes_t != !scales_t) return fail(MUONH_EINVAL, "codes_t and scales_t go together");
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int ng = plan_num_groups(plan);
  // both passes walk the same launches: the first one only counts blocks
  for (int pass = 0; pass < 2; ++pass)
    for (int g0 = 0; g0 < ng; g0 += kMaxGroups) {
      Args a{};
      a.ptrs = 1;
      a.src = W;
      a.codes = const_cast<void**>(codes);
      a.scales = const_cast<void**>(scales);
      a.codes_t = const_cast<void**>(codes_t);
      a.scales_t = const_cast<void**>(scales_t);
      int64_t blocks = 0;
      for (int i = g0; i < ng && i < g0 + kMaxGroups; ++i) {
        const PlanGroup p = plan_group(plan, i);
        const int64_t tr = ceil_div(p.rows, kBlock), tc = ceil_div(p.cols, kBlock);
        a.g[a.ngroups++] = Group{p.rows, p.cols, p.cols, (uint32_t)p.first, (uint32_t)tc,
                                 (uint32_t)(tr * tc), (uint32_t)blocks};
        blocks += tr * tc * p.count;
        if (blocks > kMaxBlocks) return fail(MUONH_ESHAPE, "2^24 tiles of 128 x 128 or more in one launch");
      }
      if (pass == 0) continue;
      a.tiles = (uint32_t)blocks;
      launch_forms<false, true>(a, true, codes_t != nullptr, s);
      if (const int err = launched("fp8 weights")) return err;
    }
  return MUONH_OK;
}

}  // extern "C"
