// Device code that the producers of block-scaled matrices share
// (fp8_quantize.hip, rms_norm.hip, fp4_quantize.hip): maxima of magnitudes, patches of a tile, and
// of the e4m3 format (include/muonh.h) scale bytes and conversions.
#pragma once

#include <type_traits>

#include "rows.h"

namespace muonh {
namespace fp8 {

using rows::f32x4_a4;
using rows::u32x4_a2;

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

}  // namespace fp8
}  // namespace muonh
