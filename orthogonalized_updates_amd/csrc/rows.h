// Rows of fp32 or bf16 entries: what the operators that go through them in
// vectors of 8 share (rms_norm.hip, embedding.hip, the quantizers), device side and argument checks.
#pragma once

#include "fp8_internal.h"

namespace muonh {
namespace rows {

using fp8::fail;
using fp8::Span;
using fp8::span;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// at any multiple of the entry's size (gfx950 takes vector accesses at any address)
typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// ---- 8 consecutive entries -----------------------------------------------------
// As loaded; n: how many of them there are (below 8 only in a row's last vector).
template <typename T>
struct Raw;
template <>
struct Raw<__bf16> {
  u32x4 v;
  __device__ __forceinline__ void load(const __bf16* p) { v = *reinterpret_cast<const u32x4_a2*>(p); }
  __device__ __forceinline__ void load(const __bf16* p, int n) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
    v = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) v[j >> 1] |= (uint32_t)q[j] << (16 * (j & 1));
  }
  __device__ __forceinline__ float at(int j) const {
    return __uint_as_float(j & 1 ? v[j >> 1] & 0xffff0000u : v[j >> 1] << 16);
  }
};
template <>
struct Raw<float> {
  f32x4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = *reinterpret_cast<const f32x4_a4*>(p);
    v[1] = *reinterpret_cast<const f32x4_a4*>(p + 4);
  }
  __device__ __forceinline__ void load(const float* p, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j >> 2][j & 3] = j < n ? p[j] : 0.f;
  }
  __device__ __forceinline__ float at(int j) const { return v[j >> 2][j & 3]; }
};

// Stores the first n of 8 values, each rounded once.
__device__ __forceinline__ void store8(__bf16* p, const float (&v)[8], int n) {
  const bf16x8 b = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3],
                    (__bf16)v[4], (__bf16)v[5], (__bf16)v[6], (__bf16)v[7]};
  if (n >= 8) {
    *reinterpret_cast<u32x4_a2*>(p) = __builtin_bit_cast(u32x4, b);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = b[j];
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8], int n) {
  if (n >= 8) {
    *reinterpret_cast<f32x4_a4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<f32x4_a4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = v[j];
  }
}

// ---- host side ----------------------------------------------------------------
inline bool bad_dtype(int32_t d) { return d != MUONH_DT_FP32 && d != MUONH_DT_BF16; }
inline bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }
inline int size_of(int32_t d) { return d == MUONH_DT_BF16 ? 2 : 4; }

// A 2-d argument: rows of `cols` entries, ld apart.
struct Mat {
  const char* name;
  const void* p;
  int32_t dtype;
  int64_t ld;
};
inline int check_mat(const Mat& m, int64_t cols) {
  if (!m.p) return fail(MUONH_EINVAL, "%s is NULL", m.name);
  if (misaligned(m.p, (uintptr_t)size_of(m.dtype)))
    return fail(MUONH_EINVAL, "%s is not aligned to its type", m.name);
  if (m.ld < cols || m.ld > (1LL << 36))
    return fail(MUONH_EINVAL, "%s's row pitch %lld out of [cols=%lld, 2^36]", m.name, (long long)m.ld, (long long)cols);
  return MUONH_OK;
}
inline Span span_of(const Mat& m, int64_t rows, int64_t cols) {
  return span(m.name, m.p, m.p ? ((rows - 1) * m.ld + cols) * size_of(m.dtype) : 0);
}
// Whether two matrices of `rows` x `cols` entries have memory in common. Rows of one pitch may lie
// between each other's, as columns of a wider matrix.
inline bool meet(const Mat& a, const Mat& b, int64_t rows, int64_t cols) {
  if (!fp8::overlap(span_of(a, rows, cols), span_of(b, rows, cols))) return false;
  const int64_t pitch = a.ld * size_of(a.dtype);
  if (rows < 2 || pitch != b.ld * size_of(b.dtype)) return true;
  const int64_t apart = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % pitch;
  const int64_t d = apart < 0 ? apart + pitch : apart;  // b's first column after a's
  return d < cols * size_of(a.dtype) || d + cols * size_of(b.dtype) > pitch;
}
inline bool same(const Mat& a, const Mat& b) { return a.p == b.p && a.ld == b.ld && a.dtype == b.dtype; }

inline int launched(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MUONH_EHIP, "%s: %s (%d)", what, hipGetErrorString(e), (int)e);
  return MUONH_OK;
}

}  // namespace rows
}  // namespace muonh
