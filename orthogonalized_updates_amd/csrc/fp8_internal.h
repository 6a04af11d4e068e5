// Shared by the block-scaled 8-bit sources (fp8_quantize.hip, fp8_matmul.hip).
// Not part of the ABI; formats as in include/muonh.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cstdarg>
#include <cstdio>

#include "../../include/muonh.h"
#include "muonh_internal.h"

namespace muonh {
namespace fp8 {

constexpr int kBlock = 128;  // entries per scale along a row

__host__ __device__ inline int64_t ceil_div(int64_t v, int64_t m) { return (v + m - 1) / m; }
__host__ __device__ inline int64_t code_ld(int64_t cols) { return ceil_div(cols, kBlock) * kBlock; }
__host__ __device__ inline int64_t scale_ld(int64_t cols) {
  return ceil_div(ceil_div(cols, kBlock), 4) * 4;
}
inline int64_t scale_rows(int64_t rows, int block) {
  return block == MUONH_FP8_TILES ? ceil_div(rows, kBlock) : rows;
}

inline int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_error(code, buf);
}

inline bool bad_dim(int64_t v) { return v < 0 || v > MUONH_MAX_FP8_DIM; }

// 128 x 128 tiles of a matrix, one workgroup each: a launch has fewer than 2^32
// threads.
constexpr int64_t kMaxBlocks = (1 << 24) - 8;
bool tiles_fit(int64_t rows, int64_t cols);

// codes, scales, codes_t, scales_t (MUONH_FP8_ROWS; codes and scales, not codes_t and scales_t, may be
// nullptr) of the matrix (src[r][c] * rstd[r]) * weight[c]. Arguments are the
// caller's to check.
int quantize_normed(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t src_ld, const float* rstd,
                    const float* weight, void* codes, void* scales, void* codes_t, void* scales_t, hipStream_t s);

// A byte range of device memory, for the overlap checks of a call.
struct Span {
  const char* name;
  uintptr_t lo, hi;
};
inline Span span(const char* name, const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Span{name, lo, p ? lo + (uintptr_t)bytes : lo};
}
// Empty ranges overlap nothing.
inline bool overlap(const Span& a, const Span& b) {
  return a.lo < a.hi && b.lo < b.hi && a.lo < b.hi && b.lo < a.hi;
}

}  // namespace fp8
}  // namespace muonh
