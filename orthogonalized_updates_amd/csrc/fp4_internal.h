// Shared by the microscaled 4-bit sources (fp4_quantize.hip, fp4_matmul.hip). Not
// part of the ABI; formats as in include/muonh.h.
#pragma once

#include "fp8_internal.h"

namespace muonh {
namespace fp4 {

using fp8::bad_dim;
using fp8::ceil_div;
using fp8::fail;
using fp8::overlap;
using fp8::Span;
using fp8::span;

constexpr int kGroup = 32;   // entries per scale
constexpr int kStep = 256;   // entries that a product takes at a time: 128 bytes of codes, 8 of scales

__host__ __device__ inline int64_t code_ld(int64_t cols) { return ceil_div(cols, kStep) * (kStep / 2); }
__host__ __device__ inline int64_t scale_ld(int64_t cols) { return ceil_div(cols, kStep) * (kStep / kGroup); }

inline int check_matrix(const char* name, const muonh_fp4_matrix* x) {
  if (!x) return fail(MUONH_EINVAL, "%s is NULL", name);
  if (bad_dim(x->rows) || bad_dim(x->cols))
    return fail(MUONH_ESHAPE, "%s: shape %lld x %lld out of [0, %d]", name, (long long)x->rows, (long long)x->cols,
                MUONH_MAX_FP8_DIM);
  if (x->rows == 0 || x->cols == 0) return MUONH_OK;
  if (!x->codes || !x->scales) return fail(MUONH_EINVAL, "%s: codes and scales must not be NULL", name);
  if (reinterpret_cast<uintptr_t>(x->codes) & 15u || reinterpret_cast<uintptr_t>(x->scales) & 7u)
    return fail(MUONH_EINVAL, "%s: codes must be 16-byte and scales 8-byte aligned", name);
  return MUONH_OK;
}

}  // namespace fp4
}  // namespace muonh
