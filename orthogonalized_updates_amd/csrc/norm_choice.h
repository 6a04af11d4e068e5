// Which lanes share a row of the RMS norm (rms_norm.hip), and how many workgroups a call has: host
// code only.
#pragma once

#include <algorithm>

#include "fp8_internal.h"

namespace muonh {
namespace norm {

using fp8::ceil_div;

// `lanes` lanes hold a row in registers, `vecs` vectors of 8 entries each; 0: rows of any length.
struct Form {
  int lanes, vecs;
};
// Rows that a workgroup takes at a time.
inline int rows_at_once(const Form& f) { return f.lanes > 0 && f.lanes < 256 ? 256 / f.lanes : 1; }

// A wave to a row where that holds it, four for the longest such rows and where rows are
// few. bf16 with a residual into 8-bit rows of 2048, a wave and four: 1 row 4.1, 2.3 us; 256 rows 5.2, 3.4;
// 4096 rows 13.5, 12.2; 8192 rows 22.3, 20.6; 16384 rows 41.7, 42.7. 8192 rows of 600 fp32 entries: 8.7, 10.5.
// 131072 rows of 128 (16 lanes each) 13.0, at 5.2 TB/s.
inline Form forward_form(int64_t rows, int64_t cols) {
  const int64_t vecs = ceil_div(cols, 8);
  if (vecs <= 16) return {16, 1};
  if (vecs <= 256 && (rows <= 256 || vecs > 192)) return {256, 1};
  if (vecs <= 192) return {64, (int)ceil_div(vecs, 64)};
  if (vecs <= 512) return {256, 2};
  if (vecs <= 1024) return {256, 4};
  if (vecs <= 2048) return {1024, 2};
  if (vecs <= 4096) return {1024, 4};  // up to 45 registers more than there are
  return {0, 0};
}
// Of up to 1024 threads: below 2^32. Rows past these go to the same workgroups again.
constexpr int kMaxGrid = 1 << 20;
inline int64_t forward_groups(int64_t rows, const Form& f) {
  return std::min<int64_t>(ceil_div(rows, rows_at_once(f)), kMaxGrid);
}

constexpr int kBackCols = 16384;  // longer rows go through k_norm_dots
inline Form backward_form(int64_t cols) {
  const int64_t vecs = ceil_div(cols, 8);
  if (cols > kBackCols) return {0, 0};
  if (vecs <= 16) return {16, 1};
  if (vecs <= 256) return {64, (int)ceil_div(vecs, 64)};
  if (vecs <= 512) return {256, 2};
  if (vecs <= 1024) return {256, 4};
  return {1024, 2};
}
// Workgroups, and so partial sums of dw: as many as a chip holds, or fewer where joining the sums
// costs more than that gains (main kernel and join, us: 131072 x 128 512 groups 22.2 + 4.7, 2048 18.5 + 4.6; 8192 x
// 2048 512 27.6 + 3.9, 1024 30.5 + 4.2; 8192 x 4096 512 62 + 4.9, 1024 48.8 + 6.6, 2048 54.8 + 11.5).
inline int back_groups(int64_t rows, int64_t cols) {
  if (cols > kBackCols) return (int)std::min<int64_t>(rows, 64);
  const int most = cols <= 128 ? 2048 : cols > 2048 && cols <= 8192 ? 1024 : 512;
  return (int)std::min<int64_t>(ceil_div(rows, rows_at_once(backward_form(cols))), most);
}

}  // namespace norm
}  // namespace muonh
