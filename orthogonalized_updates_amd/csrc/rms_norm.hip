// RMS norm with the residual's addition on gfx950, forward and backward (contract:
// include/muonh.h; the norms' weights are among the parameters that the AdamW
// step updates, model card "Puro", section "Training").
//
//   h = x + residual (rounded to h's type), r = rsqrt(mean(h^2) + eps), y = (h r) w
//   n = h r, g = dy w:  dh = r (g - n mean(g n)) + dresidual,  dw = sum over rows of dy n
//
// Both are bound by memory: every entry is read and written once, and a row
// stays in the registers of the lanes that share it between the two uses that
// its sum separates. The norm is of the h that is stored, so that y, the 8-bit
// forms and the backward pass see one h.
#include <algorithm>

#include "fp8_codes.h"
#include "norm_choice.h"
#include "rows.h"

namespace muonh {
namespace norm {
namespace {

using fp8::code_ld;
using fp8::fail;
using fp8::kBlock;
using fp8::overlap;
using fp8::Span;
using fp8::span;
using namespace rows;

__device__ __forceinline__ float rounded(float v, float) { return v; }
__device__ __forceinline__ float rounded(float v, __bf16) { return (float)(__bf16)v; }

// A lane's NV vectors of a row: vector v at column (v LPR + lane) 8. Zeros past
// the row's end. Where the columns are whole vectors, lanes past the end reload the
// last one, so that no load waits in a branch.
template <int LPR, int NV, typename T>
__device__ __forceinline__ void load_row(const T* p, int lane, int cols, Raw<T> (&raw)[NV]) {
  if ((cols & 7) == 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v) raw[v].load(p + min((v * LPR + lane) * 8, cols - 8));
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * 8;
      if (c + 8 <= cols) raw[v].load(p + c);
      else raw[v].load(p + c, cols - c);
    }
  }
}

// ---- sums over the lanes of a row, in all of them --------------------------------
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float sum_row16(float v) {
  v = add_dpp<0xB1>(v);     // quad [1,0,3,2]
  v = add_dpp<0x4E>(v);     // quad [2,3,0,1]
  v = add_dpp<0x141>(v);    // mirrored halves: the other quad of 8
  return add_dpp<0x140>(v); // mirrored row: the other 8
}
__device__ __forceinline__ float sum_wave(float v) {
  v = sum_row16(v);
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}
// LPR lanes; above 64 through `part` (one float per wave; the caller alternates
// between two of them from row to row, so that one barrier is enough).
template <int LPR>
__device__ __forceinline__ float sum_lanes(float v, float* part) {
  if constexpr (LPR == 16) return sum_row16(v);
  v = sum_wave(v);
  if constexpr (LPR > 64) {
    constexpr int W = LPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += part[w];
  }
  return v;
}
__device__ __forceinline__ uint32_t umax_row16(uint32_t v) {
  auto other = [](uint32_t a, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)a, decltype(ctrl)::value, 0xF, 0xF, false);
  };
  v = fp8::umax(v, other(v, std::integral_constant<int, 0xB1>{}));
  v = fp8::umax(v, other(v, std::integral_constant<int, 0x4E>{}));
  v = fp8::umax(v, other(v, std::integral_constant<int, 0x141>{}));
  return fp8::umax(v, other(v, std::integral_constant<int, 0x140>{}));
}

// ---- forward ----------------------------------------------------------------------
enum Out { kNone, kPlain, kCodes };  // beside h and r: nothing, y, y's 8-bit rows
struct FwdArgs {
  const void* x;
  const void* res;  // or nullptr: h = x, not stored
  void* h;
  const float* w;
  float* rstd;
  void* y;
  uint8_t *codes, *scales;
  int64_t rows, x_ld, res_ld, h_ld, y_ld;
  int cols, y_bf;
  float inv_cols, eps;
};

// One vector of y: columns c .. c + 7 of a row. In the kCodes form 16
// neighbouring lanes hold a block of 128, all of them call.
template <int OUT>
__device__ __forceinline__ void emit(const FwdArgs& a, int64_t row, int c, bool live, float (&y)[8]) {
  const int n = a.cols - c;
  if constexpr (OUT == kPlain) {
    if (!live || n <= 0) return;
    if (a.y_bf) store8(static_cast<__bf16*>(a.y) + row * a.y_ld + c, y, n);
    else store8(static_cast<float*>(a.y) + row * a.y_ld + c, y, n);
  } else if constexpr (OUT == kCodes) {
    if (n < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= n) y[j] = 0.f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t b = __float_as_uint(y[j]) & 0x7fffffffu;
      m = fp8::umax(m, b < 0x7f800000u ? b : 0u);
    }
    m = umax_row16(m);
    const uint32_t byte = fp8::scale_bytes2((m + 0xffffu) >> 16) & 0xffffu;
    const float s = fp8::scale_lo(byte);
    const int64_t ld = code_ld(a.cols);
    if (live && c < ld) {
      const uint2 q = make_uint2(fp8::codes4(y[0], y[1], y[2], y[3], s), fp8::codes4(y[4], y[5], y[6], y[7], s));
      *reinterpret_cast<uint2*>(a.codes + row * ld + c) = q;
      if ((c & (kBlock - 1)) == 0) fp8::put_scale(a.scales, row, c / kBlock, a.cols, byte);
    }
  }
}

// LPR lanes share a row, NV vectors of 8 each: a row is read once and stays in
// registers. A workgroup takes one set of rows, and further ones only in a call that would have more than
// kMaxGrid workgroups.
template <typename TX, typename TH, int LPR, int NV, int OUT>
__global__ __launch_bounds__(LPR < 256 ? 256 : LPR) void k_norm(FwdArgs a) {
  constexpr int kRows = LPR < 256 ? 256 / LPR : 1;
  __shared__ float part[2][LPR > 64 ? LPR / 64 : 1];
  const int lane = threadIdx.x & (LPR - 1);
  Raw<float> w[NV];
  if constexpr (OUT != kNone) load_row<LPR, NV>(a.w, lane, a.cols, w);
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += (int64_t)gridDim.x * kRows) {
    const int64_t mine = first + threadIdx.x / LPR;
    const bool live = mine < a.rows;
    const int64_t row = live ? mine : a.rows - 1;
    Raw<TX> x[NV];
    Raw<TH> res[NV];
    load_row<LPR, NV>(static_cast<const TX*>(a.x) + row * a.x_ld, lane, a.cols, x);
    if (a.res) load_row<LPR, NV>(static_cast<const TH*>(a.res) + row * a.res_ld, lane, a.cols, res);
    float h[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[v][j] = x[v].at(j);
        if (a.res) h[v][j] = rounded(h[v][j] + res[v].at(j), TH{});
      }
      if (c < a.cols) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(h[v][j], h[v][j], s);
        ss += s;
        if (a.res && live) store8(static_cast<TH*>(a.h) + row * a.h_ld + c, h[v], a.cols - c);
      }
    }
    ss = sum_lanes<LPR>(ss, part[turn]);
    turn ^= 1;
    const float r = rsqrtf(ss * a.inv_cols + a.eps);
    if (live && lane == 0) a.rstd[row] = r;
    if constexpr (OUT != kNone) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = (h[v][j] * r) * w[v].at(j);
        emit<OUT>(a, row, (v * LPR + lane) * 8, live, y);
      }
    }
  }
}

// Rows of any length: a workgroup to a row, which it reads twice.
template <typename TX, typename TH, int OUT>
__global__ __launch_bounds__(1024) void k_norm_long(FwdArgs a) {
  __shared__ float part[2][16];
  int turn = 0;
  const int width = (int)ceil_div(a.cols, kBlock) * kBlock;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const TX* px = static_cast<const TX*>(a.x) + row * a.x_ld;
    TH* ph = static_cast<TH*>(a.h) + row * a.h_ld;
    float ss = 0.f;
    for (int c = threadIdx.x * 8; c < a.cols; c += 8192) {
      const int n = a.cols - c;
      Raw<TX> x;
      if (n >= 8) x.load(px + c);
      else x.load(px + c, n);
      float h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = x.at(j);
      if (a.res) {
        const TH* pr = static_cast<const TH*>(a.res) + row * a.res_ld + c;
        Raw<TH> res;
        if (n >= 8) res.load(pr);
        else res.load(pr, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = rounded(h[j] + res.at(j), TH{});
        store8(ph + c, h, n);
      }
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s = __builtin_fmaf(h[j], h[j], s);
      ss += s;
    }
    ss = sum_lanes<1024>(ss, part[turn]);
    turn ^= 1;
    const float r = rsqrtf(ss * a.inv_cols + a.eps);
    if (threadIdx.x == 0) a.rstd[row] = r;
    if constexpr (OUT != kNone) {
      // whole rows of 16 lanes stay together: blocks of 128 columns
      for (int c = threadIdx.x * 8; c < width; c += 8192) {
        const int n = a.cols - c;
        float y[8];
        Raw<float> w;
        if (n >= 8) w.load(a.w + c);
        else w.load(a.w + c, n);
        auto scaled = [&](const auto& raw) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = (raw.at(j) * r) * w.at(j);
        };
        if (a.res) {  // what this thread stored above
          Raw<TH> q;
          if (n >= 8) q.load(ph + c);
          else q.load(ph + c, n);
          scaled(q);
        } else {
          Raw<TX> q;
          if (n >= 8) q.load(px + c);
          else q.load(px + c, n);
          scaled(q);
        }
        emit<OUT>(a, row, c, true, y);
      }
    }
  }
}

template <typename TX, typename TH, int OUT>
void launch_norm(const FwdArgs& a, hipStream_t s) {
  const Form f = forward_form(a.rows, a.cols);
  const dim3 grid((unsigned)forward_groups(a.rows, f));
#define MUONH_NORM(LPR, NV)             \
  if (f.lanes == LPR && f.vecs == NV) { \
    hipLaunchKernelGGL((k_norm<TX, TH, LPR, NV, OUT>), grid, dim3(LPR < 256 ? 256 : LPR), 0, s, a); \
    return;                             \
  }
  MUONH_NORM(16, 1)
  MUONH_NORM(64, 1)
  MUONH_NORM(64, 2)
  MUONH_NORM(64, 3)
  MUONH_NORM(256, 1)
  MUONH_NORM(256, 2)
  MUONH_NORM(256, 4)
  MUONH_NORM(1024, 2)
  MUONH_NORM(1024, 4)
#undef MUONH_NORM
  hipLaunchKernelGGL((k_norm_long<TX, TH, OUT>), grid, dim3(1024), 0, s, a);
}
template <typename TX, typename TH>
void launch_norm(const FwdArgs& a, Out out, hipStream_t s) {
  if (out == kNone) launch_norm<TX, TH, kNone>(a, s);
  else if (out == kPlain) launch_norm<TX, TH, kPlain>(a, s);
  else launch_norm<TX, TH, kCodes>(a, s);
}

// ---- backward ---------------------------------------------------------------------
struct BwdArgs {
  const void* dy;
  const void* h;
  const float *w, *rstd;
  const void* dres;  // or nullptr
  void* dh;
  float* part;       // [groups][cols]: sums of dy n over each group's rows
  float* mean;       // [rows]: mean(g n), of k_norm_dots
  int64_t rows, dy_ld, h_ld, dres_ld, dh_ld;
  int cols, groups;
  float inv_cols;
};

// As k_norm: LPR lanes share a row, whose dy and h they hold. Each workgroup
// takes every gridDim-th set of rows and keeps its lanes' columns of dw in
// registers, one partial sum per workgroup at the end. 8192 x 2048 bf16 with a residual's
// gradient: 27.6 us, 134 MB at 4.9 TB/s (four waves to a row: 28.3).
template <typename TD, typename TH, int LPR, int NV>
__global__ __launch_bounds__(LPR < 256 ? 256 : LPR) void k_norm_back(BwdArgs a) {
  constexpr int kRows = LPR < 256 ? 256 / LPR : 1;
  __shared__ float part[2][LPR > 64 ? LPR / 64 : 1];
  __shared__ float sums[kRows > 1 ? kRows : 1][kRows > 1 ? LPR * NV * 8 : 1];
  const int lane = threadIdx.x & (LPR - 1), group = threadIdx.x / LPR;
  Raw<float> w[NV];
  load_row<LPR, NV>(a.w, lane, a.cols, w);
  float dw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = 0.f;
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < a.rows; first += (int64_t)gridDim.x * kRows) {
    const bool live = first + group < a.rows;
    const int64_t row = live ? first + group : a.rows - 1;
    Raw<TD> dy[NV];
    Raw<TH> h[NV], res[NV];
    load_row<LPR, NV>(static_cast<const TD*>(a.dy) + row * a.dy_ld, lane, a.cols, dy);
    load_row<LPR, NV>(static_cast<const TH*>(a.h) + row * a.h_ld, lane, a.cols, h);
    if (a.dres) load_row<LPR, NV>(static_cast<const TH*>(a.dres) + row * a.dres_ld, lane, a.cols, res);
    const float r = a.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if ((v * LPR + lane) * 8 < a.cols && live) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float t = dy[v].at(j) * (h[v].at(j) * r);
          dw[v][j] += t;
          s += t * w[v].at(j);
        }
        dot += s;
      }
    }
    const float mean = sum_lanes<LPR>(dot, part[turn]) * a.inv_cols;
    turn ^= 1;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * 8;
      if (c >= a.cols || !live) continue;
      float d[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] = (dy[v].at(j) * w[v].at(j) - (h[v].at(j) * r) * mean) * r;
        if (a.dres) d[j] += res[v].at(j);
      }
      store8(static_cast<TH*>(a.dh) + row * a.dh_ld + c, d, a.cols - c);
    }
  }
  float* out = a.part + (int64_t)blockIdx.x * a.cols;
  if constexpr (kRows > 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[group][(v * LPR + lane) * 8 + j] = dw[v][j];
    __syncthreads();
    for (int c = threadIdx.x; c < a.cols; c += 256) {
      float s = sums[0][c];
#pragma unroll
      for (int k = 1; k < kRows; ++k) s += sums[k][c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * 8;
      if (c < a.cols) store8(out + c, dw[v], a.cols - c);
    }
  }
}

// Rows of any length: mean(g n) of each row first, then the rest by slabs of
// 2048 columns, in which a thread has 8 columns of every row of its group.
template <typename TD, typename TH>
__global__ __launch_bounds__(1024) void k_norm_dots(BwdArgs a) {
  __shared__ float part[2][16];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const TD* pd = static_cast<const TD*>(a.dy) + row * a.dy_ld;
    const TH* ph = static_cast<const TH*>(a.h) + row * a.h_ld;
    const float r = a.rstd[row];
    float dot = 0.f;
    for (int c = threadIdx.x * 8; c < a.cols; c += 8192) {
      const int n = a.cols - c;
      Raw<TD> dy;
      Raw<TH> h;
      Raw<float> w;
      if (n >= 8) {
        dy.load(pd + c);
        h.load(ph + c);
        w.load(a.w + c);
      } else {
        dy.load(pd + c, n);
        h.load(ph + c, n);
        w.load(a.w + c, n);
      }
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) s += (dy.at(j) * (h.at(j) * r)) * w.at(j);
      dot += s;
    }
    dot = sum_lanes<1024>(dot, part[turn]);
    turn ^= 1;
    if (threadIdx.x == 0) a.mean[row] = dot * a.inv_cols;
  }
}
template <typename TD, typename TH>
__global__ __launch_bounds__(256) void k_norm_back_long(BwdArgs a) {
  const int c = ((int)blockIdx.x * 256 + threadIdx.x) * 8, n = a.cols - c;
  if (n <= 0) return;
  Raw<float> w;
  if (n >= 8) w.load(a.w + c);
  else w.load(a.w + c, n);
  float dw[8] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += a.groups) {
    const TD* pd = static_cast<const TD*>(a.dy) + row * a.dy_ld + c;
    const TH* ph = static_cast<const TH*>(a.h) + row * a.h_ld + c;
    Raw<TD> dy;
    Raw<TH> h, res;
    if (n >= 8) {
      dy.load(pd);
      h.load(ph);
    } else {
      dy.load(pd, n);
      h.load(ph, n);
    }
    if (a.dres) {
      const TH* pr = static_cast<const TH*>(a.dres) + row * a.dres_ld + c;
      if (n >= 8) res.load(pr);
      else res.load(pr, n);
    }
    const float r = a.rstd[row], mean = a.mean[row];
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float nh = h.at(j) * r;
      dw[j] += dy.at(j) * nh;
      d[j] = (dy.at(j) * w.at(j) - nh * mean) * r;
      if (a.dres) d[j] += res.at(j);
    }
    store8(static_cast<TH*>(a.dh) + row * a.dh_ld + c, d, n);
  }
  store8(a.part + (int64_t)blockIdx.y * a.cols + c, dw, n);
}

// dw[c] (+)= the groups' partial sums, in a fixed order: 16 columns per
// workgroup, 64 lanes of groups for each 4 of them, then those 64 sums by 8.
__global__ __launch_bounds__(256) void k_norm_join(const float* part, int groups, int cols, float* dw, int accumulate) {
  __shared__ float sums[64][16 + 1], eight[8][16 + 1];
  const int x = (threadIdx.x & 3) * 4, y = threadIdx.x >> 2, c = (int)blockIdx.x * 16 + x;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (c + 4 <= cols) {
#pragma unroll 8
    for (int g = y; g < groups; g += 64) s += *reinterpret_cast<const f32x4_a4*>(part + (int64_t)g * cols + c);
  } else {
    for (int g = y; g < groups; g += 64)
      for (int j = 0; j < 4; ++j)
        if (c + j < cols) s[j] += part[(int64_t)g * cols + c + j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) sums[y][x + j] = s[j];
  __syncthreads();
  const int col = threadIdx.x & 15, k = threadIdx.x >> 4;
  if (k < 8) {
    float t = sums[8 * k][col];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += sums[8 * k + i][col];
    eight[k][col] = t;
  }
  __syncthreads();
  const int out = (int)blockIdx.x * 16 + col;
  if (k == 0 && out < cols) {
    float t = eight[0][col];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += eight[i][col];
    dw[out] = accumulate ? dw[out] + t : t;
  }
}

size_t back_bytes(int64_t rows, int64_t cols) {
  const size_t part = (size_t)back_groups(rows, cols) * (size_t)cols * sizeof(float);
  return part + (cols > kBackCols ? (size_t)rows * sizeof(float) : 0);
}

template <typename TD, typename TH>
void launch_back(const BwdArgs& a, hipStream_t s) {
  const Form f = backward_form(a.cols);
  const dim3 grid((unsigned)a.groups);
#define MUONH_NORM(LPR, NV)             \
  if (f.lanes == LPR && f.vecs == NV) { \
    hipLaunchKernelGGL((k_norm_back<TD, TH, LPR, NV>), grid, dim3(LPR < 256 ? 256 : LPR), 0, s, a); \
    return;                             \
  }
  MUONH_NORM(16, 1)
  MUONH_NORM(64, 1)
  MUONH_NORM(64, 2)
  MUONH_NORM(64, 3)
  MUONH_NORM(64, 4)
  MUONH_NORM(256, 2)
  MUONH_NORM(256, 4)
  MUONH_NORM(1024, 2)
#undef MUONH_NORM
  hipLaunchKernelGGL((k_norm_dots<TD, TH>), dim3((unsigned)std::min<int64_t>(a.rows, kMaxGrid)), dim3(1024), 0, s, a);
  hipLaunchKernelGGL((k_norm_back_long<TD, TH>), dim3((unsigned)ceil_div(ceil_div(a.cols, 8), 256), (unsigned)a.groups),
                     dim3(256), 0, s, a);
}

// A mean over no columns is no number: refused.
int check_shape(int64_t rows, int64_t cols) {
  if (fp8::bad_dim(rows) || fp8::bad_dim(cols) || cols == 0)
    return fail(MUONH_ESHAPE, "%lld x %lld: rows out of [0, %d] or columns out of [1, %d]", (long long)rows,
                (long long)cols, MUONH_MAX_FP8_DIM, MUONH_MAX_FP8_DIM);
  return MUONH_OK;
}

}  // namespace
}  // namespace norm
}  // namespace muonh

extern "C" {

int muonh_rms_norm(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t x_ld, const void* residual,
                   int32_t h_dtype, int64_t residual_ld, void* h, int64_t h_ld, const float* weight, float eps,
                   float* rstd, void* y, int32_t y_dtype, int64_t y_ld, void* codes, void* scales, void* codes_t,
                   void* scales_t, void* stream) {
  using namespace muonh;
  using namespace muonh::norm;
  if (bad_dtype(x_dtype)) return fail(MUONH_EINVAL, "x_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", x_dtype);
  if (residual && bad_dtype(h_dtype))
    return fail(MUONH_EINVAL, "h_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", h_dtype);
  if (y && bad_dtype(y_dtype)) return fail(MUONH_EINVAL, "y_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", y_dtype);
  if (const int err = check_shape(rows, cols)) return err;
  if (!(eps >= 0.f) || eps > 3.4e38f) return fail(MUONH_EINVAL, "eps=%g must be finite and >= 0", (double)eps);
  if (rows == 0) return MUONH_OK;
  if (!codes != !scales || !codes_t != !scales_t)
    return fail(MUONH_EINVAL, "codes and scales (codes_t and scales_t) go together");
  if (!y == !(codes || codes_t)) return fail(MUONH_EINVAL, "either y or 8-bit forms");
  if (!residual != !h) return fail(MUONH_EINVAL, "residual and h go together");
  const Mat in = {"x", x, x_dtype, x_ld}, res = {"residual", residual, h_dtype, residual_ld}, sum = {"h", h, h_dtype, h_ld},
            out = {"y", y, y_dtype, y_ld};
  if (const int err = check_mat(in, cols)) return err;
  if (residual) {
    if (const int err = check_mat(res, cols)) return err;
    if (const int err = check_mat(sum, cols)) return err;
  }
  if (y)
    if (const int err = check_mat(out, cols)) return err;
  if (!weight || misaligned(weight, 4)) return fail(MUONH_EINVAL, "weight must be a 4-byte aligned array of cols floats");
  if (!rstd || misaligned(rstd, 4)) return fail(MUONH_EINVAL, "rstd must be a 4-byte aligned array of rows floats");
  if (misaligned(codes, 16) || misaligned(codes_t, 16) || misaligned(scales, 4) || misaligned(scales_t, 4))
    return fail(MUONH_EINVAL, "codes must be 16-byte and scales 4-byte aligned");
  if (codes_t && !fp8::tiles_fit(rows, cols)) return fail(MUONH_ESHAPE, "2^24 tiles of 128 x 128 or more");
  // h may take the place of x or of the residual, entry by entry
  const Mat* const mats[4] = {&in, &res, &sum, &out};
  for (int i = 2; i < 4; ++i)
    for (int j = 0; j < i; ++j) {
      if (!mats[i]->p || !mats[j]->p || (i == 2 && same(*mats[i], *mats[j]))) continue;
      if (meet(*mats[i], *mats[j], rows, cols)) return fail(MUONH_EALIAS, "%s overlaps %s", mats[i]->name, mats[j]->name);
    }
  const Span spans[10] = {span_of(in, rows, cols),
                          span_of(res, rows, cols),
                          span("weight", weight, cols * 4),
                          span_of(sum, rows, cols),
                          span_of(out, rows, cols),
                          span("rstd", rstd, rows * 4),
                          span("codes", codes, rows * code_ld(cols)),
                          span("scales", scales, rows * fp8::scale_ld(cols)),
                          span("codes_t", codes_t, cols * code_ld(rows)),
                          span("scales_t", scales_t, cols * fp8::scale_ld(rows))};
  for (int i = 3; i < 10; ++i)
    for (int j = 0; j < i; ++j) {
      const bool both_mats = i < 5 && j != 2;  // done above
      if (!both_mats && overlap(spans[i], spans[j]))
        return fail(MUONH_EALIAS, "%s overlaps %s", spans[i].name, spans[j].name);
    }

  FwdArgs a{};
  a.x = x;
  a.res = residual;
  a.h = h;
  a.w = weight;
  a.rstd = rstd;
  a.y = y;
  a.rows = rows;
  a.x_ld = x_ld;
  a.res_ld = residual_ld;
  a.h_ld = h_ld;
  a.y_ld = y_ld;
  a.cols = (int)cols;
  a.y_bf = y_dtype == MUONH_DT_BF16;
  a.inv_cols = (float)(1.0 / (double)cols);
  a.eps = eps;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  // The transposed form groups along rows, so it needs whole 128 x 128 tiles
  // after the rows' sums: a second pass over h, which is still in the memory-side
  // cache, writes the 8-bit forms (8192 x 2048 bf16 with a residual: 18.2 + 17.8 us; with the plain form
  // written by the first pass 23.9 + 14.0).
  const Out form = y ? kPlain : codes_t ? kNone : kCodes;
  const int32_t hd = residual ? h_dtype : x_dtype;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (x_dtype == MUONH_DT_BF16) {
    if (hd == MUONH_DT_BF16) launch_norm<__bf16, __bf16>(a, form, s);
    else launch_norm<__bf16, float>(a, form, s);
  } else {
    if (hd == MUONH_DT_BF16) launch_norm<float, __bf16>(a, form, s);
    else launch_norm<float, float>(a, form, s);
  }
  if (const int err = launched("rms norm")) return err;
  if (!codes_t) return MUONH_OK;
  return fp8::quantize_normed(residual ? h : x, hd, rows, cols, residual ? h_ld : x_ld, rstd, weight, codes, scales,
                              codes_t, scales_t, s);
}

size_t muonh_rms_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  using namespace muonh;
  if (fp8::bad_dim(rows) || fp8::bad_dim(cols) || rows == 0 || cols == 0) return 0;
  return norm::back_bytes(rows, cols);
}

int muonh_rms_norm_backward(const void* dy, int32_t dy_dtype, int64_t dy_ld, const void* h, int32_t h_dtype,
                            int64_t rows, int64_t cols, int64_t h_ld, const float* weight, const float* rstd,
                            const void* dresidual, int64_t dresidual_ld, void* dh, int64_t dh_ld, float* dweight,
                            int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace muonh;
  using namespace muonh::norm;
  if (bad_dtype(dy_dtype)) return fail(MUONH_EINVAL, "dy_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", dy_dtype);
  if (bad_dtype(h_dtype)) return fail(MUONH_EINVAL, "h_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", h_dtype);
  if (const int err = check_shape(rows, cols)) return err;
  if (!dweight || misaligned(dweight, 4)) return fail(MUONH_EINVAL, "dweight must be a 4-byte aligned array of cols floats");
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 join((unsigned)ceil_div(cols, 16));
  if (rows == 0) {  // the sum over no rows
    if (accumulate) return MUONH_OK;
    hipLaunchKernelGGL(k_norm_join, join, dim3(256), 0, s, nullptr, 0, (int)cols, dweight, 0);
    return launched("rms norm backward");
  }
  const Mat d = {"dy", dy, dy_dtype, dy_ld}, x = {"h", h, h_dtype, h_ld}, res = {"dresidual", dresidual, h_dtype, dresidual_ld},
            out = {"dh", dh, h_dtype, dh_ld};
  if (const int err = check_mat(d, cols)) return err;
  if (const int err = check_mat(x, cols)) return err;
  if (dresidual)
    if (const int err = check_mat(res, cols)) return err;
  if (const int err = check_mat(out, cols)) return err;
  if (!weight || misaligned(weight, 4)) return fail(MUONH_EINVAL, "weight must be a 4-byte aligned array of cols floats");
  if (!rstd || misaligned(rstd, 4)) return fail(MUONH_EINVAL, "rstd must be a 4-byte aligned array of rows floats");
  const size_t need = back_bytes(rows, cols);
  if (!workspace) return fail(MUONH_EWORKSPACE, "workspace is NULL, the call needs %zu bytes", need);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(MUONH_EWORKSPACE, "workspace must be 256-byte aligned");
  if (workspace_bytes < need)
    return fail(MUONH_EWORKSPACE, "workspace has %zu bytes, the call needs %zu", workspace_bytes, need);
  // dh may take the place of dy or of dresidual, entry by entry
  const Mat* const mats[3] = {&d, &x, &res};
  for (int j = 0; j < 3; ++j) {
    if (!mats[j]->p || (j != 1 && same(out, *mats[j]))) continue;
    if (meet(out, *mats[j], rows, cols)) return fail(MUONH_EALIAS, "dh overlaps %s", mats[j]->name);
  }
  const Span spans[8] = {span_of(d, rows, cols),          span_of(x, rows, cols),
                         span_of(res, rows, cols),        span("weight", weight, cols * 4),
                         span("rstd", rstd, rows * 4),    span_of(out, rows, cols),
                         span("dweight", dweight, cols * 4), span("workspace", workspace, (int64_t)need)};
  for (int i = 5; i < 8; ++i)
    for (int j = i == 5 ? 3 : 0; j < i; ++j)
      if (overlap(spans[i], spans[j])) return fail(MUONH_EALIAS, "%s overlaps %s", spans[i].name, spans[j].name);

  BwdArgs a{};
  a.dy = dy;
  a.h = h;
  a.w = weight;
  a.rstd = rstd;
  a.dres = dresidual;
  a.dh = dh;
  a.rows = rows;
  a.dy_ld = dy_ld;
  a.h_ld = h_ld;
  a.dres_ld = dresidual_ld;
  a.dh_ld = dh_ld;
  a.cols = (int)cols;
  a.groups = back_groups(rows, cols);
  a.inv_cols = (float)(1.0 / (double)cols);
  a.part = static_cast<float*>(workspace);
  a.mean = a.part + (size_t)a.groups * (size_t)cols;
  if (dy_dtype == MUONH_DT_BF16) {
    if (h_dtype == MUONH_DT_BF16) launch_back<__bf16, __bf16>(a, s);
    else launch_back<__bf16, float>(a, s);
  } else {
    if (h_dtype == MUONH_DT_BF16) launch_back<float, __bf16>(a, s);
    else launch_back<float, float>(a, s);
  }
  hipLaunchKernelGGL(k_norm_join, join, dim3(256), 0, s, a.part, a.groups, (int)cols, dweight, accumulate != 0);
  return launched("rms norm backward");
}

}  // extern "C"
