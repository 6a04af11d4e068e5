// Quantization to microscaled 4-bit floats on gfx950, and back (formats:
// include/muonh.h).
//
// As for 8 bits (fp8_quantize.hip), one workgroup takes one 128 x 128 tile of
// the source: 16 x 16 threads, each an 8 x 8 patch. A group of 32 along a row is
// 4 neighbouring lanes, one of 32 along a column the 4 thread rows of a wave, so that
// maxima are lane exchanges. 4 (fp32) or 2 (bf16) bytes read and 1/2 + 1/32 or
// twice that written per entry: HBM-bound.
//
// A scale is a power of two, so the conversion instruction, which divides by
// it, rounds once (to nearest, ties to even).
#include "fp4_internal.h"
#include "fp8_codes.h"

namespace muonh {
namespace fp4 {
namespace {

using fp8::pmax;
using fp8::u16x2;
using fp8::umax;
using rows::bad_dtype;
using rows::launched;
using rows::misaligned;

constexpr int kThreads = 256;
constexpr int kTile = 128;

struct Args {
  const void* src;
  uint8_t *codes, *scales, *codes_t, *scales_t;
  int64_t rows, cols, src_ld;
  uint32_t tiles, tiles_c;
};

// Maxima are of magnitudes' bits, in pairs of 16 (the upper halves of fp32's,
// rounded up); from kNotFinite on an entry is an infinity or a NaN.
constexpr uint32_t kNotFinite = 0x7f80u;
__device__ __forceinline__ uint32_t upper16(uint32_t m) {
  return m >= 0x7f800000u ? kNotFinite : min((m + 0xffffu) >> 16, kNotFinite - 1);
}
// Scale bytes e + 127, e >= -126, 255 (NaN) for a group that is not finite: with a =
// 1.f * 2^E and 6 = 1.5 * 2^2, e = E - 2 where 1.f <= 1.5 (0x40 of the 7 bits), else E - 1.
__device__ __forceinline__ uint32_t scale_bytes2(uint32_t m) {
  const u16x2 e =
      __builtin_elementwise_max((__builtin_bit_cast(u16x2, m) + u16x2{0x3f, 0x3f}) >> u16x2{7, 7}, u16x2{3, 3}) - u16x2{2, 2};
  const uint32_t b = __builtin_bit_cast(uint32_t, e);
  return ((m & 0xffffu) >= kNotFinite ? 0xffu : b & 0xffffu) | (m >= kNotFinite << 16 ? 0xff0000u : b & 0xffff0000u);
}

// 8 entries (4 pairs of bf16, or floats) over a scale to 8 codes, the first in the low bits.
// A group whose byte is 255 gets zeros.
__device__ __forceinline__ uint32_t codes8(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  uint32_t q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, __builtin_bit_cast(fp8::bf16x2, a), s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(fp8::bf16x2, b), s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(fp8::bf16x2, c), s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(fp8::bf16x2, d), s, 3);
  return byte == 255 ? 0u : q;
}
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], uint32_t byte) {
  const float s = __uint_as_float(byte << 23);
  uint32_t q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], s, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], s, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], s, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], s, 3);
  return byte == 255 ? 0u : q;
}

// The 4 scale bytes of tile column t (of the last one, `tiles_c` - 1, also the zeros to the row's end).
__device__ __forceinline__ void put_scales(uint8_t* s, int64_t row, int64_t cols, uint32_t t, uint32_t tiles_c, uint32_t bytes) {
  const int64_t ld = scale_ld(cols);
  uint32_t* p = reinterpret_cast<uint32_t*>(s + row * ld);
  const int left = (int)(ceil_div(cols, kGroup) - 4 * (int64_t)t);  // groups from here on
  p[t] = left >= 4 ? bytes : bytes & ((1u << (8 * left)) - 1);
  if (t == tiles_c - 1)
    for (uint32_t j = tiles_c; j < ld / 4; ++j) p[j] = 0;
}

// Lane t of a quad holds dword t of rows 0 .. 3, in q[0] .. q[3]: afterwards all 4 of row t, by two
// exchanges of halves.
template <int CTRL>
__device__ __forceinline__ uint32_t from(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}
__device__ __forceinline__ uint4 quad_rows(const uint32_t* q, int t) {
  const bool odd = t & 1, high = t & 2;
  uint32_t u[2][2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t got = from<0xB1>(odd ? q[2 * p] : q[2 * p + 1]);  // quad [1,0,3,2]
    u[p][0] = odd ? got : q[2 * p];
    u[p][1] = odd ? q[2 * p + 1] : got;
  }
  uint32_t got[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) got[e] = from<0x4E>(high ? u[0][e] : u[1][e]);  // quad [2,3,0,1]
  return high ? make_uint4(got[0], got[1], u[1][0], u[1][1]) : make_uint4(u[0][0], u[0][1], got[0], got[1]);
}

// Thread (ty, tx) = (tid / 16, tid % 16) holds rows 8 ty .. +7, columns
// 8 tx .. +7 of the tile. PLAIN, TRANS: the forms written. Tiles are dealt to
// the XCDs as in the 8-bit kernel.
template <bool BF, bool PLAIN, bool TRANS>
__global__ __launch_bounds__(kThreads, 4) void k_quantize4(Args a) {
  __shared__ __attribute__((aligned(16))) uint32_t row_bytes[kTile];      // 4 scale bytes of each row
  __shared__ __attribute__((aligned(16))) uint8_t col_bytes[4][kTile];    // one of each column for each wave's 32 rows
  __shared__ __attribute__((aligned(16))) uint8_t stage[TRANS ? kTile * kTile / 2 : 16];  // transposed codes
  const uint32_t x = blockIdx.x & 7;
  const uint32_t lo = (uint32_t)(((uint64_t)x * a.tiles) >> 3);
  const uint32_t count = (uint32_t)(((uint64_t)(x + 1) * a.tiles) >> 3) - lo;
  if ((blockIdx.x >> 3) >= count) return;
  uint32_t index = (blockIdx.x >> 3) + ((x * count) >> 3);
  if (index >= count) index -= count;
  index += lo;
  // two tile rows at a time: neighbours in both directions, whose codes share cache lines (64 bytes of either
  // form a row and tile), come one after the other
  const uint32_t tiles_r = a.tiles / a.tiles_c, band = index / (2 * a.tiles_c), in = index - band * (2 * a.tiles_c);
  const uint32_t high = min(2u, tiles_r - 2 * band);
  const uint32_t tc = high == 2 ? in >> 1 : in, tr = 2 * band + (high == 2 ? in & 1 : 0);
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t rows = a.rows, cols = a.cols;
  const int64_t r0 = (int64_t)tr * kTile + 8 * ty, c0 = (int64_t)tc * kTile + 8 * tx;

  float v[BF ? 1 : 8][8];
  fp8::u32x4_a2 w[BF ? 8 : 1];
  uint32_t rmax[4], cmax[4];  // of rows 2k, 2k + 1 and of columns 2k, 2k + 1
  if constexpr (BF) {
    fp8::load_patch(static_cast<const uint16_t*>(a.src), a.src_ld, r0, c0, rows, cols, w);
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t m = w[i][d] & 0x7fff7fffu;
        r[i] = d ? pmax(r[i], m) : m;
        cmax[d] = i ? pmax(cmax[d], m) : m;
      }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      rmax[k] = pmax(fp8::low_halves(r[2 * k], r[2 * k + 1]), fp8::high_halves(r[2 * k], r[2 * k + 1]));
  } else {
    fp8::load_patch(static_cast<const float*>(a.src), a.src_ld, r0, c0, rows, cols, v);
    uint32_t r[8], c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t m = __float_as_uint(v[i][j]) & 0x7fffffffu;
        r[i] = j ? umax(r[i], m) : m;
        c[j] = i ? umax(c[j], m) : m;
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      rmax[k] = upper16(r[2 * k]) | upper16(r[2 * k + 1]) << 16;
      cmax[k] = upper16(c[2 * k]) | upper16(c[2 * k + 1]) << 16;
    }
  }

  if constexpr (PLAIN) {
    const int64_t ld = code_ld(cols);
    uint32_t rows8[8], mine = 0;  // mine: the 4 bytes of row tx, in the lanes tx < 8
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // the 4 lanes of a group
      const uint32_t b = scale_bytes2(fp8::pmax_dpp<0x4E>(fp8::pmax_dpp<0xB1>(rmax[k])));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 2 * k + h;
        const uint32_t byte = h ? b >> 16 : b & 0xffu;
        if constexpr (BF) rows8[i] = codes8(w[i][0], w[i][1], w[i][2], w[i][3], byte);
        else rows8[i] = codes8(v[i], byte);
        // the 4 quads' bytes together (a byte's store by each quad: lanes that write to one word wait for each other)
        uint32_t all = byte << (8 * (tx >> 2));
        all |= from<0x124>(all);  // row rotated by 4
        all |= from<0x128>(all);  // and by 8
        mine = tx == i ? all : mine;
      }
    }
    if (tx < 8) row_bytes[8 * ty + tx] = mine;
    // 16 bytes a lane, a quad's group of a row each (8192 x 2048 bf16 in both forms 13.4 -> 12.5
    // us against 4-byte stores)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 q = quad_rows(rows8 + 4 * h, tx & 3);
      const int64_t r = r0 + 4 * h + (tx & 3);
      if (r < rows) *reinterpret_cast<uint4*>(a.codes + r * ld + (int64_t)tc * (kTile / 2) + (tx >> 2) * 16) = q;
    }
  }

  if constexpr (TRANS) {
    uint32_t bytes8[2] = {0, 0};  // of the lane's 8 columns
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      // the 4 thread rows of the wave
      auto p = __builtin_amdgcn_permlane16_swap(cmax[d], cmax[d], false, false);
      uint32_t m = pmax(p[0], p[1]);
      p = __builtin_amdgcn_permlane32_swap(m, m, false, false);
      const uint32_t b = scale_bytes2(pmax(p[0], p[1]));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 2 * d + h;
        const uint32_t byte = h ? b >> 16 : b & 0xffu;
        uint32_t q;
        if constexpr (BF) {
          auto rows2 = [&](int i) { return h ? fp8::high_halves(w[i][d], w[i + 1][d]) : fp8::low_halves(w[i][d], w[i + 1][d]); };
          q = codes8(rows2(0), rows2(2), rows2(4), rows2(6), byte);
        } else {
          const float col[8] = {v[0][j], v[1][j], v[2][j], v[3][j], v[4][j], v[5][j], v[6][j], v[7][j]};
          q = codes8(col, byte);
        }
        // Column 8 tx + j is the stage's row 16 j + tx (64 bytes), and its piece ty lies at ty ^ (tx & 12): the
        // 64 lanes of a store, 4 pieces of 16 columns, fall on 64 banks.
        *reinterpret_cast<uint32_t*>(stage + ((16 * j + tx) * 16 + (ty ^ (tx & 12))) * 4) = q;
        bytes8[j >> 2] |= byte << (8 * (j & 3));
      }
    }
    if ((ty & 3) == 0) *reinterpret_cast<uint2*>(&col_bytes[ty >> 2][8 * tx]) = make_uint2(bytes8[0], bytes8[1]);
  }
  __syncthreads();
  if constexpr (PLAIN) {
    const int64_t r = (int64_t)tr * kTile + tid;
    if (tid < kTile && r < rows) {
      put_scales(a.scales, r, cols, tc, a.tiles_c, row_bytes[tid]);
      // codes to a multiple of 256: an odd last tile's other half
      if (tc == a.tiles_c - 1 && (tc & 1) == 0) {
        uint4* p = reinterpret_cast<uint4*>(a.codes + r * code_ld(cols) + (int64_t)(tc + 1) * (kTile / 2));
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = make_uint4(0, 0, 0, 0);
      }
    }
  }
  if constexpr (TRANS) {
    const int64_t ld = code_ld(rows);
    const int u = tid & 3;
    const bool pad = tr == tiles_r - 1 && (tr & 1) == 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = (tid >> 2) + 64 * k, sx = c >> 3;
      const int64_t col = (int64_t)tc * kTile + c;
      const uint4 q = *reinterpret_cast<const uint4*>(stage + ((16 * (c & 7) + sx) * 16 + ((4 * u) ^ (sx & 12))) * 4);
      if (col >= cols) continue;
      uint8_t* p = a.codes_t + col * ld + (int64_t)tr * (kTile / 2) + 16 * u;
      *reinterpret_cast<uint4*>(p) = q;
      if (pad) *reinterpret_cast<uint4*>(p + kTile / 2) = make_uint4(0, 0, 0, 0);
    }
    const int c = tid - (kThreads - kTile);
    if (c >= 0 && (int64_t)tc * kTile + c < cols)
      put_scales(a.scales_t, (int64_t)tc * kTile + c, rows, tr, tiles_r,
                 (uint32_t)col_bytes[0][c] | (uint32_t)col_bytes[1][c] << 8 | (uint32_t)col_bytes[2][c] << 16 |
                     (uint32_t)col_bytes[3][c] << 24);
  }
}

// ---- values -----------------------------------------------------------------------
struct ValArgs {
  const uint8_t *codes, *scales;
  void* out;
  int64_t rows, ld, sld, out_ld;
  int cols, vecs;
};
// A thread takes kPer times 8 codes of the workgroup's stretch of the list of all rows' eights, whose
// loads run together. Exact in either type. 8192 x 2048 to bf16: 9.2 us (4.6 TB/s).
constexpr int kPer = 4;
template <typename T>
__global__ __launch_bounds__(256) void k_values(ValArgs a) {
  const uint64_t total = (uint64_t)a.rows * (uint32_t)a.vecs;
  for (uint64_t base = (uint64_t)blockIdx.x * (256 * kPer); base < total; base += (uint64_t)gridDim.x * (256 * kPer)) {
    const int64_t r0 = (int64_t)(base / (uint32_t)a.vecs);
    const uint32_t rest = (uint32_t)(base - (uint64_t)r0 * (uint32_t)a.vecs);
    int64_t r[kPer];
    int c[kPer];
    uint32_t q[kPer], e[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const uint32_t i = rest + k * 256 + threadIdx.x, d = i / (uint32_t)a.vecs;
      r[k] = min(r0 + d, a.rows);
      c[k] = (int)(i - d * (uint32_t)a.vecs);
      const int64_t row = min(r[k], a.rows - 1);
      q[k] = *reinterpret_cast<const uint32_t*>(a.codes + row * a.ld + 4 * c[k]);
      e[k] = a.scales[row * a.sld + (c[k] >> 2)];
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (r[k] >= a.rows) continue;
      const float s = __uint_as_float(e[k] << 23);
      float v[8];
      auto two = [&](auto n) {
        const auto f = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[k], s, decltype(n)::value);
        v[2 * decltype(n)::value] = f[0];
        v[2 * decltype(n)::value + 1] = f[1];
      };
      two(std::integral_constant<int, 0>{});
      two(std::integral_constant<int, 1>{});
      two(std::integral_constant<int, 2>{});
      two(std::integral_constant<int, 3>{});
      rows::store8(static_cast<T*>(a.out) + r[k] * a.out_ld + 8 * c[k], v, a.cols - 8 * c[k]);
    }
  }
}

template <bool BF>
void launch_forms(const Args& a, hipStream_t s) {
  const dim3 grid((unsigned)(8 * ceil_div(a.tiles, 8))), thr(kThreads);
  if (a.codes && a.codes_t) hipLaunchKernelGGL((k_quantize4<BF, true, true>), grid, thr, 0, s, a);
  else if (a.codes) hipLaunchKernelGGL((k_quantize4<BF, true, false>), grid, thr, 0, s, a);
  else hipLaunchKernelGGL((k_quantize4<BF, false, true>), grid, thr, 0, s, a);
}

}  // namespace
}  // namespace fp4
}  // namespace muonh

extern "C" {

int64_t muonh_fp4_ld(int64_t cols) { return muonh::fp8::bad_dim(cols) ? 0 : muonh::fp4::code_ld(cols); }

int64_t muonh_fp4_scale_ld(int64_t cols) { return muonh::fp8::bad_dim(cols) ? 0 : muonh::fp4::scale_ld(cols); }

int muonh_fp4_quantize(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t src_ld, void* codes,
                       void* scales, void* codes_t, void* scales_t, void* stream) {
  using namespace muonh;
  using namespace muonh::fp4;
  if (bad_dtype(dtype)) return fail(MUONH_EINVAL, "dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", dtype);
  if (bad_dim(rows) || bad_dim(cols))
    return fail(MUONH_ESHAPE, "shape %lld x %lld out of [0, %d]", (long long)rows, (long long)cols, MUONH_MAX_FP8_DIM);
  if (src_ld < cols || src_ld > (1LL << 36))
    return fail(MUONH_EINVAL, "src_ld=%lld out of [cols=%lld, 2^36]", (long long)src_ld, (long long)cols);
  if (rows == 0 || cols == 0) return MUONH_OK;
  if (!src) return fail(MUONH_EINVAL, "src is NULL");
  if (!codes != !scales || !codes_t != !scales_t)
    return fail(MUONH_EINVAL, "codes and scales (codes_t and scales_t) go together");
  if (!codes && !codes_t) return fail(MUONH_EINVAL, "no output given");
  const int esize = dtype == MUONH_DT_BF16 ? 2 : 4;
  if (misaligned(src, esize)) return fail(MUONH_EINVAL, "src is not aligned to its type");
  if (misaligned(codes, 16) || misaligned(codes_t, 16) || misaligned(scales, 8) || misaligned(scales_t, 8))
    return fail(MUONH_EINVAL, "codes must be 16-byte and scales 8-byte aligned");
  if (!fp8::tiles_fit(rows, cols)) return fail(MUONH_ESHAPE, "2^24 tiles of 128 x 128 or more");
  const Span spans[5] = {span("src", src, ((rows - 1) * src_ld + cols) * esize), span("codes", codes, rows * code_ld(cols)),
                         span("scales", scales, rows * scale_ld(cols)), span("codes_t", codes_t, cols * code_ld(rows)),
                         span("scales_t", scales_t, cols * scale_ld(rows))};
  for (int i = 0; i < 5; ++i)
    for (int j = i + 1; j < 5; ++j)
      if (overlap(spans[i], spans[j])) return fail(MUONH_EALIAS, "%s overlaps %s", spans[j].name, spans[i].name);
  Args a{};
  a.src = src;
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  a.codes_t = static_cast<uint8_t*>(codes_t);
  a.scales_t = static_cast<uint8_t*>(scales_t);
  a.rows = rows;
  a.cols = cols;
  a.src_ld = src_ld;
  a.tiles_c = (uint32_t)ceil_div(cols, kTile);
  a.tiles = (uint32_t)ceil_div(rows, kTile) * a.tiles_c;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == MUONH_DT_BF16) launch_forms<true>(a, s);
  else launch_forms<false>(a, s);
  return launched("fp4 quantize");
}

int muonh_fp4_dequantize(const muonh_fp4_matrix* x, void* out, int32_t out_dtype, int64_t out_ld, void* stream) {
  using namespace muonh;
  using namespace muonh::fp4;
  if (const int err = check_matrix("x", x)) return err;
  if (bad_dtype(out_dtype)) return fail(MUONH_EINVAL, "out_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", out_dtype);
  if (x->rows == 0 || x->cols == 0) return MUONH_OK;
  const rows::Mat to = {"out", out, out_dtype, out_ld};
  if (const int err = rows::check_mat(to, x->cols)) return err;
  const Span w = rows::span_of(to, x->rows, x->cols);
  if (overlap(w, span("x", x->codes, x->rows * code_ld(x->cols))) || overlap(w, span("x", x->scales, x->rows * scale_ld(x->cols))))
    return fail(MUONH_EALIAS, "out overlaps x");
  ValArgs a{};
  a.codes = static_cast<const uint8_t*>(x->codes);
  a.scales = static_cast<const uint8_t*>(x->scales);
  a.out = out;
  a.rows = x->rows;
  a.ld = code_ld(x->cols);
  a.sld = scale_ld(x->cols);
  a.out_ld = out_ld;
  a.cols = (int)x->cols;
  a.vecs = (int)ceil_div(x->cols, 8);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const int64_t blocks = ceil_div(a.rows * a.vecs, 256 * kPer);
  const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
  if (out_dtype == MUONH_DT_BF16) hipLaunchKernelGGL((k_values<__bf16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_values<float>), grid, dim3(256), 0, s, a);
  return launched("fp4 dequantize");
}

}  // extern "C"
