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

#include "fp8_codes.h"

namespace muonh {
namespace fp8 {
namespace {

using rows::launched;
using rows::misaligned;

constexpr int kThreads = 256;
constexpr int kMaxGroups = 16;

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
  const float *rstd, *weight;  // NORM: a factor for each row and for each column
};

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
//
// NORM: entry (r, c) is src's times rstd[r] times weight[c], in that order, in
// fp32: RMS norm's output, whose row sums are there already (rms_norm.hip). From bf16 the products take 64
// registers beside the 32 of the pairs, 7 or 8 more than there are: 8192 x 2048 into both forms 17.3 us, 67 MB at 3.9 TB/s.
template <bool BF, bool TILES, bool PLAIN, bool TRANS, bool NORM>
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
  constexpr bool kRows = PLAIN && !TILES, kCols = TRANS || TILES, kPairs = BF && !NORM;
  float v[kPairs ? 1 : 8][8];
  u32x4_a2 w[BF ? 8 : 1];
  uint32_t rmax[4], cmax[4];
  if constexpr (kPairs) {
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
    if constexpr (BF) {
      load_patch(static_cast<const uint16_t*>(src), g.src_ld, r0, c0, rows, cols, w);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = __uint_as_float(j & 1 ? w[i][j >> 1] & 0xffff0000u : w[i][j >> 1] << 16);
    } else {
      load_patch(static_cast<const float*>(src), g.src_ld, r0, c0, rows, cols, v);
    }
    if constexpr (NORM) {
      float by_row[8], by_col[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        by_row[i] = a.rstd[r0 + i < rows ? r0 + i : rows - 1];
        by_col[i] = a.weight[c0 + i < cols ? c0 + i : cols - 1];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = (v[i][j] * by_row[i]) * by_col[j];
      // past the matrix: zeros, whatever the factors are
      if (r0 + 8 > rows || c0 + 8 > cols)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (r0 + i >= rows || c0 + j >= cols) v[i][j] = 0.f;
    }
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
      if constexpr (kPairs) {
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
      if constexpr (kPairs) {
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

template <bool BF, bool TILES, bool NORM = false>
void launch_forms(const Args& a, bool plain, bool trans, hipStream_t s) {
  const dim3 grid((unsigned)(8 * ceil_div(a.tiles, 8))), thr(kThreads);
  if (plain && trans)
    hipLaunchKernelGGL((k_quantize<BF, TILES, true, true, NORM>), grid, thr, 0, s, a);
  else if (trans)
    hipLaunchKernelGGL((k_quantize<BF, TILES, false, true, NORM>), grid, thr, 0, s, a);
  else if constexpr (!NORM)  // the norm's own kernel writes a plain form alone
    hipLaunchKernelGGL((k_quantize<BF, TILES, true, false, false>), grid, thr, 0, s, a);
}

}  // namespace

bool tiles_fit(int64_t rows, int64_t cols) { return ceil_div(rows, kBlock) * ceil_div(cols, kBlock) <= kMaxBlocks; }

int quantize_normed(const void* src, int32_t dtype, int64_t rows, int64_t cols, int64_t src_ld, const float* rstd,
                    const float* weight, void* codes, void* scales, void* codes_t, void* scales_t, hipStream_t s) {
  const int64_t tr = ceil_div(rows, kBlock), tc = ceil_div(cols, kBlock);
  Args a{};
  a.ngroups = 1;
  a.g[0] = Group{rows, cols, src_ld, 0, (uint32_t)tc, (uint32_t)(tr * tc), 0};
  a.tiles = (uint32_t)(tr * tc);
  a.src = src;
  a.codes = codes;
  a.scales = scales;
  a.codes_t = codes_t;
  a.scales_t = scales_t;
  a.rstd = rstd;
  a.weight = weight;
  if (dtype == MUONH_DT_BF16) launch_forms<true, false, true>(a, codes != nullptr, true, s);
  else launch_forms<false, false, true>(a, codes != nullptr, true, s);
  return launched("rms norm in 8 bits");
}

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
  if (!tiles_fit(rows, cols)) return fail(MUONH_ESHAPE, "2^24 tiles of 128 x 128 or more");
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
