// Products of microscaled 4-bit matrices on gfx950 (formats and contract:
// include/muonh.h): out[i][j] = sum_k a[i][k] b[j][k], both operands read along
// their rows.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with e2m1 operands covers 4 groups of 32 along k
// and applies the E8M0 scale of each group and row itself: lane l holds 32 codes (16 bytes) of row
// l%16, group l/16, and their scale byte. A product of two codes is a multiple of 1/4 of at most 36, so the
// sum of a group is a whole number of quarters below 2^13, which the instruction adds
// exactly; sums of different groups and the accumulators are fp32 (measured on random
// codes with scales spread over 2^40: at most 2^-22.8 of sum |a b| per instruction). So, unlike 8-bit
// codes, these need not be widened to bf16: the full 4-bit rate, with sums of fp32.
//
// The kernels are those of the 8-bit products (fp8_matmul.hip, which explains their tiles,
// rings and phases), with blocks of 256 along k instead of 128: the same 128 bytes of codes per
// row, two instructions of half the time instead of one, and 8 bytes of scales per row.
#include "block_matmul.h"
#include "fp4_choice.h"

namespace muonh {
namespace fp4 {
namespace {

using namespace fp8;  // what block_matmul.h holds; constants below shadow its 8-bit ones
using fp4::ceil_div;
constexpr int kRow = kStep / 2;  // bytes of codes of a row in a block: an LDS row

typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// A fragment: 16 rows' codes of a block, lane l's the chunks l/16 and l/16 + 4 of row l%16;
// the scale bytes of these two groups, in the low 8 bits.
struct Frag {
  i32x4 lo, hi;
};
struct Scales {
  int lo, hi;
};
__device__ __forceinline__ f32x4 mma(i32x4 x, i32x4 y, f32x4 c, int sx, int sy) {
  const i32x8 wx = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
  const i32x8 wy = __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wx, wy, c, 4, 4, 0, sx, 0, sy);  // 4: e2m1
}
template <int NX, int NY>
__device__ __forceinline__ void mma_block(const Frag (&x)[NX], const Frag (&y)[NY], const Scales (&sx)[NX],
                                          const Scales (&sy)[NY], f32x4 (&acc)[NX][NY]) {
#pragma unroll
  for (int i = 0; i < NX; ++i)
#pragma unroll
    for (int j = 0; j < NY; ++j) acc[i][j] = mma(x[i].lo, y[j].lo, acc[i][j], sx[i].lo, sy[j].lo);
#pragma unroll
  for (int i = 0; i < NX; ++i)
#pragma unroll
    for (int j = 0; j < NY; ++j) acc[i][j] = mma(x[i].hi, y[j].hi, acc[i][j], sx[i].hi, sy[j].hi);
}
// A lane's two of a row's 8 scale bytes.
__device__ __forceinline__ Scales scales_of(u32x2 b, int shift) { return Scales{(int)(b[0] >> shift), (int)(b[1] >> shift)}; }

// Scales in LDS. A block's 8 bytes per row are too few for a DMA of their own: each lane of it would
// touch a cache line of its own, as many lines as the codes' DMA touches altogether. So a DMA of 4 bytes per
// lane brings 8 rows' scales of a quad, 4 blocks: 32 bytes per row, a quarter of a tile's rows
// with each block. Of LDS row r, block b of the quad lies at 8 (b ^ (r / 8 & 1)), so that the 16 rows
// of a fragment fall on different banks. Past the row's end the last 4 bytes come again (products of 8192 x 8192 x
// 8192: 300 us with two DMAs per block, 4 bytes of 64 rows each, 273 so).
constexpr int kQuadRow = 32;
// The lane's offset for LDS rows 8 i .. + 7 (i: the parity), lane l: row l / 8, dword l % 8; row: the matrix row
// from the base, quad: which 4 blocks.
__device__ __forceinline__ uint32_t quad_off(int row, int quad, int i, int lane, int sld) {
  const int dw = (((lane & 7) >> 1) ^ (i & 1)) * 2 + (lane & 1);
  return (uint32_t)row * (uint32_t)sld + (uint32_t)min(quad * kQuadRow + dw * 4, sld - 4);
}
// Row `first` + l%16's 8 bytes of block s, first a multiple of 16. The lane's two of them (scales_of) are
// shifted out where they were read, before the phase's barrier. (Reads of single bytes: lanes that want
// different bytes of one word wait for each other, 2 cycles each.)
__device__ __forceinline__ u32x2 row_scales(const char* quad, int first, int lane, int s) {
  const int r = lane & 15;
  return *reinterpret_cast<const u32x2*>(quad + (first + r) * kQuadRow + (((s & 3) ^ (r >> 3)) << 3));
}

// ---- 128 x 128 tiles: two groups of 4 waves that take the blocks in turn, a ring of 4 stages ----
constexpr int kOpStage = kT * kRow;        // 16 KB
constexpr int kStageBytes = 2 * kOpStage;  // A, then B
constexpr int kQuadBytes = 2 * kT * kQuadRow;  // a quad's scales, A's then B's
constexpr int kRing = 4;                   // of stages, and of quads

template <typename T>
__global__ __launch_bounds__(512, 2) void k_matmul4_tile(MatArgs a) {
  constexpr bool kPair = sizeof(T) == 2;
  __shared__ __attribute__((aligned(1024))) char lds[kRing * (kStageBytes + kQuadBytes)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int w4 = wave & 3, group = wave >> 2;
  int ti, tj;
  if (!map_tile(a, blockIdx.x, ti, tj)) return;
  const int nk = a.nkb;
  const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr)lds;
  const int64_t ra = (int64_t)ti * kT, rb = (int64_t)tj * kT;

  // DMA of a block by one group: waves 0, 1 fill a's 128 rows, waves 2, 3 b's;
  // 8 instructions of 8 rows, then with block s a quarter of the scales of the quad that
  // block s + 3 is in: 16 rows a wave. All of a quad have landed when its first block has.
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
  const int sld = (int)op.sld;
  const uint8_t* codes = op.codes + first * op.ld;
  const uint8_t* scales = op.scales + first * op.sld;
  const uint32_t dst = base + (is_a ? 0 : kOpStage) + (w4 & 1) * 64 * kRow;
  auto fetch_scales = [&](int s) {
    const int quad = (s + 3) >> 2, r0 = 32 * ((s + 3) & 3) + 16 * (w4 & 1);
    const uint32_t to = base + kRing * kStageBytes + (quad & (kRing - 1)) * kQuadBytes + (is_a ? 0 : kT * kQuadRow) + r0 * kQuadRow;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      dma4s(scales, quad_off((int)(row(r0 + 8 * i + (lane >> 3)) - first), quad, i, lane, sld), to + i * 8 * kQuadRow);
  };
  auto fetch_part = [&](int s, int c) {  // quarter c
    const int slot = s & (kRing - 1);
    const int64_t k = (int64_t)s * kRow;
#pragma unroll
    for (int q = 2 * c; q < 2 * c + 2; ++q) dma16s(codes + k, off[q], dst + slot * kStageBytes + q * 1024);
    if (c == 3) fetch_scales(s);
  };
  auto fetch = [&](int s) {
#pragma unroll
    for (int c = 0; c < 4; ++c) fetch_part(s, c);
  };
  constexpr int kOps = 10;  // memory operations of fetch(): 8 of codes, 2 of scales

  const int wm = w4 >> 1, wn = w4 & 1, r16 = lane & 15, g = lane >> 4;
  const int foff = r16 * kRow + ((g ^ (r16 & 7)) << 4);
  f32x4 acc[4][4];  // [b fragment][a fragment]
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{};
  auto block = [&](int s, auto more) {
    constexpr bool kMore = decltype(more)::value;
    const char* st = lds + (s & (kRing - 1)) * kStageBytes;
    const char* ss = lds + kRing * kStageBytes + ((s >> 2) & (kRing - 1)) * kQuadBytes;
    auto frag = [&](const char* p) {
      return Frag{*reinterpret_cast<const i32x4*>(p + foff), *reinterpret_cast<const i32x4*>(p + (foff ^ 64))};
    };
    Frag fa[4], fb[4];
    u32x2 ba[4], bb[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      fa[f] = frag(st + (64 * wm + 16 * f) * kRow);
      fb[f] = frag(st + kOpStage + (64 * wn + 16 * f) * kRow);
      ba[f] = row_scales(ss, 64 * wm + 16 * f, lane, s);
      bb[f] = row_scales(ss, kT + 64 * wn + 16 * f, lane, s);
      if constexpr (kMore) fetch_part(s + 3, f);
    }
    Scales sa[4], sb[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      sa[f] = scales_of(ba[f], 8 * g);
      sb[f] = scales_of(bb[f], 8 * g);
    }
    stage_barrier<(kMore ? kOps : 0)>();
    mma_block<4, 4>(fb, fa, sb, sa, acc);
    stage_barrier<63>();
  };
  // the first quad: what blocks -3, -2, -1 and 0 would bring; it is waited for with block 0, by group 1
  if (group == 0) {
    if (nk > 1) fetch(1);
    stage_barrier<63>();
  } else {
    if (nk > 0) {
      fetch_scales(-3);
      fetch_scales(-2);
      fetch_scales(-1);
      fetch(0);
    }
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

  // each wave hands half of its sums to its partner in the other group
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

// ---- 256 x 256 and 192 x 256 tiles: two groups of 4 waves, four phases per block, two stages ----
constexpr int kBigOp = kB * kRow;       // 32 KB
constexpr int kBigStage = 2 * kBigOp;   // A, then B
constexpr int kBigQuad = 2 * kB * kQuadRow;  // a quad's scales: a's rows, then b's

template <typename T, int FA, int G>
__device__ __forceinline__ void big_loop(const char* lds, uint32_t base, const uint8_t* pa, const uint8_t* pb,
                                         const uint8_t* sca, const uint8_t* scb, const uint32_t (&off)[10],
                                         int last_a, int last_b, int sld, int nk, int wave, int lane,
                                         f32x4 (&acc)[4][2 * FA]) {
  constexpr bool kPair = sizeof(T) == 2;
  const int w4 = wave & 3, r16 = lane & 15, g = lane >> 4;
  const int foff = r16 * kRow + ((g ^ (r16 & 7)) << 4);
  Frag fa[FA], fb[4];
  u32x2 ba[FA], bb[4];
  Scales sa[FA], sb[4];
  auto frag = [&](const char* p) {
    return Frag{*reinterpret_cast<const i32x4*>(p + foff), *reinterpret_cast<const i32x4*>(p + (foff ^ 64))};
  };
  auto bytes = [&](int s, int row) {
    return row_scales(lds + 2 * kBigStage + ((s >> 2) & 1) * kBigQuad, row, lane, s);
  };
  constexpr int kA1 = 2 * FA - 3;         // a's rows by a wave of group 0, 8 per instruction
  constexpr int kOps[2] = {G == 1 ? 6 : 5, kA1 + 4};  // memory operations of a part
  // Part 1 of block s, which is sent in the first phase of block s - 1, also brings a quarter of the
  // scales of the quad after block s - 1's: q = 0, 1 a's, 2, 3 b's, 8 rows a wave each. All of
  // a quad have landed when its first block has; it takes the place of the quad before block s - 1's, whose last
  // reads are over.
  auto fetch_scales = [&](int s, int q) {
    const int quad = ((s - 1) >> 2) + 1, r0 = 64 * ((s - 1) & 3), i = q & 1, r8 = 8 * i + (lane >> 3);
    const uint32_t to = base + 2 * kBigStage + (quad & 1) * kBigQuad + (r0 + 16 * w4 + 8 * i) * kQuadRow;
    if (q < 2) dma4s(sca, quad_off(min(r0 + 16 * w4 + r8, last_a), quad, i, lane, sld), to);
    else dma4s(scb, quad_off(min(r0 + b_row<kPair>(w4, r8), last_b), quad, i, lane, sld), to + kB * kQuadRow);
  };
  auto fetch = [&](int s, int part, int q) {
    const uint32_t st = base + (s & 1) * kBigStage;
    const int64_t k = (int64_t)s * kRow;
    if (G == 1) {
      if (q < 3) dma16s(pb + k, off[q], st + kBigOp + (20 + 3 * w4 + q) * 1024);
      else dma16s(pa + k, off[q], st + (3 * w4 + q - 3) * 1024);
    } else if (part == 0) {
      dma16s(pb + k, off[q], st + kBigOp + (5 * w4 + q) * 1024);
    } else {
      if (q < kA1) dma16s(pa + k, off[5 + q], st + (12 + kA1 * w4 + q) * 1024);
      else fetch_scales(s, q - kA1);
    }
  };
  auto fetch_all = [&](int s, int part) {
#pragma unroll
    for (int q = 0; q < kOps[part]; ++q) fetch(s, part, q);
  };
  auto load_a = [&](int s, int half, auto dma, int t) {
    const char* p = lds + (s & 1) * kBigStage + (2 * G + half) * 16 * FA * kRow;
#pragma unroll
    for (int f = 0; f < FA; ++f) {
      fa[f] = frag(p + 16 * f * kRow);
      ba[f] = bytes(s, (2 * G + half) * 16 * FA + 16 * f);
      if constexpr (decltype(dma)::value)
#pragma unroll
        for (int q = kOps[0] * f / FA; q < kOps[0] * (f + 1) / FA; ++q) fetch(t, 0, q);
    }
  };
  auto load_b = [&](int s, auto dma, int t) {
    const char* p = lds + (s & 1) * kBigStage + kBigOp + 64 * w4 * kRow;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      fb[f] = frag(p + 16 * f * kRow);
      bb[f] = bytes(s, kB + 64 * w4 + 16 * f);
      if constexpr (decltype(dma)::value)
#pragma unroll
        for (int q = kOps[1] * f / 4; q < kOps[1] * (f + 1) / 4; ++q) fetch(t, 1, q);
    }
  };
  auto shift_a = [&] {
#pragma unroll
    for (int f = 0; f < FA; ++f) sa[f] = scales_of(ba[f], 8 * g);
  };
  auto shift_b = [&] {
#pragma unroll
    for (int q = 0; q < 4; ++q) sb[q] = scales_of(bb[q], 8 * g);
  };
  auto mul = [&](int half) {
#pragma unroll
    for (int f = 0; f < FA; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4& c = acc[q][FA * half + f];
        c = mma(fb[q].lo, fa[f].lo, c, sb[q].lo, sa[f].lo);
      }
#pragma unroll
    for (int f = 0; f < FA; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4& c = acc[q][FA * half + f];
        c = mma(fb[q].hi, fa[f].hi, c, sb[q].hi, sa[f].hi);
      }
  };
  if (G == 0)  // the first quad: what blocks -3, -2, -1 and 0 would bring
#pragma unroll
    for (int q = 0; q < 12; ++q) fetch_scales(q / 4 - 3, q & 3);
  fetch_all(0, 0);
  if (G == 0) fetch_all(0, 1);
  if (nk > 1) {
    fetch_all(1, 0);
    stage_barrier<kOps[0]>();
  } else {
    stage_barrier<0>();
  }
  if (G == 1) stage_barrier<63>();  // phase 0
  // One block of k; LEFT: how many more blocks follow (2: at least two).
  auto block = [&](int s, auto left) {
    constexpr int kLeft = decltype(left)::value;
    constexpr std::false_type none{};
    load_b(s, std::bool_constant<G == 0 && kLeft >= 1>{}, s + 1);
    load_a(s, 0, none, 0);
    shift_b();
    shift_a();
    stage_barrier<63>();
    mul(0);
    stage_barrier<63>();
    load_a(s, 1, std::bool_constant<kLeft >= 2>{}, s + 2);
    shift_a();
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

template <typename T, int FA>
__global__ __launch_bounds__(512, 2) void k_matmul4_big(MatArgs a) {
  constexpr bool kPair = sizeof(T) == 2;
  __shared__ __attribute__((aligned(1024))) char lds[2 * kBigStage + 2 * kBigQuad];
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
    const int last_a = (int)min(a.m - 1 - ra, (int64_t)kB), last_b = (int)min(a.n - 1 - rb, (int64_t)kB);
    big_loop<T, FA, 0>(lds, base, pa, pb, scalar(a.a.scales + ra * a.a.sld), scalar(a.b.scales + rb * a.b.sld), off,
                       last_a, last_b, (int)a.a.sld, nk, wave, lane, acc);
  } else {
#pragma unroll
    for (int q = 0; q < 6; ++q) off[q] = q < 3 ? off_b(20 + 3 * w4 + q) : off_a(3 * w4 + q - 3);
    big_loop<T, FA, 1>(lds, base, pa, pb, nullptr, nullptr, off, 0, 0, 0, nk, wave, lane, acc);
  }
  store_wave<T, 2 * FA>(a, ra + 32 * FA * (wave >> 2), rb + 64 * w4, lane, acc);
}

// ---- 16 x 16 tiles: fragments straight from global memory, the waves take the blocks in turn ----
template <typename T>
__global__ __launch_bounds__(64 * kWaves) void k_matmul4_direct(MatArgs a) {
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
  const uint8_t *sa = a.a.scales + ra * a.a.sld, *sb = a.b.scales + rb * a.b.sld;
  struct Set {
    Frag a[1], b[1];
    u32x2 sa, sb;
  };
  auto frag = [](const uint8_t* p) {
    return Frag{*reinterpret_cast<const i32x4*>(p), *reinterpret_cast<const i32x4*>(p + 64)};
  };
  auto load = [&](Set& s, int kb) {
    const int64_t k = (int64_t)kb * kRow;
    s.a[0] = frag(ca + k);
    s.b[0] = frag(cb + k);
    s.sa = *reinterpret_cast<const u32x2*>(sa + (int64_t)kb * 8);
    s.sb = *reinterpret_cast<const u32x2*>(sb + (int64_t)kb * 8);
  };
  f32x4 acc[1][1] = {{f32x4{}}};
  auto mul = [&](const Set& s) {
    const Scales ea[1] = {scales_of(s.sa, 8 * g)}, eb[1] = {scales_of(s.sb, 8 * g)};
    mma_block<1, 1>(s.b, s.a, eb, ea, acc);
  };
  int kb = wave;
  Set s0, s1;
  if (kb < kb1) load(s0, kb);
  for (; kb + kWaves < kb1; kb += 2 * kWaves) {
    load(s1, kb + kWaves);
    mul(s0);
    if (kb + 2 * kWaves < kb1) load(s0, kb + 2 * kWaves);
    mul(s1);
  }
  if (kb < kb1) mul(s0);
  join_waves<T, 1, 1>(a, 0, i0, j0, red, 64, acc);
}

// ---- 64 x 64 tiles: an LDS stage per wave, the waves share out the blocks ----
constexpr int kSmallOp = kS * kRow;                      // 8 KB
constexpr int kSmallStage = 2 * kSmallOp + 2 * kS * kQuadRow;  // both operands, then a quad's scales

template <typename T>
__global__ __launch_bounds__(64 * kWaves, 2) void k_matmul4_small(MatArgs a) {
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
  auto row_a = [&](int r) { return min(i0 + r, a.m - 1) - i0; };
  auto row_b = [&](int r) { return min(j0 + b_row<kPair>(r >> 4, r & 15), a.n - 1) - j0; };
  uint32_t off[16];
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const int lr = 8 * (q & 7) + (lane >> 3);
    off[q] = (uint32_t)(q < 8 ? row_a(lr) : row_b(lr)) * (uint32_t)(q < 8 ? a.a.ld : a.b.ld) +
             (uint32_t)(((lane & 7) ^ (lr & 7)) << 4);
  }
  const int sld = (int)a.a.sld;
  const uint8_t *pa = a.a.codes + i0 * a.a.ld, *pb = a.b.codes + j0 * a.b.ld;
  const uint8_t *sa = a.a.scales + i0 * a.a.sld, *sb = a.b.scales + j0 * a.b.sld;
  char* st = lds + wave * kSmallStage;
  const uint32_t base = (uint32_t)(uintptr_t)(lds_ptr)lds + wave * kSmallStage;
  auto fetch = [&](int kb, bool first) {
    const int64_t k = (int64_t)kb * kRow;
#pragma unroll
    for (int q = 0; q < 16; ++q) dma16s((q < 8 ? pa : pb) + k, off[q], base + q * 1024);
    if (first || (kb & 3) == 0) {
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int r = 8 * (q & 7) + (lane >> 3);
        dma4s(q < 8 ? sa : sb, quad_off((int)(q < 8 ? row_a(r) : row_b(r)), kb >> 2, q, lane, sld),
              base + 2 * kSmallOp + q * 8 * kQuadRow);
      }
    }
  };
  const int foff = r16 * kRow + ((g ^ (r16 & 7)) << 4);
  f32x4 acc[4][4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[q][f] = f32x4{};
  // an eighth of the blocks for each wave, consecutive ones
  const int order = 2 * (wave & 3) + (wave >> 2), nk = max(kb1 - kb0, 0);
  int kb = kb0 + (int)((int64_t)order * nk >> 3);
  const int end = kb0 + (int)((int64_t)(order + 1) * nk >> 3);
  if (kb < end) fetch(kb, true);
  for (; kb < end; ++kb) {
    // this wave's block has landed; the empty asm keeps the reads below the wait
    __builtin_amdgcn_s_waitcnt(0 | (0x7 << 4) | (0xF << 8));  // vmcnt(0)
    asm volatile("" ::: "memory");
    Frag fa[4], fb[4];
    u32x2 ba[4], bb[4];
    auto frag = [&](const char* p) {
      return Frag{*reinterpret_cast<const i32x4*>(p + foff), *reinterpret_cast<const i32x4*>(p + (foff ^ 64))};
    };
    const char* ss = st + 2 * kSmallOp;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      fa[f] = frag(st + 16 * f * kRow);
      fb[f] = frag(st + kSmallOp + 16 * f * kRow);
      ba[f] = row_scales(ss, 16 * f, lane, kb);
      bb[f] = row_scales(ss, kS + 16 * f, lane, kb);
    }
    if (kb + 1 < end) {
      // the reads have retired before the stage is refilled
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(0xF | (3 << 14) | (0x7 << 4) | (0 << 8));  // lgkmcnt(0)
      asm volatile("" ::: "memory");
      fetch(kb + 1, false);
    }
    Scales ea[4], eb[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      ea[f] = scales_of(ba[f], 8 * g);
      eb[f] = scales_of(bb[f], 8 * g);
    }
    mma_block<4, 4>(fb, fa, eb, ea, acc);
  }
  join_waves<T, 4, 4>(a, split, i0, j0, reinterpret_cast<f32x4*>(lds), kSmallStage / 16, acc);
}

// ---- host side ----------------------------------------------------------------------
template <typename T>
int launch(const MatArgs& a, const Choice& c, hipStream_t s) {
  const dim3 grid((unsigned)map_grid((int64_t)a.tm * a.tn), (unsigned)a.splits), wg(64 * kWaves);
  if (c.kind == kBig) {
    if (c.em == kB) hipLaunchKernelGGL((k_matmul4_big<T, 4>), grid, wg, 0, s, a);
    else hipLaunchKernelGGL((k_matmul4_big<T, 3>), grid, wg, 0, s, a);
  } else if (c.kind == kTile) {
    hipLaunchKernelGGL((k_matmul4_tile<T>), grid, wg, 0, s, a);
  } else if (c.kind == kSmall) {
    hipLaunchKernelGGL((k_matmul4_small<T>), grid, wg, 0, s, a);
  } else {
    hipLaunchKernelGGL((k_matmul4_direct<T>), grid, wg, 0, s, a);
  }
  if (a.part)
    hipLaunchKernelGGL((k_matmul_join<T>), dim3((unsigned)ceil_div(a.m * (a.pld >> 2), 256)), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MUONH_EHIP, "fp4 matmul: %s (%d)", hipGetErrorString(e), (int)e);
  return MUONH_OK;
}

Operand operand(const muonh_fp4_matrix* x) {
  return Operand{static_cast<const uint8_t*>(x->codes), static_cast<const uint8_t*>(x->scales), x->rows,
                 fp4::code_ld(x->cols), fp4::scale_ld(x->cols), 0};
}

}  // namespace
}  // namespace fp4
}  // namespace muonh

extern "C" {

size_t muonh_fp4_matmul_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  using namespace muonh;
  if (fp8::bad_dim(m) || fp8::bad_dim(n) || fp8::bad_dim(k) || m == 0 || n == 0) return 0;
  return fp4::choose(m, n, k).ws_bytes;
}

int muonh_fp4_matmul(const muonh_fp4_matrix* a, const muonh_fp4_matrix* b, void* out, int32_t out_dtype, int64_t out_ld,
                     int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace muonh;
  namespace f4 = muonh::fp4;
  using fp8::ceil_div;
  using fp8::fail;
  using fp8::overlap;
  using fp8::Span;
  using fp8::span;
  if (const int err = f4::check_matrix("a", a)) return err;
  if (const int err = f4::check_matrix("b", b)) return err;
  if (a->cols != b->cols)
    return fail(MUONH_ESHAPE, "a has %lld columns, b %lld", (long long)a->cols, (long long)b->cols);
  if (out_dtype != MUONH_DT_FP32 && out_dtype != MUONH_DT_BF16)
    return fail(MUONH_EINVAL, "out_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", out_dtype);
  const bool bf16 = out_dtype == MUONH_DT_BF16;
  const int64_t m = a->rows, n = b->rows, k = a->cols;
  if (out_ld < n || out_ld > (1LL << 36))
    return fail(MUONH_EINVAL, "out_ld=%lld out of [n=%lld, 2^36]", (long long)out_ld, (long long)n);
  if (m == 0 || n == 0) return MUONH_OK;
  if (!out) return fail(MUONH_EINVAL, "out is NULL");
  const int esize = bf16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(out) & (uintptr_t)(esize - 1))
    return fail(MUONH_EINVAL, "out is not aligned to its type");
  if (ceil_div(m, fp8::kT) * ceil_div(n, fp8::kT) > fp8::kMaxTiles)
    return fail(MUONH_ESHAPE, "2^21 output tiles of 128 x 128 or more");
  const fp8::Choice c = f4::choose(m, n, k);
  if (c.ws_bytes) {
    if (!workspace) return fail(MUONH_EWORKSPACE, "workspace is NULL, the product needs %zu bytes", c.ws_bytes);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
      return fail(MUONH_EWORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < c.ws_bytes)
      return fail(MUONH_EWORKSPACE, "workspace has %zu bytes, the product needs %zu", workspace_bytes, c.ws_bytes);
  }
  const Span written[2] = {span("out", out, ((m - 1) * out_ld + n) * esize),
                           span("workspace", c.ws_bytes ? workspace : nullptr, (int64_t)c.ws_bytes)};
  const Span read[4] = {span("a's codes", a->codes, m * f4::code_ld(k)), span("a's scales", a->scales, m * f4::scale_ld(k)),
                        span("b's codes", b->codes, n * f4::code_ld(k)), span("b's scales", b->scales, n * f4::scale_ld(k))};
  if (overlap(written[0], written[1])) return fail(MUONH_EALIAS, "out overlaps the workspace");
  for (const Span& w : written)
    for (const Span& r : read)
      if (overlap(w, r)) return fail(MUONH_EALIAS, "%s overlaps %s", w.name, r.name);

  fp8::MatArgs x{};
  x.a = f4::operand(a);
  x.b = f4::operand(b);
  x.m = m;
  x.n = n;
  x.nkb = (int)ceil_div(k, f4::kStep);
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
  return bf16 ? f4::launch<__bf16>(x, c, s) : f4::launch<float>(x, c, s);
}

}  // extern "C"
