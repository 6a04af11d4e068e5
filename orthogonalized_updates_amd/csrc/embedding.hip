// Embedding lookup with scaling and its gradient on gfx950 (contract:
// include/muonh.h; the table is the largest of the parameters that the AdamW step
// updates, model card "Puro", section "Training").
//
//   out[t] = scale * table[ids[t]];   G[v] (+)= scale * sum of dy[t] over ids[t] = v
//
// Both are bound by memory. The gradient brings a row's tokens together, in their order, so
// that a row of G is read and written once, by whom is known, and its sum has a fixed
// order: no atomics, the same bits every time.
#include <algorithm>

#include "embedding_plan.h"
#include "rows.h"

namespace muonh {
namespace embed {
namespace {

using fp8::overlap;
using namespace rows;

constexpr int kMaxGrid = 1 << 20;

struct Ids {
  const void* p;
  int wide;  // int64, else int32
  int64_t first, rows;
};
// The row of token t's id; `rows` for an id that is no row.
__device__ __forceinline__ uint32_t row_of(const Ids& ids, int64_t t) {
  const int64_t id = ids.wide ? static_cast<const int64_t*>(ids.p)[t] : (int64_t) static_cast<const int32_t*>(ids.p)[t];
  // as unsigned, so that ids below `first` are past the end too; first >= 0, so only from a negative id may
  // the difference pass 2^64
  const uint64_t r = (uint64_t)id - (uint64_t)ids.first;
  return id >= 0 && r < (uint64_t)ids.rows ? (uint32_t)r : (uint32_t)ids.rows;
}

// The rows of tokens t, t + step, ... (N of them; `rows` from n on), whose loads run together.
template <int N>
__device__ __forceinline__ void rows_of(const Ids& ids, int t, int step, int n, uint32_t (&r)[N]) {
  int64_t id[N];
  if (ids.wide) {
#pragma unroll
    for (int k = 0; k < N; ++k) id[k] = static_cast<const int64_t*>(ids.p)[min(t + k * step, n - 1)];
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) id[k] = static_cast<const int32_t*>(ids.p)[min(t + k * step, n - 1)];
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint64_t v = (uint64_t)id[k] - (uint64_t)ids.first;
    r[k] = t + k * step < n && id[k] >= 0 && v < (uint64_t)ids.rows ? (uint32_t)v : (uint32_t)ids.rows;
  }
}

// ---- lookup -------------------------------------------------------------------
struct LookArgs {
  Ids ids;
  const void* table;
  void* out;
  int64_t n, table_ld, out_ld;
  int cols, vecs;
  float scale;
};

// A thread takes kPer vectors of 8 entries, one after the other in the list of
// all tokens' vectors in the workgroup's stretch of it; their loads run together.
constexpr int kPer = 4;
template <typename TT, typename TO>
__global__ __launch_bounds__(256) void k_lookup(LookArgs a) {
  const uint64_t total = (uint64_t)a.n * (uint32_t)a.vecs;
  const uint64_t stretch = (uint64_t)gridDim.x * (256 * kPer);
  for (uint64_t base = (uint64_t)blockIdx.x * (256 * kPer); base < total; base += stretch) {
    const uint64_t t0 = base / (uint32_t)a.vecs;
    const uint32_t rest = (uint32_t)(base - t0 * (uint32_t)a.vecs);  // of the first vector in its row
    int64_t t[kPer];
    int c[kPer];
    uint32_t r[kPer];
    Raw<TT> raw[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const uint32_t i = rest + k * 256 + threadIdx.x, q = i / (uint32_t)a.vecs;
      t[k] = (int64_t)t0 + q;
      c[k] = (int)(i - q * (uint32_t)a.vecs) * 8;
      r[k] = t[k] < a.n ? row_of(a.ids, t[k]) : (uint32_t)a.ids.rows;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const bool found = r[k] < (uint32_t)a.ids.rows;
      const TT* p = static_cast<const TT*>(a.table) + (found ? (int64_t)r[k] * a.table_ld : 0) + c[k];
      if (c[k] + 8 <= a.cols) raw[k].load(p);
      else raw[k].load(p, a.cols - c[k]);
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (t[k] >= a.n) continue;
      const bool found = r[k] < (uint32_t)a.ids.rows;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = found ? raw[k].at(j) * a.scale : 0.f;
      store8(static_cast<TO*>(a.out) + t[k] * a.out_ld + c[k], v, a.cols - c[k]);
    }
  }
}

// ---- the gradient of few tokens ------------------------------------------------------
// Up to kFewMax tokens, in one launch (777 tokens into 5003 x 1001 from zero: 9 us, of which the
// clearing is 5; ordered, summed and joined in three launches 19 and the time between them): a workgroup to each token and 512 columns,
// which does nothing unless its token is the first of its row, and else sums the row's tokens in their order:
// up to 8 of them by one wave, more by 4, a quarter each, joined in order. Where G starts
// at zero, the first `clearing` workgroups clear the rows that do not occur.
struct FewArgs {
  Ids ids;
  const void* dy;
  float* g;
  int64_t dy_ld, g_ld;
  int n, cols, slabs, clearing, accumulate;
  float scale;
};

// Zeros in the rows that no token has, in stretches of kStretch rows: flags in LDS, then
// the lanes' rows, as many lanes to a row as it has vectors of 4, up to 64.
constexpr int kStretch = 512;
__device__ __forceinline__ void clear_others(const FewArgs& a, int64_t block, int64_t blocks, uint32_t* flags) {
  const int vecs = (a.cols + 3) >> 2;
  const int lanes = vecs >= 64 ? 64 : vecs > 1 ? 1 << (32 - __builtin_clz((unsigned)vecs - 1)) : 1;
  const int at = threadIdx.x & (lanes - 1), first = threadIdx.x / lanes, step = 256 / lanes;
  // equal stretches, so that all workgroups have one where rows are few
  const int64_t per = min((int64_t)kStretch, max((int64_t)1, ceil_div(a.ids.rows, blocks)));
  for (int64_t r0 = block * per; r0 < a.ids.rows; r0 += blocks * per) {
    const int count = (int)min(per, a.ids.rows - r0);
    __syncthreads();
    for (int i = threadIdx.x; i < kStretch / 32; i += 256) flags[i] = 0;
    __syncthreads();
    uint32_t occur[kFewMax / 256];
    rows_of<kFewMax / 256>(a.ids, threadIdx.x, 256, a.n, occur);
#pragma unroll
    for (int k = 0; k < kFewMax / 256; ++k) {
      const int64_t r = (int64_t)occur[k] - r0;
      if (r >= 0 && r < count) atomicOr(&flags[r >> 5], 1u << (r & 31));
    }
    __syncthreads();
    for (int r = first; r < count; r += step) {
      if (flags[r >> 5] >> (r & 31) & 1) continue;
      // stores of 16 bytes at multiples of 16: single floats before the first and after the last
      float* p = a.g + (r0 + r) * a.g_ld;
      const int head = min((int)((0 - (reinterpret_cast<uintptr_t>(p) >> 2)) & 3), a.cols);
      const int body = (a.cols - head) >> 2;
      for (int v = at; v < body; v += lanes) *reinterpret_cast<f32x4*>(p + head + 4 * v) = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int j = at; j < a.cols - 4 * body; j += lanes) p[j < head ? j : 4 * body + j] = 0.f;
    }
  }
}

template <typename TD>
__global__ __launch_bounds__(256) void k_few(FewArgs a) {
  __shared__ uint64_t masks[kFewMax / 64];  // the tokens of this row, t itself and after
  __shared__ uint16_t list[kFewMax];        // them in their order
  __shared__ float sums[4][64 * 8 + 8];
  static_assert(sizeof masks >= kStretch / 8, "the masks also hold the flags");
  if ((int)blockIdx.x < a.clearing) {
    clear_others(a, blockIdx.x, a.clearing, reinterpret_cast<uint32_t*>(masks));
    return;
  }
  const int b = (int)blockIdx.x - a.clearing, t = b / a.slabs, slab = b - t * a.slabs;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t mine = row_of(a.ids, t);
  if (mine >= (uint32_t)a.ids.rows) return;
  int earlier = 0;
  constexpr int kMine = kFewMax / 256;
  uint32_t theirs[kMine];
  uint64_t mask[kMine];
  rows_of<kMine>(a.ids, threadIdx.x, 256, a.n, theirs);
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int u = k * 256 + (int)threadIdx.x;
    earlier |= theirs[k] == mine && u < t;
    mask[k] = __ballot(theirs[k] == mine && u >= t);
    if (lane == 0) masks[k * 4 + wave] = mask[k];
  }
  if (__syncthreads_or(earlier)) return;
  int count = 0, before[kMine] = {};
#pragma unroll
  for (int i = 0; i < kFewMax / 64; ++i) {
    const int c = __popcll(masks[i]);
    count += c;
#pragma unroll
    for (int k = 0; k < kMine; ++k) before[k] += i < k * 4 + wave ? c : 0;
  }
#pragma unroll
  for (int k = 0; k < kMine; ++k)
    if (mask[k] >> lane & 1)
      list[before[k] + __popcll(mask[k] & ((1ull << lane) - 1))] = (uint16_t)(k * 256 + threadIdx.x);
  __syncthreads();
  const bool shared = count > 8;
  if (!shared && wave) return;
  const int lo = shared ? wave * count >> 2 : 0, hi = shared ? (wave + 1) * count >> 2 : count;
  const int col = (slab * 64 + lane) * 8, left = a.cols - col;
  float* o = a.g + (int64_t)mine * a.g_ld + col;
  Raw<float> old;
  if (a.accumulate && wave == 0) {
    if (left >= 8) old.load(o);
    else old.load(o, left);
  }
  float acc[8] = {};
  for (int i = lo; i < hi; i += 8) {
    Raw<TD> raw[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (i + k >= hi) continue;
      const int u = __builtin_amdgcn_readfirstlane(list[i + k]);
      const TD* q = static_cast<const TD*>(a.dy) + (int64_t)u * a.dy_ld + col;
      if (left >= 8) raw[k].load(q);
      else raw[k].load(q, left);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < hi)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += raw[k].at(j);
  }
  if (shared) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[wave][lane * 8 + j] = acc[j];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = acc[j] + sums[1][lane * 8 + j] + sums[2][lane * 8 + j] + sums[3][lane * 8 + j];
  }
  if (left <= 0) return;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = a.accumulate ? __builtin_fmaf(acc[j], a.scale, old.at(j)) : acc[j] * a.scale;
  store8(o, v, left);
}

// ---- tokens in the order of their rows ---------------------------------------------
// Zeros over rows x cols floats, ld apart, by blocks `block` of `blocks`.
struct FillArgs {
  float* p;
  int64_t rows, cols, ld;
};
__device__ __forceinline__ void fill(const FillArgs& f, int64_t block, int64_t blocks) {
  const int64_t vecs = (f.cols + 3) >> 2, step = blocks * blockDim.x;
  const float zero[4] = {};
  for (int64_t i = block * blockDim.x + threadIdx.x; i < f.rows * vecs; i += step) {
    const int64_t r = f.rows == 1 ? 0 : i / vecs, c = (i - r * vecs) * 4;
    float* p = f.p + r * f.ld + c;
    if (c + 4 <= f.cols) *reinterpret_cast<f32x4_a4*>(p) = f32x4{0.f, 0.f, 0.f, 0.f};
    else
      for (int j = 0; c + j < f.cols; ++j) p[j] = zero[j];
  }
}
__global__ __launch_bounds__(1024) void k_fill(FillArgs f) { fill(f, blockIdx.x, gridDim.x); }

struct Sorted {
  uint32_t *key, *tok;  // rows, equal ones together, and whose they are, ascending for each
};

// Up to kOrderMax tokens, in one launch: a workgroup to each of 256 buckets of rows reads all ids, takes
// its own and counts those of the buckets before, which is where its part of the order begins. A row's
// bucket is the high byte of row * kMul mod 2^24, which spreads neighbouring and evenly spaced rows over all of
// them, and the product's other 16 bits name the row in its bucket. Entries of these 16 bits and
// the token are all different, and their order is the tokens' within a row. The workgroups past the first
// 256 fill G with zeros.
//
// A frequent row may leave more entries than the kCounted that are sorted by counting the smaller ones: up to kFrequent
// times the row of the first entry is set apart. What then is still too much is sorted bit by bit.
//
// 4096, 8192, 16384, 32768 tokens of 151936 rows: 5.3, 7.0, 12, 18.5 us, most of it the ids' way to
// all workgroups (n^2 comparisons 6.8, 10.4, 27.8 up to 16384; the passes below 52, 62, 64, launches apart).
// 8192 tokens of different rows in one bucket, the worst there is: 54 us, 32768 of them 210. Rows in ascending order
// would save the sums 1 us of 22.7 (pages of neighbours), and buckets of neighbours fill unevenly.
constexpr int kBuckets = 256, kCounted = 256, kFrequent = 4;
constexpr uint32_t kMul = 0x9e3779, kInv = 0xb382c9, kNoRow = 1u << 24;
static_assert((kMul * kInv & 0xffffffu) == 1, "rows from their products");
static_assert(MUONH_MAX_FP8_DIM <= 1 << 24 && kOrderMax <= 1 << 16, "rows of 24 bits, tokens of 16");

// K: tokens per thread.
template <int K>
__global__ __launch_bounds__(1024) void k_order(Ids ids, int n, Sorted out, FillArgs f) {
  __shared__ __attribute__((aligned(16))) uint32_t list[1024 * K], sums[2][16];
  if ((int)blockIdx.x >= kBuckets) {
    fill(f, (int64_t)blockIdx.x - kBuckets, (int64_t)gridDim.x - kBuckets);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t bucket = blockIdx.x;
  const uint64_t lower = (1ull << lane) - 1;
  auto total = [&](int which) {  // over the waves
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += sums[which][w];
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)s);
  };
  auto before = [&](int which) {  // over the waves before this one
    uint32_t s = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += w < wave ? sums[which][w] : 0;
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)s);
  };

  int m, begin;
  {
    const int per = (int)ceil_div(n, 1024) * 64, t0 = wave * per, end = min(t0 + per, n);
    uint32_t h[K];
    int own = 0, below = 0;
    constexpr int kStep = K < 8 ? K : 8;
#pragma unroll
    for (int k0 = 0; k0 < K; k0 += kStep) {
      uint32_t r[kStep];
      rows_of<kStep>(ids, t0 + k0 * 64 + lane, 64, end, r);
#pragma unroll
      for (int k = 0; k < kStep; ++k) {
        const uint32_t v = r[k] < (uint32_t)ids.rows ? r[k] * kMul & (kNoRow - 1) : kNoRow;
        h[k0 + k] = v;
        own += __popcll(__ballot(v >> 16 == bucket));
        below += __popcll(__ballot(v >> 16 < bucket));
      }
    }
    if (lane == 0) {
      sums[0][wave] = (uint32_t)own;
      sums[1][wave] = (uint32_t)below;
    }
    __syncthreads();
    m = (int)total(0);
    begin = (int)total(1);
    int at = (int)before(0);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool is = h[k] >> 16 == bucket;
      const uint64_t mask = __ballot(is);
      if (is) list[at + __popcll(mask & lower)] = h[k] << 16 | (uint32_t)(t0 + k * 64 + lane);
      at += __popcll(mask);
    }
    __syncthreads();
  }

  // The first `count` entries in two parts, each in its old order; returns how many the first has.
  auto split = [&](int count, auto second) -> int {
    const int per = (int)ceil_div(count, 1024) * 64, i0 = wave * per + lane;
    uint32_t e[K];
    uint64_t masks[2];
    uint32_t firsts = 0, seconds = 0;
    auto part = [&](int k) {
      const bool live = i0 + k * 64 < count, b = second(e[k]);
      masks[0] = __ballot(live && !b);
      masks[1] = __ballot(live && b);
      return b;
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k * 64 >= per) continue;
      e[k] = list[min(i0 + k * 64, count - 1)];
      part(k);
      firsts += __popcll(masks[0]);
      seconds += __popcll(masks[1]);
    }
    if (lane == 0) {
      sums[0][wave] = firsts;
      sums[1][wave] = seconds;
    }
    __syncthreads();
    const int middle = (int)total(0);
    int at[2] = {(int)before(0), middle + (int)before(1)};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k * 64 >= per) continue;
      const bool b = part(k);
      if (i0 + k * 64 < count) list[b ? at[1] + __popcll(masks[1] & lower) : at[0] + __popcll(masks[0] & lower)] = e[k];
      at[0] += __popcll(masks[0]);
      at[1] += __popcll(masks[1]);
    }
    __syncthreads();
    return middle;
  };
  int rest = m;
  for (int i = 0; i < kFrequent && rest > kCounted; ++i) {
    const uint32_t frequent = list[0] >> 16;
    rest = split(rest, [&](uint32_t e) { return e >> 16 == frequent; });
  }
  if (rest > kCounted) {
    for (int b = 16; b < 32; ++b) split(rest, [&](uint32_t e) { return (e >> b & 1) != 0; });
  } else {  // 4 lanes an entry, each a quarter of the others
    static_assert(4 * kCounted == 1024, "a turn");
    const int mine = tid >> 2;
    const uint32_t e = list[min(mine, max(rest - 1, 0))];
    int place = 0;
#pragma unroll 4
    for (int i = 4 * (tid & 3); i < rest; i += 16) {
      const u32x4 other = *reinterpret_cast<const u32x4*>(list + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) place += other[j] < e && i + j < rest ? 1 : 0;
    }
    place += __builtin_amdgcn_mov_dpp(place, 0xB1, 0xF, 0xF, false);  // quad [1,0,3,2]
    place += __builtin_amdgcn_mov_dpp(place, 0x4E, 0xF, 0xF, false);  // quad [2,3,0,1]
    __syncthreads();
    if ((tid & 3) == 0 && mine < rest) list[place] = e;
    __syncthreads();
  }
  for (int i = tid; i < m; i += 1024) {
    const uint32_t e = list[i];
    out.key[begin + i] = (bucket << 16 | e >> 16) * kInv & (kNoRow - 1);
    out.tok[begin + i] = e & 0xffffu;
  }
  if (bucket == kBuckets - 1)  // ids that are no row
    for (int i = begin + m + tid; i < n; i += 1024) {
      out.key[i] = (uint32_t)ids.rows;
      out.tok[i] = 0;
    }
}

// More tokens: by 8 bits of the row at a time, from the lowest. A pass counts
// each tile's digits, sums the counts up over digits and tiles, and moves the tokens. 40000, 65536, 131072 tokens
// of 151936 rows, three passes: 62, 64, 66 us (sums of counts 14, 14, 22), of calls of 180, 226, 357 with 2048 columns.
struct PassArgs {
  Ids ids;
  Sorted in, out;  // in.key == nullptr: the ids themselves
  uint32_t* counts;  // [digit][tile]
  int n, tiles, shift;
};
__device__ __forceinline__ uint32_t key_at(const PassArgs& a, int i) { return a.in.key ? a.in.key[i] : row_of(a.ids, i); }

__global__ __launch_bounds__(256) void k_digits(PassArgs a) {
  __shared__ uint32_t hist[kDigits];
  hist[threadIdx.x] = 0;
  __syncthreads();
  const int lo = (int)blockIdx.x * kTile, hi = min(lo + kTile, a.n);
  for (int i = lo + threadIdx.x; i < hi; i += 256) atomicAdd(&hist[key_at(a, i) >> a.shift & 255], 1u);
  __syncthreads();
  a.counts[(int64_t)threadIdx.x * a.tiles + blockIdx.x] = hist[threadIdx.x];
}

// counts[i] <- the sum of those before it; one workgroup, 4096 at a time.
__global__ __launch_bounds__(1024) void k_sum_up(uint32_t* counts, int total) {
  __shared__ uint32_t part[2][1024];
  uint32_t before = 0;
  for (int base = 0; base < total; base += 4096) {
    const int i = base + threadIdx.x * 4;
    uint32_t v[4], s = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = i + k < total ? counts[i + k] : 0;
      s += v[k];
    }
    int cur = 0;
    part[0][threadIdx.x] = s;
    __syncthreads();
    for (int d = 1; d < 1024; d <<= 1) {
      part[cur ^ 1][threadIdx.x] = part[cur][threadIdx.x] + ((int)threadIdx.x >= d ? part[cur][threadIdx.x - d] : 0);
      cur ^= 1;
      __syncthreads();
    }
    uint32_t at = before + part[cur][threadIdx.x] - s;
    before += part[cur][1023];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i + k < total) counts[i + k] = at;
      at += v[k];
    }
    __syncthreads();
  }
}

// Each of the 4 waves takes a quarter of the tile, 64 tokens at a time in their
// order; those with equal digits find each other by ballots.
__global__ __launch_bounds__(256) void k_move(PassArgs a) {
  __shared__ uint32_t at[4][kDigits];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int kQuarter = kTile / 4;
  const int lo = (int)blockIdx.x * kTile + wave * kQuarter;
#pragma unroll
  for (int w = 0; w < 4; ++w) at[w][threadIdx.x] = 0;
  __syncthreads();
  uint32_t key[kQuarter / 64];
#pragma unroll
  for (int k = 0; k < kQuarter / 64; ++k) {
    const int i = lo + k * 64 + lane;
    key[k] = i < a.n ? key_at(a, i) : 0;
    if (i < a.n) atomicAdd(&at[wave][key[k] >> a.shift & 255], 1u);
  }
  __syncthreads();
  {  // the waves' counts to their first places
    uint32_t p = a.counts[(int64_t)threadIdx.x * a.tiles + blockIdx.x];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t c = at[w][threadIdx.x];
      at[w][threadIdx.x] = p;
      p += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kQuarter / 64; ++k) {
    const int i = lo + k * 64 + lane;
    const bool live = i < a.n;
    const uint32_t digit = key[k] >> a.shift & 255;
    uint64_t same = __ballot(live);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint64_t set = __ballot(digit >> b & 1);
      same &= digit >> b & 1 ? set : ~set;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    if (live) {
      const uint32_t to = at[wave][digit] + before;
      a.out.key[to] = key[k];
      a.out.tok[to] = a.in.key ? a.in.tok[i] : (uint32_t)i;
    }
    // the wave's places move on before its next 64 (its own lanes only: LDS operations of a wave are in order)
    __builtin_amdgcn_wave_barrier();
    if (live && before == 0) at[wave][digit] += (uint32_t)__popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
}

// ---- the sums -----------------------------------------------------------------------
// The ordered tokens are cut into chunks of `chunk`. The chunk in which a row's
// tokens begin sums them to the end of the next chunk and, if that is all of them,
// stores the row; what lies in later chunks is summed there (`head`) and joined to
// the first sum (`tail`) by k_join. So most rows are stored at once, and a frequent token's
// sum is shared out. 8192 tokens, 4000 different ones, added to 151936 x 2048 from bf16, 99 MB: 22.7 us where these are
// in the memory-side cache (4.4 TB/s; k_join 4.8; chunks of 16: 23.9 and 5.2), 34.4 from memory (2.9 TB/s). This form,
// with 8 tokens in flight, needs 2 vector and 41 scalar registers more than there are.
struct SumArgs {
  Sorted s;
  const void* dy;
  float* g;
  float *tail, *head;  // [chunk][cols]
  int64_t dy_ld, g_ld;
  int n, chunk, chunks, slabs, cols, accumulate;
  uint32_t rows;
  float scale;
};

// LPR lanes take a chunk's LPR * 8 columns, kRows tokens at a time: their keys and places come by one
// load, a lane each, before the rows of the tokens before them are summed.
template <typename TD, int LPR>
__global__ __launch_bounds__(256, 4) void k_sums(SumArgs a) {
  constexpr int kRows = sizeof(TD) == 2 && LPR == 64 ? 8 : 4;
  static_assert(kRows + 1 <= 16, "a group's lanes hold a turn's keys");
  int64_t g = (int64_t)blockIdx.x * (256 / LPR);
  if constexpr (LPR == 64) g += __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  else g += threadIdx.x / LPR;
  const bool mine = g < (int64_t)a.chunks * a.slabs;
  if (!mine) g = 0;
  const int c = (int)(g / a.slabs), slab = (int)(g - (int64_t)c * a.slabs);
  const int lane = threadIdx.x & 63, gl = lane & (LPR - 1);
  const int col = (slab * LPR + gl) * 8, left = a.cols - col;
  const int p0 = c * a.chunk, p1 = min(p0 + a.chunk, a.n), lim = min(p1 + a.chunk, a.n);
  const uint32_t* key = a.s.key;
  uint32_t kv, tv;  // of tokens p + gl
  auto fetch = [&](int p) {
    const int i = min(p + gl, a.n - 1);
    kv = p + gl < a.n ? key[i] : 0xffffffffu;
    tv = a.s.tok[i];
  };
  auto of = [&](uint32_t v, int i) -> uint32_t {
    if constexpr (LPR == 64) return (uint32_t)__builtin_amdgcn_readlane((int)v, i);
    else return (uint32_t)__shfl((int)v, (lane & ~(LPR - 1)) + i, 64);
  };
  fetch(p0);
  const uint32_t first = key[p0], last = key[p1 - 1];
  // first's tokens began before this chunk: in the one before, which sums them (skip), or earlier (head)
  const bool cont = p0 > 0 && key[max(p0 - 1, 0)] == first;
  const bool head = cont && p0 - a.chunk > 0 && key[max(p0 - a.chunk - 1, 0)] == first;
  const bool skip = cont && !head;
  float acc[8] = {};
  bool open = head, pending = false;
  for (int p = p0; p < lim; p += kRows) {
    uint32_t k[kRows + 1], t[kRows];
    bool valid[kRows], end[kRows], store[kRows];
    Raw<TD> raw[kRows];
    Raw<float> old[kRows];
#pragma unroll
    for (int i = 0; i <= kRows; ++i) k[i] = of(kv, i);
#pragma unroll
    for (int i = 0; i < kRows; ++i) t[i] = of(tv, i);
    fetch(p + kRows);
    bool any = false, still = open;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      valid[i] = mine && p + i < lim && k[i] < a.rows && !(skip && k[i] == first) &&
                 (p + i < p1 || (k[i] == last && !(cont && last == first)));
      end[i] = valid[i] && k[i + 1] != k[i];
      store[i] = end[i] && !still;
      if (end[i]) still = false;
      any |= valid[i];
      if (valid[i]) {
        const TD* q = static_cast<const TD*>(a.dy) + (int64_t)t[i] * a.dy_ld + col;
        if (left >= 8) raw[i].load(q);
        else raw[i].load(q, left);
        if (store[i] && a.accumulate) {
          const float* o = a.g + (int64_t)k[i] * a.g_ld + col;
          if (left >= 8) old[i].load(o);
          else old[i].load(o, left);
        }
      }
    }
    if (LPR == 64 && !any && p >= p1) break;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (!valid[i]) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += raw[i].at(j);
      pending = !end[i];
      if (!end[i]) continue;
      if (store[i]) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = a.accumulate ? __builtin_fmaf(acc[j], a.scale, old[i].at(j)) : acc[j] * a.scale;
        if (left > 0) store8(a.g + (int64_t)k[i] * a.g_ld + col, v, left);
      } else if (left > 0) {
        store8(a.head + (int64_t)c * a.cols + col, acc, left);
      }
      open = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    }
  }
  if (pending && left > 0) store8((open ? a.head : a.tail) + (int64_t)c * a.cols + col, acc, left);
}

// Rows whose tokens go on past the chunk after the one they begin in: the tail
// and the heads, each of the waves a part of them, then the parts in order. A
// workgroup to each chunk and slab; most of them have nothing to do.
template <int LPR, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void k_join(SumArgs a) {
  __shared__ float sums[WAVES][64 * 8 + 8];
  constexpr int kFlight = 8;  // sums whose loads run together
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = (int)(blockIdx.x / a.slabs), slab = (int)(blockIdx.x % a.slabs);
  const int col = (slab * LPR + (lane & (LPR - 1))) * 8, left = lane < LPR ? a.cols - col : 0;
  const uint32_t* key = a.s.key;
  auto key_of = [&](int64_t chunk) { return key[chunk * a.chunk]; };
  const uint32_t k = key[(int64_t)(c + 1) * a.chunk - 1];
  if (k >= a.rows || key_of((int64_t)c + 2) != k || (c > 0 && key[(int64_t)c * a.chunk - 1] == k)) return;
  auto load = [&](Raw<float>& t, const float* p) {
    if (left >= 8) t.load(p);
    else t.load(p, left);
  };
  float* o = a.g + (int64_t)k * a.g_ld + col;
  float acc[8] = {};
  Raw<float> old, tail;
  if (wave == 0 && left > 0) {
    load(tail, a.tail + (int64_t)c * a.cols + col);
    if (a.accumulate) load(old, o);
  }
  int heads = 0;  // chunks c + 2 .. c + 1 + heads
  for (;;) {
    const int64_t q = (int64_t)c + 2 + heads + lane;
    const uint64_t eq = __ballot(q < a.chunks && key_of(q) == k);
    const int run = ~eq ? __builtin_ctzll(~eq) : 64;
    heads += run;
    if (run < 64) break;
  }
  const int lo = (int)((int64_t)wave * heads / WAVES), hi = (int)((int64_t)(wave + 1) * heads / WAVES);
  if (left > 0) {
    const float* p = a.head + ((int64_t)c + 2) * a.cols + col;
    if (wave == 0)
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = tail.at(j);
    for (int h = lo; h < hi; h += kFlight) {
      Raw<float> t[kFlight];
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (h + i < hi) load(t[i], p + (int64_t)(h + i) * a.cols);
#pragma unroll
      for (int i = 0; i < kFlight; ++i)
        if (h + i < hi)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] += t[i].at(j);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[wave][lane * 8 + j] = acc[j];
  __syncthreads();
  if (wave || left <= 0) return;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float s = acc[j];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) s += sums[w][lane * 8 + j];
    v[j] = a.accumulate ? __builtin_fmaf(s, a.scale, old.at(j)) : s * a.scale;
  }
  store8(o, v, left);
}

// ---- host side ----------------------------------------------------------------------
int check_ids(const void* ids, int32_t id_bytes, int64_t n, int64_t rows, int64_t cols, int64_t first) {
  if (id_bytes != 4 && id_bytes != 8) return fail(MUONH_EINVAL, "id_bytes=%d is neither 4 nor 8", id_bytes);
  if (fp8::bad_dim(n)) return fail(MUONH_ESHAPE, "%lld ids out of [0, %d]", (long long)n, MUONH_MAX_FP8_DIM);
  if (fp8::bad_dim(rows) || fp8::bad_dim(cols))
    return fail(MUONH_ESHAPE, "shape %lld x %lld out of [0, %d]", (long long)rows, (long long)cols, MUONH_MAX_FP8_DIM);
  if (first < 0) return fail(MUONH_EINVAL, "first=%lld must be >= 0", (long long)first);
  if (n > 0 && cols > 0) {
    if (!ids) return fail(MUONH_EINVAL, "ids is NULL");
    if (reinterpret_cast<uintptr_t>(ids) & (uintptr_t)(id_bytes - 1))
      return fail(MUONH_EINVAL, "ids is not aligned to its type");
  }
  return MUONH_OK;
}

}  // namespace
}  // namespace embed
}  // namespace muonh

extern "C" {

int muonh_embedding(const void* ids, int32_t id_bytes, int64_t n, int64_t first, const void* table, int32_t table_dtype,
                    int64_t rows, int64_t cols, int64_t table_ld, float scale, void* out, int32_t out_dtype,
                    int64_t out_ld, void* stream) {
  using namespace muonh;
  using namespace muonh::embed;
  if (bad_dtype(table_dtype))
    return fail(MUONH_EINVAL, "table_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", table_dtype);
  if (bad_dtype(out_dtype)) return fail(MUONH_EINVAL, "out_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", out_dtype);
  if (const int err = check_ids(ids, id_bytes, n, rows, cols, first)) return err;
  if (!(scale - scale == 0.f)) return fail(MUONH_EINVAL, "scale=%g must be finite", (double)scale);
  if (n == 0 || cols == 0) return MUONH_OK;
  if (rows == 0) return fail(MUONH_ESHAPE, "a table of no rows");
  const Mat from = {"table", table, table_dtype, table_ld}, to = {"out", out, out_dtype, out_ld};
  if (const int err = check_mat(from, cols)) return err;
  if (const int err = check_mat(to, cols)) return err;
  const Span written = span_of(to, n, cols);
  if (overlap(written, span_of(from, rows, cols))) return fail(MUONH_EALIAS, "out overlaps table");
  if (overlap(written, span("ids", ids, n * id_bytes))) return fail(MUONH_EALIAS, "out overlaps ids");
  LookArgs a{};
  a.ids = Ids{ids, id_bytes == 8, first, rows};
  a.table = table;
  a.out = out;
  a.n = n;
  a.table_ld = table_ld;
  a.out_ld = out_ld;
  a.cols = (int)cols;
  a.vecs = (int)ceil_div(cols, 8);
  a.scale = scale;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)std::min<int64_t>(ceil_div(n * a.vecs, 256 * kPer), kMaxGrid));
  const bool tb = table_dtype == MUONH_DT_BF16, ob = out_dtype == MUONH_DT_BF16;
  if (tb && ob) hipLaunchKernelGGL((k_lookup<__bf16, __bf16>), grid, dim3(256), 0, s, a);
  else if (tb) hipLaunchKernelGGL((k_lookup<__bf16, float>), grid, dim3(256), 0, s, a);
  else if (ob) hipLaunchKernelGGL((k_lookup<float, __bf16>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_lookup<float, float>), grid, dim3(256), 0, s, a);
  return launched("embedding");
}

size_t muonh_embedding_backward_workspace_bytes(int64_t n, int64_t cols) {
  using namespace muonh;
  if (fp8::bad_dim(n) || fp8::bad_dim(cols) || n == 0 || cols == 0 ||
      n * cols > embed::kMaxEntries)
    return 0;
  return embed::plan_of(n, cols).bytes;
}

int muonh_embedding_backward(const void* ids, int32_t id_bytes, int64_t n, int64_t first, const void* dy, int32_t dy_dtype,
                             int64_t dy_ld, float scale, float* grad, int64_t rows, int64_t cols, int64_t grad_ld,
                             int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace muonh;
  using namespace muonh::embed;
  if (bad_dtype(dy_dtype)) return fail(MUONH_EINVAL, "dy_dtype=%d is neither MUONH_DT_FP32 nor MUONH_DT_BF16", dy_dtype);
  if (const int err = check_ids(ids, id_bytes, n, rows, cols, first)) return err;
  if (!(scale - scale == 0.f)) return fail(MUONH_EINVAL, "scale=%g must be finite", (double)scale);
  if (rows == 0 || cols == 0) return MUONH_OK;
  const Mat to = {"grad", grad, MUONH_DT_FP32, grad_ld}, from = {"dy", dy, dy_dtype, dy_ld};
  if (const int err = check_mat(to, cols)) return err;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  // whole rows without gaps are one long row of zeros
  FillArgs f = grad_ld == cols ? FillArgs{grad, 1, rows * cols, rows * cols} : FillArgs{grad, rows, cols, grad_ld};
  if (accumulate) f.rows = 0;
  const int fills = accumulate ? 0 : (int)std::min<int64_t>(ceil_div(f.rows * ceil_div(f.cols, 4), 1024), 2048);
  if (n == 0) {
    if (!fills) return MUONH_OK;
    hipLaunchKernelGGL(k_fill, dim3((unsigned)fills), dim3(1024), 0, s, f);
    return launched("embedding backward");
  }
  if (const int err = check_mat(from, cols)) return err;
  if (n * cols > kMaxEntries) return fail(MUONH_ESHAPE, "dy has more than 2^38 entries");
  const Plan p = plan_of(n, cols);
  if (p.bytes) {
    if (!workspace) return fail(MUONH_EWORKSPACE, "workspace is NULL, the call needs %zu bytes", p.bytes);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(MUONH_EWORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < p.bytes)
      return fail(MUONH_EWORKSPACE, "workspace has %zu bytes, the call needs %zu", workspace_bytes, p.bytes);
  }
  const Span read[2] = {span_of(from, n, cols), span("ids", ids, n * id_bytes)};
  const Span written[2] = {span_of(to, rows, cols), span("workspace", p.bytes ? workspace : nullptr, (int64_t)p.bytes)};
  for (const Span& w : written)
    for (const Span& r : read)
      if (overlap(w, r)) return fail(MUONH_EALIAS, "%s overlaps %s", w.name, r.name);
  if (overlap(written[0], written[1])) return fail(MUONH_EALIAS, "grad overlaps the workspace");

  const Ids which{ids, id_bytes == 8, first, rows};
  if (few(n, cols)) {
    FewArgs a{};
    a.ids = which;
    a.dy = dy;
    a.g = grad;
    a.dy_ld = dy_ld;
    a.g_ld = grad_ld;
    a.n = (int)n;
    a.cols = (int)cols;
    a.slabs = (int)ceil_div(cols, 512);
    a.accumulate = accumulate != 0;
    a.scale = scale;
    // a workgroup clears 32 KB or more, 2048 of them at most
    a.clearing = accumulate ? 0 : (int)std::min(std::min<int64_t>(ceil_div(rows * cols, 8192), rows), (int64_t)2048);
    const dim3 grid((unsigned)(a.clearing + a.n * a.slabs));
    if (dy_dtype == MUONH_DT_BF16) hipLaunchKernelGGL((k_few<__bf16>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_few<float>), grid, dim3(256), 0, s, a);
    return launched("embedding backward");
  }

  char* ws = static_cast<char*>(workspace);
  auto sorted = [&](int i) {
    return Sorted{reinterpret_cast<uint32_t*>(ws + p.key[i]), reinterpret_cast<uint32_t*>(ws + p.tok[i])};
  };
  SumArgs a{};
  if (n <= kOrderMax) {
    const dim3 grid((unsigned)(kBuckets + fills));
    auto order = [&](auto per) { hipLaunchKernelGGL((k_order<decltype(per)::value>), grid, dim3(1024), 0, s, which, (int)n, sorted(0), f); };
    if (n <= 4096) order(std::integral_constant<int, 4>{});
    else if (n <= 8192) order(std::integral_constant<int, 8>{});
    else if (n <= 16384) order(std::integral_constant<int, 16>{});
    else order(std::integral_constant<int, 32>{});
    a.s = sorted(0);
  } else {
    if (fills) hipLaunchKernelGGL(k_fill, dim3((unsigned)fills), dim3(1024), 0, s, f);
    PassArgs b{};
    b.ids = which;
    b.counts = reinterpret_cast<uint32_t*>(ws + p.counts);
    b.n = (int)n;
    b.tiles = p.tiles;
    int side = 0;
    for (b.shift = 0; b.shift == 0 || rows >> b.shift; b.shift += 8) {
      b.out = sorted(side);
      hipLaunchKernelGGL(k_digits, dim3((unsigned)p.tiles), dim3(256), 0, s, b);
      hipLaunchKernelGGL(k_sum_up, dim3(1), dim3(1024), 0, s, b.counts, kDigits * p.tiles);
      hipLaunchKernelGGL(k_move, dim3((unsigned)p.tiles), dim3(256), 0, s, b);
      b.in = b.out;
      side ^= 1;
    }
    a.s = b.in;
  }
  a.dy = dy;
  a.g = grad;
  a.tail = reinterpret_cast<float*>(ws + p.tail);
  a.head = reinterpret_cast<float*>(ws + p.head);
  a.dy_ld = dy_ld;
  a.g_ld = grad_ld;
  a.n = (int)n;
  a.chunk = p.chunk;
  a.chunks = p.chunks;
  a.slabs = p.slabs;
  a.cols = (int)cols;
  a.accumulate = accumulate != 0;
  a.rows = (uint32_t)rows;
  a.scale = scale;
  const int64_t groups = (int64_t)p.chunks * p.slabs;
  const dim3 sums((unsigned)ceil_div(groups, 256 / p.lpr));
  auto run = [&](auto type) {
    using T = decltype(type);
    if (p.lpr == 16) hipLaunchKernelGGL((k_sums<T, 16>), sums, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_sums<T, 64>), sums, dim3(256), 0, s, a);
  };
  if (dy_dtype == MUONH_DT_BF16) run(__bf16{});
  else run(float{});
  if (p.chunks > 2) {
    const dim3 join((unsigned)((p.chunks - 2) * p.slabs));
    if (p.lpr == 16) hipLaunchKernelGGL((k_join<16, 8>), join, dim3(512), 0, s, a);
    else if (join_waves(p) == 8) hipLaunchKernelGGL((k_join<64, 8>), join, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((k_join<64, 4>), join, dim3(256), 0, s, a);
  }
  return launched("embedding backward");
}

}  // extern "C"
