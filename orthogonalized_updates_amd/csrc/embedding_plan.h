// How the embedding gradient (embedding.hip) takes a call apart: which kernels, how the tokens
// are cut, where things are in the workspace. Host code only.
#pragma once

#include "fp8_internal.h"

namespace muonh {
namespace embed {

using fp8::ceil_div;

// of dy: the launches of k_sums and k_few stay below 2^32 threads
constexpr int64_t kMaxEntries = 1LL << 38;
constexpr int kFewMax = 1024;                 // tokens that k_few takes
constexpr int kOrderMax = 32768;              // and k_order
constexpr int kTile = 4096, kDigits = 256;    // tokens of a workgroup in a pass over more, its counts

struct Plan {
  int64_t n;
  int lpr, slabs, chunk, chunks, tiles;
  size_t key[2], tok[2], counts, tail, head, bytes;
};
// Whether k_few takes the call: a launch has fewer than 2^32 threads.
inline bool few(int64_t n, int64_t cols) { return n <= kFewMax && n * ceil_div(cols, 512) < (1 << 23); }
inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
inline Plan plan_of(int64_t n, int64_t cols) {
  Plan p{};
  p.n = n;
  if (few(n, cols)) return p;
  p.lpr = cols <= 128 ? 16 : 64;
  p.slabs = (int)ceil_div(cols, p.lpr * 8);
  // about 4096 waves, 16 a CU; each chunk pays for its ends
  p.chunk = 4;
  while (p.chunk < 256 && n * p.slabs * (p.lpr / 16) > (int64_t)p.chunk * 16384) p.chunk *= 2;
  p.chunks = (int)ceil_div(n, p.chunk);
  p.tiles = (int)ceil_div(n, kTile);
  const bool ordered = n <= kOrderMax;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = up256(at + bytes);
    return here;
  };
  for (int i = 0; i < (ordered ? 1 : 2); ++i) {
    p.key[i] = take((size_t)n * 4);
    p.tok[i] = take((size_t)n * 4);
  }
  p.counts = ordered ? 0 : take((size_t)kDigits * p.tiles * 4);
  p.tail = take((size_t)p.chunks * cols * 4);
  p.head = take((size_t)p.chunks * cols * 4);
  p.bytes = at;
  return p;
}

// Waves that share a row's sums in k_join. Waves that start only to stop cost as much as the sums do, and one
// workgroup to a chunk and slab has about as many of them whatever the columns are. With several slabs chunks are
// fewer, so that a frequent row has fewer sums: 4 waves; with one slab 8. k_join in us with 4 and 8 waves,
// ids as in text (the i-th word's share about 1/i) of 151936 rows and of 1208:
//   500 columns, 2000 tokens   4.0  3.9   4.9  4.0    1000 columns,  6000   5.7  6.4   7.2  6.7
//                8000          8.2  6.1  11.9  8.5                   8000   6.6  7.6   8.7  8.4
//               16000         14.8 10.4  23.0 15.2    2048 columns,  4000   4.9  7.4   6.3  8.2
//               32000         14.5 11.1  23.1 15.9                   8192   5.5  7.5   5.5  7.5
// Where one row has a quarter or half of all tokens (a padding id that is a row), 8 waves are the faster ones
// everywhere: 8192 tokens x 2048 11.8, 9.3 and 20.2, 15.7; the host does not see the ids.
inline int join_waves(const Plan& p) { return p.slabs == 1 ? 8 : 4; }

}  // namespace embed
}  // namespace muonh
