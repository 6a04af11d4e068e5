// Which kernel multiplies block-scaled 8-bit matrices (fp8_matmul.hip): host code
// only.
#pragma once

#include <algorithm>
#include <cmath>

#include "fp8_internal.h"

namespace muonh {
namespace fp8 {

constexpr int kS = 64, kT = 128, kB = 256;  // tile edges
// 32-bit offsets from a tile's first row: 256 rows of less than 2^23 bytes
constexpr int64_t kMaxTileLd = 1 << 23;
constexpr int64_t kCUs = 256;
// Output tiles of 128 x 128. Every kernel runs a tile on 512 threads, and a launch
// has fewer than 2^32: at most kMaxLaunchTiles tiles, whose number is rounded
// up to a multiple of 8. Tiles of 64 x 64 are at most 4 times as many as those of
// 128 x 128, which stays below that; tiles of 16 x 16 may be 64 times as many, and
// are taken only where they fit.
constexpr int64_t kMaxTiles = (1 << 21) - 8;
constexpr int64_t kMaxLaunchTiles = (1 << 23) - 8;
static_assert(4 * kMaxTiles <= kMaxLaunchTiles, "64 x 64 tiles always fit");

enum Kind { kDirect, kSmall, kTile, kBig };
struct Choice {
  Kind kind;
  int em, en;  // tile rows and columns
  int splits, per;
  size_t ws_bytes;
};

// Estimated time in us of a kernel on `tiles` tiles of nkb blocks: a launch,
// then rounds of one tile per CU, each a fixed part (first loads, last stores)
// and a part per block, which is less where a round leaves CUs idle (power,
// cache bandwidth). Fitted to times of 130 random products up to 12288 x 8192 x
// 12288 on the 8-bit path and, widened, with fp32 results: off by 6 (64-tiles) to
// 14 % (256-tiles). On 132 others of these sizes the kernel taken is on average
// as fast as the best of its kind (8-bit path), 1.3 and 1.1 % slower (widened,
// bf16 and fp32 results) and 1.3 and 0.7 % where it adds to them, which the
// estimate does not count; 27 % at worst (10213 x 440 x 94 added to bf16: 15.2
// us with 192 x 256 tiles, 11.9 with 128).
struct Cost {
  double fixed, block;
};
inline double estimate(const Cost& c, int64_t tiles, double nkb) {
  const int64_t part = tiles % kCUs;
  double t = 1.5 + (double)(tiles / kCUs) * (c.fixed + c.block * nkb);
  if (part) t += c.fixed + c.block * nkb * (0.6 + 0.4 * std::sqrt((double)part / (double)kCUs));
  return t;
}

// The kernel for a product: the cheapest by the estimate. Examples (measured
// us, tiles of 16, 64, 128, 192 x 256, 256). Widened, bf16 results:
// 1x6144x2048: 5.5, 7.5, 15, 32, 41; 512x2048x2048: 39, 8.3, 15, 32, 42;
// 1024x4096x4096: -, 47, 33, 61, 78; 6144x2048x8192: -, 204, 155, 133, 151;
// 8192x6144x2048: -, 295, 182, 171, 143. 8-bit path: 1x6144x2048: 5.4, 6.6, -, -,
// 21; 512x2048x2048: 39, 7.7, 11, -, 24; 1024x4096x4096: -, 37, 21, -, 43;
// 6144x2048x8192: -, 192, 107, 78, 81; 8192x6144x2048: -, -, 122, 106, 90.
inline Choice choose(int64_t m, int64_t n, int64_t k, bool wide) {
  const int64_t nkb = ceil_div(k, kBlock);
  auto tiles = [&](int64_t e) { return ceil_div(m, e) * ceil_div(n, e); };
  Choice c{kSmall, kS, kS, 1, (int)nkb, 0};
  if (m == 0 || n == 0) return c;
  if (nkb == 0) return Choice{kTile, kT, kT, 1, 0, 0};  // zeros; that kernel's loop may be empty
  const Cost small = wide ? Cost{3.1, 0.261} : Cost{2.7, 0.204};
  double best = 0;
  // 64 x 64, the k blocks split over up to 16 workgroups where tiles are few:
  // a second launch joins the partial sums
  for (int s = 1; s <= 16 && (s == 1 || (s * tiles(kS) <= kCUs && nkb >= 8 * s)); s *= 2) {
    const double t = estimate(small, s * tiles(kS), (double)nkb / s) + (s > 1 ? 2.5 + 2e-6 * s * m * n : 0.0);
    if (s > 1 && t >= best) continue;
    best = t;
    c.per = (int)ceil_div(nkb, s);
    c.splits = s == 1 ? 1 : (int)ceil_div(nkb, c.per);
  }
  // 16 x 16 tiles, all at once: a floor of latency per block, then the rate
  // at which the caches deliver both operands' rows, which are up to 32 a tile
  // and 17 for a single token
  const double rows = 1.0 + (double)std::min<int64_t>(std::min(m, n), 16) / 24.0;
  const double t16 = 2.8 + (double)nkb * rows * std::max(0.08, 5e-4 * (double)tiles(16));
  if (t16 < best && tiles(16) <= kMaxLaunchTiles) {
    best = t16;
    c = Choice{kDirect, 16, 16, 1, (int)nkb, 0};
  }
  if (code_ld(k) < kMaxTileLd) {
    auto take = [&](Kind kind, int em, int en, const Cost& cost) {
      const double t = estimate(cost, ceil_div(m, em) * ceil_div(n, en), (double)nkb);
      if (t >= best) return;
      best = t;
      c = Choice{kind, em, en, 1, (int)nkb, 0};
    };
    take(kTile, kT, kT, wide ? Cost{4.6, 0.831} : Cost{3.6, 0.503});
    take(kBig, kB, kB, wide ? Cost{8.9, 2.91} : Cost{7.0, 1.39});
    take(kBig, kB - 64, kB, wide ? Cost{7.4, 2.2} : Cost{5.5, 1.15});
  }
  if (c.splits > 1) c.ws_bytes = (size_t)c.splits * m * (ceil_div(n, 4) * 4) * sizeof(float);
  return c;
}

}  // namespace fp8
}  // namespace muonh
