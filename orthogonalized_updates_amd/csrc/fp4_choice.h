// Which kernel multiplies microscaled 4-bit matrices (fp4_matmul.hip): host code only.
#pragma once

#include "fp4_internal.h"
#include "fp8_choice.h"

namespace muonh {
namespace fp4 {

using fp8::Choice;
using fp8::Cost;
using fp8::estimate;
using fp8::kBig;
using fp8::kCUs;
using fp8::kDirect;
using fp8::kSmall;
using fp8::kTile;

// As choose() of fp8_choice.h, with blocks of 256 along k and constants fitted to these kernels'
// times on 138 random products up to 12288 x 8192 x 12288 (bf16 results). On 216 others the kernel
// taken is on average 0.7 (bf16) and 0.4 % (fp32 results) slower than the best, 21 % at worst (42 x 7470 x 232:
// 5.7 us with 16-tiles, 4.8 with 64). Examples (us, tiles of 16, 64, 128, 192 x 256, 256):
// 1x6144x2048: 4.4, 5.9, 8.9, 14, 17; 512x2048x2048: 25, 6.6, 9.2, 15, 17; 1024x4096x4096: 170,
// 27, 17, 27, 31; 6144x2048x8192: -, 117, 72, 58, 66; 8192x6144x2048: -, 212, 109, 84, 69.
inline Choice choose(int64_t m, int64_t n, int64_t k) {
  using fp8::kB;
  using fp8::kMaxLaunchTiles;
  using fp8::kMaxTileLd;
  using fp8::kS;
  using fp8::kT;
  const int64_t nkb = ceil_div(k, kStep);
  auto tiles = [&](int64_t e) { return ceil_div(m, e) * ceil_div(n, e); };
  Choice c{kSmall, kS, kS, 1, (int)nkb, 0};
  if (m == 0 || n == 0) return c;
  if (nkb == 0) return Choice{kTile, kT, kT, 1, 0, 0};  // zeros; that kernel's loop may be empty
  const Cost small{2.63, 0.273};
  double best = 0;
  // 64 x 64, the k blocks split over up to 16 workgroups where tiles are few:
  // a second launch joins the partial sums
  for (int s = 1; s <= 16 && (s == 1 || (s * tiles(kS) <= kCUs && nkb >= 4 * s)); s *= 2) {
    const double t = estimate(small, s * tiles(kS), (double)nkb / s) + (s > 1 ? 2.5 + 2e-6 * s * m * n : 0.0);
    if (s > 1 && t >= best) continue;
    best = t;
    c.per = (int)ceil_div(nkb, s);
    c.splits = s == 1 ? 1 : (int)ceil_div(nkb, c.per);
  }
  const double rows = 1.0 + (double)std::min<int64_t>(std::min(m, n), 16) / 24.0;
  const double t16 = 3.38 + (double)nkb * rows * std::max(0.054, 3.77e-4 * (double)tiles(16));
  if (t16 < best && tiles(16) <= kMaxLaunchTiles) {
    best = t16;
    c = Choice{kDirect, 16, 16, 1, (int)nkb, 0};
  }
  if (code_ld(k) < kMaxTileLd) {
    auto take = [&](fp8::Kind kind, int em, int en, const Cost& cost) {
      const double t = estimate(cost, ceil_div(m, em) * ceil_div(n, en), (double)nkb);
      if (t >= best) return;
      best = t;
      c = Choice{kind, em, en, 1, (int)nkb, 0};
    };
    take(kTile, kT, kT, Cost{4.12, 0.633});
    take(kBig, kB, kB, Cost{4.34, 1.75});
    take(kBig, kB - 64, kB, Cost{4.25, 1.6});
  }
  if (c.splits > 1) c.ws_bytes = (size_t)c.splits * m * (ceil_div(n, 4) * 4) * sizeof(float);
  return c;
}

}  // namespace fp4
}  // namespace muonh
