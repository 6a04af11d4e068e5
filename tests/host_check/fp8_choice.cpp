// Reads "m n k wide" lines and prints the kernel that the library takes for such
// a product: tile rows and columns, splits of k, k blocks per split, workspace
// bytes, workgroups of the launch.
#include <cstdio>

#include "fp8_choice.h"

namespace muonh {
int set_error(int code, const char*) { return code; }
}  // namespace muonh

int main() {
  using namespace muonh::fp8;
  long long m, n, k;
  int wide;
  while (std::scanf("%lld %lld %lld %d", &m, &n, &k, &wide) == 4) {
    const Choice c = choose(m, n, k, wide != 0);
    const long long tiles = (long long)(ceil_div(m, c.em) * ceil_div(n, c.en));
    std::printf("%d %d %d %d %zu %lld\n", c.em, c.en, c.splits, c.per, c.ws_bytes,
                8 * (long long)ceil_div(tiles, 8) * c.splits);
  }
  return 0;
}
