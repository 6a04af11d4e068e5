// Reads "n cols" lines and prints how the library takes the embedding gradient of n tokens
// apart: lanes to a row (0: one launch for few tokens), slabs, tokens of a chunk, chunks,
// waves of k_join, workspace bytes.
#include <cstdio>

#include "embedding_plan.h"

namespace muonh {
int set_error(int code, const char*) { return code; }
}  // namespace muonh

int main() {
  using namespace muonh::embed;
  long long n, cols;
  while (std::scanf("%lld %lld", &n, &cols) == 2) {
    const Plan p = plan_of(n, cols);
    std::printf("%d %d %d %d %d %zu\n", p.lpr, p.slabs, p.chunk, p.chunks, join_waves(p), p.bytes);
  }
  return 0;
}
