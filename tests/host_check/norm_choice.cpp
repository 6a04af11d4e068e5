// Reads "rows cols" lines and prints how the library takes the RMS norm of such a matrix: lanes of a row,
// vectors each (0 0: rows of any length), workgroups, rows that a workgroup takes at a time; then the same of its
// gradient.
#include <cstdio>

#include "norm_choice.h"

namespace muonh {
int set_error(int code, const char*) { return code; }
}  // namespace muonh

int main() {
  using namespace muonh::norm;
  long long rows, cols;
  while (std::scanf("%lld %lld", &rows, &cols) == 2) {
    const Form f = forward_form(rows, cols), b = backward_form(cols);
    std::printf("%d %d %lld %d %d %d %d %d\n", f.lanes, f.vecs, (long long)forward_groups(rows, f), rows_at_once(f), b.lanes,
                b.vecs, back_groups(rows, cols), rows_at_once(b));
  }
  return 0;
}
