// Host-side check of the plan by which rows are brought to 4 bits (rows_plan, zi_fp4.cuh): for every width, row counts
// on both sides of the plan's border and both input types, each 16-column span of a row belongs to a thread of the
// launch.  Built and run by tests/test_fp4_plan.py; prints "plan ok <cases>" on success.
#include <cstdio>
#include <vector>

#include "zi_fp4.cuh"

using namespace zi::fp4;

int main() {
  int cases = 0, failures = 0;
  for (int bytes : {2, 4})
    for (int rows : {1, 127, 1023, 1024, 1025, 4128, 20480})
      for (int cols = 32; cols <= kRowsMaxCols; cols += 32) {
        const RowsPlan p = rows_plan(rows, cols, bytes);
        std::vector<int> taken(size_t(cols / 16), 0);
        for (int sub = 0; sub < p.tpr; ++sub)
          for (int k = 0; k < p.spans; ++k)  // as quantize_kernel walks them
            if (sub + k * p.tpr < cols / 16) ++taken[size_t(sub + k * p.tpr)];
        bool ok = p.tpr >= 8 && p.tpr <= kRowsThreads && (p.tpr & (p.tpr - 1)) == 0 &&
                  p.spans >= 1 && p.spans <= kMaxSpans;
        for (int n : taken) ok = ok && n == 1;
        if (!ok && ++failures <= 20)
          std::printf("FAIL rows %d cols %d bytes %d: %d threads x %d spans\n", rows, cols, bytes, p.tpr, p.spans);
        ++cases;
      }
  if (failures) {
    std::printf("plan FAILED %d of %d\n", failures, cases);
    return 1;
  }
  std::printf("plan ok %d\n", cases);
  return 0;
}
