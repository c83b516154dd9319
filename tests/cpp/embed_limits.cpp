// What rs_embed_workspace answers for tables of any size, without a device: a
// plan object that holds one ROWS tensor and nothing else. Reads lines
// "rows cols n_ids" on stdin and prints status and bytes for each. Link with
// librs_hip.so.
#include "rs_internal.h"

#include <cstdio>

int main() {
  long rows, cols, n_ids;
  while (std::scanf("%ld %ld %ld", &rows, &cols, &n_ids) == 3) {
    rs_plan p;
    rs::Tensor t{};
    t.rows = rows;
    t.cols = cols;
    t.n = rows * cols;
    t.g = cols;
    t.kind = RS_ROWS;
    p.n = 1;
    p.t.push_back(t);
    int64_t bytes = -1;
    const int status = rs_embed_workspace(&p, 0, n_ids, &bytes);
    std::printf("%d %ld\n", status, static_cast<long>(bytes));
  }
  return 0;
}
