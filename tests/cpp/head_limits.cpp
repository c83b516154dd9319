// What rs_head_workspace and rs_layer_norm_workspace answer for tables and rows
// of any size, without a device: a plan object that holds one ROWS tensor and
// nothing else. Reads lines "rows cols n top grad dtype piece" on stdin and prints
// status and bytes of the head's workspace, then status and bytes of layer
// norm's on rows of rows * cols values. Link with librs_hip.so.
#include "rs_internal.h"

#include <cstdio>

int main() {
  long rows, cols, n, top, piece;
  int grad, dt;
  while (std::scanf("%ld %ld %ld %ld %d %d %ld", &rows, &cols, &n, &top, &grad, &dt, &piece) == 7) {
    rs_plan p;
    rs::Tensor t{};
    t.rows = rows;
    t.cols = cols;
    t.n = rows * cols;
    t.g = cols;
    t.kind = RS_ROWS;
    p.n = 1;
    p.t.push_back(t);
    int64_t head = -1, norm = -1;
    const int status = rs_head_workspace(&p, 0, n, top, grad, dt, piece, &head);
    const int norm_status = rs_layer_norm_workspace(&p, 0, n, &norm);
    std::printf("%d %ld %d %ld\n", status, static_cast<long>(head), norm_status, static_cast<long>(norm));
  }
  return 0;
}
