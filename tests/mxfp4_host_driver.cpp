// Choice of kernels of the microscaled 4-bit path, asked line by line (CPU only):
//   dense T N D             -> "rows R X8 WAVES", "tile 64" or "tile 256"
//   grouped N D SEGMENTS ROWS MOST GLU -> "rows X8 WAVES", "tile 64" or "tile 256"
#include <cstdio>
#include <cstring>

#include "qmm_mx4.h"

int main() {
  char line[256];
  while (std::fgets(line, sizeof line, stdin)) {
    qmm::Mx4GemmArgs a{};
    long t = 0;
    int glu = 0;
    if (std::sscanf(line, "dense %ld %d %d", &t, &a.n, &a.d) == 3) {
      a.t = t;
    } else if (std::sscanf(line, "grouped %d %d %d %d %d %d", &a.n, &a.d, &a.n_seg, &a.m_total, &a.max_seg_rows, &glu) == 6) {
      a.t = a.m_total;
      a.glu = glu != 0;
    } else {
      return 1;
    }
    const qmm::MxKernel k = qmm::mx4_kernel(a);
    if (k != qmm::MxKernel::kRows) {
      std::printf("tile %d\n", k == qmm::MxKernel::kTile64 ? 64 : 256);
    } else if (a.n_seg == 0) {
      const qmm::Mx4RowsShape p = qmm::mx4_rows_shape(a.t, a.n, a.d);
      std::printf("rows %d %d %d\n", p.r, p.x8, qmm::mx4_rows_waves(p.r, p.x8));
    } else {
      const qmm::Mx4GroupedShape p = qmm::mx4_grouped_shape(a);
      std::printf("rows %d %d\n", p.x8, p.waves);
    }
  }
  return 0;
}
