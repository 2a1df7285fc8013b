// Host checks of the block-scaled e4m3 path's addresses, driven by
// tests/test_fp8_host.py: the functions that the kernels take them from, over
// every size at which they can leave a buffer.  Exits 0, or prints the first
// size that fails.
#include <hip/hip_runtime.h>

#include <stdio.h>
#include <string.h>

#include "qmm_fp8.h"

#define CHECK(ok, ...)                         \
  do {                                         \
    if (!(ok)) {                               \
      printf("line %d: ", __LINE__);           \
      printf(__VA_ARGS__);                     \
      printf("\n");                            \
      return 1;                                \
    }                                          \
  } while (0)

namespace {

// Tiles of `cols` columns whose waves take `step` columns each, as the tile kernels
// have them: no wave's scale row is past the ceil(n / 128) of the matrix, and a wave
// with a live column has that column's.
int scale_rows() {
  const int shapes[][2] = {{256, 64}, {128, 32}, {64, 16}};
  for (const auto& s : shapes)
    for (int n = 1; n <= 2 * 256 + 128; ++n)
      for (int n0 = 0; n0 < n; n0 += s[0])
        for (int c = n0; c < n0 + s[0]; c += s[1]) {
          const int row = qmm::fp8_scale_row(c, n);
          CHECK(row >= 0 && row < qmm::fp8_blocks(n), "n %d, columns from %d: scale row %d", n, c, row);
          for (int u = c; u < c + s[1] && u < n; ++u)
            CHECK(row == u / qmm::kFp8Block, "n %d, column %d: scale row %d", n, u, row);
        }
  return 0;
}

}  // namespace

int main(int argc, char** argv) {
  if (argc > 1 && !strcmp(argv[1], "scale_rows")) return scale_rows();
  printf("no such check\n");
  return 2;
}
