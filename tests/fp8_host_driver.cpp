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

// What a lane's copy of `bytes` from a buffer of `records` bytes may read, for each way
// in which a machine may hold the offsets against the size: the lane's offset alone,
// the sum, or the lane's against the size less the scalar offset, in 32 bits.
bool inside(uint32_t records, uint32_t voff, uint32_t soff, uint32_t bytes, uint64_t owned) {
  for (uint32_t i = 0; i < bytes; i += 4) {
    const uint64_t at = uint64_t(voff) + i, end = at + soff + 4;
    const bool reads = at + 4 <= records || end <= records || (at <= 0xFFFFFFFFu && uint32_t(at) < records - soff);
    if (reads && end > owned) return false;
  }
  return true;
}

// The few-row kernel's copies, block by block of every wave's share and the ring's depth
// past it: codes of a row (the last one), and the scales of four blocks from a share's
// first block on.
int rows_copies() {
  for (int waves = 2; waves <= 8; waves *= 2)
    for (int d = 16; d <= 128 * 40; d += 16) {
      const int nb = qmm::fp8_blocks(d);
      for (int rows = 1; rows <= 64; rows = rows < 3 ? rows + 1 : 21 * rows + 1)
        for (int wave = 0; wave < waves; ++wave) {
          const int b_begin = nb * wave / waves, b_end = nb * (wave + 1) / waves;
          for (int b = b_begin; b < b_end + 4; ++b) {
            const bool in = b < b_end;
            const uint32_t k = qmm::fp8_block_at(b, b_end);
            CHECK(!in || k == 128u * b, "block %d", b);
            const uint64_t owned = uint64_t(rows) * d;
            for (int chunk = 0; chunk < 128; chunk += 16) {
              const uint32_t past = qmm::fp8_past(chunk, b, d);
              CHECK(!in || (past == 0) == (128 * b + chunk < d), "chunk %d of block %d", chunk, b);
              for (uint32_t row : {uint32_t((rows - 1) * d + chunk), qmm::kOOB8})
                CHECK(inside(in ? uint32_t(owned) : 0u, row | past, k, 16, owned),
                      "codes: %d waves, %d rows, d %d, block %d, chunk %d", waves, rows, d, b, chunk);
            }
            if ((b - b_begin) % 4) continue;
            const uint64_t scales = uint64_t(rows) * nb * 4;
            for (uint32_t row : {uint32_t((rows - 1) * nb * 4), qmm::kOOB8})
              CHECK(inside(in ? uint32_t(scales) : 0u, qmm::fp8_scales_at(row, b), 0, 16, scales),
                    "scales: %d waves, %d rows, d %d, block %d", waves, rows, d, b);
            CHECK(qmm::fp8_scales_at(0, b) == 4u * b, "block %d", b);
          }
        }
    }
  return 0;
}

// The kernel that a call takes, for "dense t n d", "grouped n d n_seg m_total
// max_seg_rows" and "norm t d" lines on stdin.
int kernels() {
  char what[16];
  while (scanf("%15s", what) == 1) {
    qmm::Fp8GemmArgs a{};
    long long t = 0;
    if (!strcmp(what, "norm")) {
      int d = 0;
      if (scanf("%lld %d", &t, &d) != 2) return 2;
      const qmm::NormShape p = qmm::norm_shape(t, d);
      printf("norm %d %d\n", p.waves, p.groups);
      continue;
    }
    if (!strcmp(what, "dense")) {
      if (scanf("%lld %d %d", &t, &a.n, &a.d) != 3) return 2;
      a.t = t;
    } else {
      if (scanf("%d %d %d %d %d", &a.n, &a.d, &a.n_seg, &a.m_total, &a.max_seg_rows) != 5) return 2;
      a.t = a.m_total;
      a.max_seg_rows = std::min(a.max_seg_rows, a.m_total);
    }
    const qmm::Fp8Kernel k = qmm::fp8_kernel(a);
    const qmm::Fp8RowsShape p = qmm::fp8_rows_shape(a);
    if (k == qmm::Fp8Kernel::kRows)
      printf("rows %d %d %d\n", p.waves, p.r, p.x8);
    else
      printf("tile %d\n", k == qmm::Fp8Kernel::kTile64 ? 64 : 256);
  }
  return 0;
}

}  // namespace

int main(int argc, char** argv) {
  if (argc > 1 && !strcmp(argv[1], "scale_rows")) return scale_rows();
  if (argc > 1 && !strcmp(argv[1], "rows_copies")) return rows_copies();
  if (argc > 1 && !strcmp(argv[1], "kernels")) return kernels();
  printf("no such check\n");
  return 2;
}
