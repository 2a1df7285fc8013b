// Microscaled 4-bit path (E2M1 codes in blocks of 32 with an E8M0 exponent, on both sides
// of the product): launch arguments, limits and kernel choice shared by the entry points
// (qmm_mx4_api.cpp) and the kernels.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "qmm_internal.h"

namespace qmm {

constexpr int kMxBlock = 32;    // codes that share one exponent
constexpr int kMxStep = 256;    // codes of a K step: two matrix instructions of 128, half a slab

// Slabs of a row, and the bytes of an activation row's exponents: 16 a slab, zeros past
// the row's blocks, so that the exponents of a slab are one aligned read.
__host__ __device__ constexpr int mx_slabs(int d) { return (d + kSlabCodes - 1) / kSlabCodes; }
__host__ __device__ constexpr int mx_scale_bytes(int d) { return 16 * mx_slabs(d); }
__host__ __device__ constexpr int mx_steps(int d) { return (d + kMxStep - 1) / kMxStep; }

struct Mx4QuantArgs {
  const uint16_t* x;   // [t][ldx] bf16
  int64_t t, ldx;
  int d;
  bool fit;            // exponents without saturation, else those of the maximum's binade
  uint8_t* q;          // [t][d/2]
  uint8_t* scales;     // [t][mx_scale_bytes]
};
int launch_mx4_quant(const Mx4QuantArgs& a, void* stream);

// One product Y = X·Wᵀ, or one for each segment of grouped rows.
struct Mx4GemmArgs {
  const uint8_t* packed;   // blob of [n][d], or the stack's first
  int64_t expert_stride;
  const uint8_t* x;        // [t][d/2] (grouped: [t_x][d/2])
  const uint8_t* xs;       // [t][mx_scale_bytes]
  int64_t t, ldy;
  uint16_t* y;             // [t][ldy] (grouped: [m_total][n], or [m_total][n/2] with the activation)
  int n, d;
  // grouped only (n_seg > 0)
  int64_t t_x;
  const int32_t* row_index;
  const int32_t* seg_expert;
  const int32_t* seg_offsets;
  int n_experts, n_seg, m_total, max_seg_rows;
  bool glu;                // gate rows [0, n/2), up rows [n/2, n): silu(gate)·up
  bool fit;                // how hq is scaled
  uint8_t* hq;             // [m_total][n/4], or NULL: y
  uint8_t* hs;             // [m_total][mx_scale_bytes(n/2)]
};
// Shape of the few-row kernel: 16·r weight rows a workgroup, 8·x8 activation rows a pass,
// and its waves, which split the reduction axis, each with a ring of kMxRing steps: four, or
// two where the LDS does not hold more.
//
// Dense: the shape of the least estimated time, in us.  A round of the workgroups that the CUs
// hold takes 1.5 and its waves' steps, each 0.2 and 0.028 for a KB that it copies, or as long as
// the CU's waves copy at 66 KB a us; never less than the weights at 7 TB/s.  Measured: 47 x 5120
// x 13824 11.8 us with (r 2, x8 6), one workgroup a CU, 16.9 with (2, 4), two passes, 17.9 with
// (1, 6), two rounds; 64 x 4096 x 7168 6.7 with (2, 4), two passes on 256 workgroups, 8.0 with
// (1, 8); 1 x 13824 x 5120 8.4 with (4, 1), 9.6 with (2, 1); 1 x 5120 x 13824 8.3 with (2, 1),
// 9.5 with (4, 1).  Over 14 sizes of 1 to 333 rows the choice took 1.003 of the best shape's time.
// All with weights that a call before has left in the Infinity Cache (three copies in turn).
constexpr int kMxRing = 3;
constexpr int kMxRowsMax = 64;
constexpr int mx4_rows_lds(int r, int x8, int waves) {
  return waves * (kMxRing * 2048 * (r + (x8 + 1) / 2) + (kMxRing + 1) / 2 * 2048);
}
constexpr int mx4_rows_waves(int r, int x8) { return mx4_rows_lds(r, x8, 4) <= 160 * 1024 ? 4 : 2; }
struct Mx4RowsShape {
  int r, x8;
  double us;   // estimated
};
inline Mx4RowsShape mx4_rows_shape(int64_t t, int n, int d) {
  Mx4RowsShape best{0, 0, 0.0};
  for (const int r : {1, 2, 4})
    for (const int x8 : {1, 2, 4, 6, 8}) {
      if ((8 * x8 >= 2 * t && x8 > 1) || (r == 1 && x8 == 8)) continue;   // more than twice the rows; never the least
      const int w = mx4_rows_waves(r, x8), kb = 2 * r + x8;
      const int64_t groups = (int64_t(n) + 16 * r - 1) / (16 * r) * ((t + 8 * x8 - 1) / (8 * x8)), each = (groups + 255) / 256;
      const int64_t resident = 160 * 1024 / mx4_rows_lds(r, x8, w), rounds = (each + resident - 1) / resident;
      const double step = std::max(0.2 + 0.028 * kb, double(std::min(each, resident)) * w * kb / 66);
      const double us = std::max(2.2 + double(rounds) * (1.5 + mx_steps(d) * step / w), 3.2 + double(n) * d * 17 / 32 / 7e6);
      if (best.r == 0 || us < best.us) best = {r, x8, us};
    }
  return best;
}
// Grouped: 8 rows a pass, 16 where segments have more than two on average (64 of 128 experts'
// tokens x 8, 5 rows each, SwiGLU 4096 x 3584 131 us, 150 with 8; 1 row each 95 and 94), and two
// waves; four where there are no more workgroups than CUs and few rows (1 token, 2 of 8
// experts, SwiGLU 2048 x 4096: 7.3 us, 8.7 with two; 8 of 64, 2816 x 2048, 352 workgroups, 11.6
// and 8.2).  R is 4 with the activation, whose 32 outputs are a block, else 2.  The average counts
// empty segments: 128 of them, 126 empty, 64 rows in each of two others, SwiGLU 4096 x 3584 are 8
// passes and take 41.5 us, with 64 x 128 tiles 14.3.
struct Mx4GroupedShape {
  int x8, waves;
};
inline Mx4GroupedShape mx4_grouped_shape(const Mx4GemmArgs& a) {
  if (a.m_total > 2 * int64_t(a.n_seg)) return {2, 2};
  const int64_t groups = (int64_t(a.n) / 2 + 31) / 32 * std::min(a.n_seg, a.m_total);
  return {1, a.glu && groups <= 256 ? 4 : 2};
}
// few rows: weights from memory, once for a pass of the shape's rows
int launch_mx4_rows(const Mx4GemmArgs& a, void* stream);
// many rows: LDS tiles of 256 x 256 (large) or 64 x 128
int launch_mx4_tile(const Mx4GemmArgs& a, bool large, void* stream);
// Tiles of either kind along the rows and the columns of Y; a grid may have fewer than 2^32 threads
// along x.  Grouped: no more row tiles than whole tiles of rows and one part tile a segment.
struct Mx4Tiles {
  int64_t t, n;
  bool fit;
};
inline Mx4Tiles mx4_tiles(const Mx4GemmArgs& a, bool large) {
  const int rows = large ? 256 : 64, cols = (large ? 256 : 128) / (a.glu ? 2 : 1), threads = large ? 512 : 256;
  const int64_t t = a.n_seg ? int64_t(a.m_total) / rows + std::min(a.n_seg, a.m_total) : (a.t + rows - 1) / rows;
  const int64_t n = (int64_t(a.glu ? a.n / 2 : a.n) + cols - 1) / cols;
  return {t, n, t * n * threads < (int64_t(1) << 32)};
}
// the choice between them, and its launch
enum class MxKernel { kRows, kTile64, kTile256 };
inline MxKernel mx4_kernel(const Mx4GemmArgs& a) {
  const int steps = 4 * mx_slabs(a.d);   // of the tile kernels
  if (a.n_seg == 0) {
    // Estimates in us.  Small tiles: a start and end for each round of the 256 CUs and a step of
    // 0.335 us, or 0.24 for each tile that shares a CU; large ones, one a CU: 0.62 us a step
    // while half of the CUs have one, 0.88 when all do.  Measured few-row, 64 x 128, 256 x 256:
    // 128 x 5120 x 5120 10.5, 17.0, 29.8; 333 x 1000 x 2080 5.5, 9.6, 16; 100 x 13824 x 5120
    // 22.4, 17.9, 24.0; 300 x 4096 x 7168 23.0, 23.2, 40.4; 512 x 4096 x 4096 19.4, 15.2, 25.8;
    // 400 x 8192 x 8192 59.8, 31.8, 45.9; 1024 x 5120 x 13824 112, 92.6, 75.3; 1500 x 5120 x
    // 5120 83.5, 46.1, 33.2; 1052 x 10215 x 1312 63.3, 25.1, 19.3; 4096 x 4096 x 512 63.8,
    // 19.4, 13.3; 777 x 1029 x 1184 7.3, 8.1, 14.8.
    if (a.t <= kMxRowsMax) return MxKernel::kRows;
    auto tiles = [&](int rows, int cols) { return double((a.t + rows - 1) / rows) * double((int64_t(a.n) + cols - 1) / cols); };
    const double few = mx4_rows_shape(a.t, a.n, a.d).us;
    const double r64 = tiles(64, 128) / 256, small = 3.5 + steps * std::max(0.335, 0.24 * r64) + std::max(1.0, r64);
    const double t256 = tiles(256, 256), whole = double(int64_t(t256) / 256), rest = t256 - 256 * whole;
    const double large = 3.5 + whole * (7.5 + 0.88 * steps) +
                         (rest > 0 ? 4 + (0.62 + 0.26 * std::max(0.0, rest / 128 - 1)) * steps : 0.0);
    if ((few <= small && few <= large) || !mx4_tiles(a, large < small).fit) return MxKernel::kRows;
    return large < small ? MxKernel::kTile256 : MxKernel::kTile64;
  }
  // The few-row kernel up to 8 rows a segment on average, if none can be long: 64 experts of
  // SwiGLU 4096 x 3584 with 512 rows 90 us, 96 with 64 x 128 tiles; 128 experts, 2048 rows, 230
  // and 158.  Large tiles from 48 rows on, if enough CUs have one: 64 experts of SwiGLU 4096 x
  // 3584, 40 rows each 123 us (64 x 128), 125 (256 x 256), 50 rows 133 and 127, 128 rows 210 and
  // 161; 16 experts of 2048 x 1408, 64 rows each, 128 large tiles, 10.7 and 14.7.
  if (a.max_seg_rows <= kMxRowsMax && a.m_total <= 8 * int64_t(a.n_seg)) return MxKernel::kRows;
  const int64_t tiles = std::max<int64_t>(a.n_seg, a.m_total / 256) * ((int64_t(a.n) + 255) / 256);
  const bool large = a.m_total >= 48 * int64_t(a.n_seg) && tiles >= 160;
  // more tiles than a grid has: the few-row kernel, whose workgroups take turns
  if (!mx4_tiles(a, large).fit) return MxKernel::kRows;
  return large ? MxKernel::kTile256 : MxKernel::kTile64;
}
int launch_mx4_product(const Mx4GemmArgs& a, void* stream);

}  // namespace qmm
