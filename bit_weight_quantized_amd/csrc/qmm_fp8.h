// Block-scaled e4m3 path: launch arguments, limits and kernel choice shared by
// the entry points (qmm_fp8_api.cpp) and the kernels.
#pragma once

#include <stdint.h>

#include <algorithm>

#include "qmm_internal.h"

namespace qmm {

constexpr int kFp8Block = 128;   // codes that share one scale along the reduction axis
inline int fp8_blocks(int64_t d) { return int((d + kFp8Block - 1) / kFp8Block); }
// Scale row of a weight row (of one half with the activation): rows past the matrix,
// which the last tile of a matrix has, take the last one, since ceil(n / 128) is all
// there are.
__host__ __device__ constexpr int fp8_scale_row(int row, int n) { return (row < n ? row : n - 1) / kFp8Block; }

// Offsets of the buffer -> LDS copies.  Only the lane's offset is taken to be held
// against the buffer's size, never the scalar one, and nothing is taken from how the
// machine forms their sum: a copy that may not read everything behind its lane offset
// has all of its offset there, and one from an empty buffer no scalar offset.
constexpr uint32_t kOOB8 = 0x80000000u;   // past every range: reads zero
// activation scales of block b and the three after it, of the row at `row` (or kOOB8)
__host__ __device__ constexpr uint32_t fp8_scales_at(uint32_t row, int b) {
  return (row + 4u * uint32_t(b)) | (row & kOOB8);
}
// scalar offset of block b's codes; past the share that ends at b_end the buffer is empty
__host__ __device__ constexpr uint32_t fp8_block_at(int b, int b_end) {
  return b < b_end ? uint32_t(kFp8Block) * uint32_t(b) : 0u;
}
// set in the lane offset of the 16 codes `chunk` bytes into block b where d ends before
__host__ __device__ constexpr uint32_t fp8_past(int chunk, int b, int d) {
  return kFp8Block * b + chunk < d ? 0u : kOOB8;
}

struct Fp8QuantArgs {
  const uint16_t* x;   // [t][ldx] bf16
  int64_t t, ldx;
  int d;
  uint8_t* q;          // [t][d]
  float* scales;       // [t][blocks]
};
int launch_fp8_quant(const Fp8QuantArgs& a, void* stream);

// One product Y = X·Wᵀ, or one for each segment of grouped rows.
struct Fp8GemmArgs {
  const uint8_t* w;      // [n][d], or [n_experts][n][d]
  const float* ws;       // [scale rows][blocks] of each matrix
  const uint8_t* x;      // [t][d] (grouped: [t_x][d])
  const float* xs;       // [t][blocks]
  uint16_t* y;           // [t][ldy] (grouped: [m_total][n], or [m_total][n/2] with the activation)
  int64_t t, ldy;
  int n, d;
  // grouped only (n_seg > 0)
  int64_t t_x;
  const int32_t* row_index;
  const int32_t* seg_expert;
  const int32_t* seg_offsets;
  int n_experts, n_seg, m_total, max_seg_rows;
  bool glu;              // gate rows [0, n/2), up rows [n/2, n): y = silu(gate)·up
};
// Shape of the few-row kernel: 16·r weight rows a workgroup, whose waves split the
// reduction axis, and 8·x8 activation rows a pass (the smallest of 1, 2, 4, 8 that
// holds the rows, in several passes beyond 64).
//
// Dense: mostly four waves; r the largest that gives more than 128 workgroups: a larger
// r reads the activations less often (64 x 13824 x 5120: 15.6 us with r = 4, 19.6 with
// 2), a smaller one fills 256 CUs (64 x 4096 x 7168: 9.8 us with r = 1, 11.0 with 2, 14.0
// with 4), but half of r at more than 128 workgroups is a second round of the CUs (64 x
// 4352 x 7168: r = 2 11.1, r = 1 17.6; 64 x 9216 x 4096: r = 4 10.8, r = 2 14.2; 1 x 4224
// x 13824: r = 2 13.3, r = 1 14.0).  Up to 16 rows r = 4 was never faster than 2.
// Eight waves instead, for 32 rows a pass at most, which is what their LDS holds, where
// even r = 1 leaves CUs without a workgroup, their own workgroups are one round, and
// every wave still has two blocks: 1 x 3584 x 7168 5.8 us, 6.9 with four; 81 x 525 x
// 11360 8.3, 11.3; 20 x 2304 x 7168 6.1, 6.8; 64 x 2048 x 7168 6.8, 8.2, but 64 x 2304 x
// 7168, of 288 workgroups, 11.0, 8.2; 32 x 4000 x 4096 6.0, 5.4 (beyond 16 rows 160
// workgroups); with r = 2 1 x 8000 x 8192 14.4, 12.0.
//
// Grouped: 8 rows a pass and r = 2 (the tile kernel has the longer segments).  Two
// waves, each with a longer run of blocks, but four where there may be fewer than 512
// workgroups (1 token, 8 experts, 1024 x 3584: 7.9 us, 10.4 with two; 2 tokens, 6 of 64
// experts, 2816 x 2048: 15.9 us, 14.0 with two).
constexpr int kFp8RowsMax = 64;
inline int64_t fp8_usual_rows(const Fp8GemmArgs& a) { return (int64_t(a.m_total) + a.n_seg - 1) / a.n_seg; }
struct Fp8RowsShape {
  int r, x8, waves;
  int64_t workgroups;   // dense
};
inline Fp8RowsShape fp8_rows_shape(const Fp8GemmArgs& a) {
  if (a.n_seg > 0) return {2, 1, (int64_t(a.n) + 31) / 32 * std::min(a.n_seg, a.m_total) < 512 ? 4 : 2, 0};
  int x8 = a.t <= 8 ? 1 : a.t <= 16 ? 2 : a.t <= 32 ? 4 : 8;
  auto workgroups = [&](int r) { return (int64_t(a.n) + 16 * r - 1) / (16 * r) * ((a.t + 8 * x8 - 1) / (8 * x8)); };
  int r = x8 <= 2 ? 2 : 4;
  while (r > 1 && workgroups(r) <= 128) r /= 2;
  const int x4 = std::min(x8, 4);   // eight waves: 32 rows a pass
  const int64_t four = workgroups(1), eight = (int64_t(a.n) + 15) / 16 * ((a.t + 8 * x4 - 1) / (8 * x4));
  if (r > 1 || eight > 256 || four > (x8 <= 2 ? 256 : 160) || a.d < 16 * kFp8Block) return {r, x8, 4, workgroups(r)};
  return {1, x4, 8, eight};
}
// few rows: every weight read once for up to 64 rows
int launch_fp8_rows(const Fp8GemmArgs& a, void* stream);
// many rows: LDS tiles of 256 x 256 (large) or 64 x 128
int launch_fp8_tile(const Fp8GemmArgs& a, bool large, void* stream);
// the choice between them, and its launch
enum class Fp8Kernel { kRows, kTile64, kTile256 };
inline Fp8Kernel fp8_kernel(const Fp8GemmArgs& a) {
  if (a.n_seg == 0) {
    // Estimates in us of the three kernels from nb steps and the rounds of workgroups
    // that 256 CUs take: a start and end, and a time for each step, which for the
    // few-row kernel (its waves share the steps) depends on its weight blocks and on
    // rows that share their cache lines, and of which three 64 x 128 tiles a CU hide
    // a part from each other.  Measured few-row, 64 x 128, 256 x 256: 768 x 1903 x
    // 4240 29.4, 24.7, 50.5; 512 x 4096 x 4096 19.8, 23.0, 42.9; 1024 x 4096 x 4096
    // 38.4, 28.6, 43.5; 1052 x 10215 x 1296 63.3, 33.2, 24.9; 129 x 5619 x 4352 18.7,
    // 23.9, 42.4; 1500 x 5120 x 5120 90.5, 64.5, 55.4.  Over 157 drawn sizes of 17 ..
    // 4096 rows the choice took 1.02 of the time of the best kernel (geometric mean).
    auto rounds = [](int64_t workgroups) { return double((workgroups + 255) / 256); };
    auto tiles = [&](int rows, int cols) { return ((a.t + rows - 1) / rows) * ((int64_t(a.n) + cols - 1) / cols); };
    const Fp8RowsShape p = fp8_rows_shape(a);
    const int nb = fp8_blocks(a.d);
    const double step = (p.r == 4 ? 0.95 : p.r == 2 ? 0.8 : 0.6) * (a.d % kFp8Block ? 1.4 : 1.0);
    const double few = rounds(p.workgroups) * (3 + (nb + p.waves - 1) / p.waves * step);
    const double r64 = rounds(tiles(64, 128)), small = 3 + nb * std::max(0.65, 0.4 * r64) + 0.6 * r64;
    const double large = rounds(tiles(256, 256)) * (8 + 1.5 * nb);
    if (a.t <= kFp8RowsMax || (few <= small && few <= large)) return Fp8Kernel::kRows;
    return large < small ? Fp8Kernel::kTile256 : Fp8Kernel::kTile64;
  }
  // The few-row kernel up to 3 rows a segment on average, if none can be long: 128
  // experts, 32 rows of SwiGLU 4096 x 3584 (25 experts have rows) 66.6 us few-row, 78.6
  // (64 x 128); plain 3584 x 2048, 128 rows (54 experts) 64.9 and 66.4, 384 rows (88
  // experts) 118.5 and 115.0, 512 rows 125.5 and 113.5; 8 rows of 8 experts, SwiGLU 1024
  // x 3584, 7.9 and 25.4.  Large tiles from 80 rows on, if half of the CUs have one: 64
  // experts of SwiGLU 2816 x 2048, 63 rows each 80.3 us (64 x 128), 84.2 (256 x 256), 96
  // rows 98.1 and 88.0, 192 rows 149.7 and 119.7; 8 of 704 x 4080 with 150 rows, 24
  // large tiles, 25.4 and 47.1.
  if (a.max_seg_rows <= kFp8RowsMax && fp8_usual_rows(a) <= 3) return Fp8Kernel::kRows;
  const int64_t tiles = std::max<int64_t>(a.n_seg, a.m_total / 256) * ((int64_t(a.n) + 255) / 256);
  return int64_t(a.m_total) >= int64_t(80) * a.n_seg && tiles >= 128 ? Fp8Kernel::kTile256 : Fp8Kernel::kTile64;
}
int launch_fp8_product(const Fp8GemmArgs& a, void* stream);

struct TopkArgs {
  const void* logits;   // [t][ld], bf16 or fp32
  bool bf16;
  int64_t t, ld;
  int ne;
  bool sigmoid;
  const float* bias;    // [ne] or NULL
  int groups, keep;
  bool top2;
  int k;
  bool renorm;
  float scale;
  int32_t* topk;        // [t][k]
  float* weights;       // [t][k]
  int32_t* seg_expert;  // [ne]
  int32_t* seg_offsets; // [ne + 1]
  int32_t* row_index;   // [t·k]
  int32_t* slot_row;    // [t][k]
  int32_t* ws;          // counts [chunks][ne], or NULL for one chunk
};
// Tokens of one workgroup: up to kTopkChunk in one (no workspace); else 16 or more,
// up to kTopkMaxChunks chunks, one for each CU (the second kernel adds every chunk's
// counts up itself).
constexpr int kTopkWaves = 16;
constexpr int kTopkChunk = 128;
constexpr int64_t kTopkMaxChunks = 256;
inline int64_t topk_chunk(int64_t t, int ne) {
  if (t <= kTopkChunk) return kTopkChunk;
  int64_t c = ne > 1 ? 16 : 32;   // a single expert's count takes a whole word
  while (c < kTopkChunk && (t + c - 1) / c > kTopkMaxChunks) c *= 2;
  if ((t + c - 1) / c > kTopkMaxChunks) c = round_up((t + kTopkMaxChunks - 1) / kTopkMaxChunks, kTopkChunk);
  return c;
}
// The workspace: a chunk's counts by expert, a byte each where they fit, in rows of
// whole words, else 4 bytes.
__host__ __device__ constexpr bool topk_bytes(int64_t chunk) { return chunk <= kTopkChunk; }
__host__ __device__ constexpr int topk_row(int ne) { return (ne + 3) / 4 * 4; }
inline size_t topk_ws_bytes(int64_t t, int ne) {
  const int64_t c = topk_chunk(t, ne);
  return t <= c ? 0 : size_t((t + c - 1) / c) * (topk_bytes(c) ? size_t(topk_row(ne)) : size_t(ne) * 4);
}
int launch_topk(const TopkArgs& a, void* stream);

struct GatherArgs {
  const uint16_t* o;         // [m_total][d]
  int m_total, d, k;
  int64_t t;
  const int32_t* slot_row;   // [t][k]
  const float* weights;      // [t][k]
  const uint16_t* shared;    // [t][d] or NULL
  uint16_t* out;             // [t][d]
};
int launch_gather(const GatherArgs& a, void* stream);

struct NormArgs {
  int64_t t;
  int d;
  const uint16_t* o;        // [t][ldo] or NULL
  int64_t ldo;
  const uint16_t* post_w;   // [d] or NULL
  const uint16_t* gate;     // [ceil(t / gate_rows)][ldg] or NULL
  int64_t ldg, gate_rows;
  const void* r;            // [t][ldr], bf16 or fp32
  bool r_f32;
  int64_t ldr;
  float res_scale;
  void* r_out;              // [t][ldr_out], type of r, or NULL
  int64_t ldr_out;
  const uint16_t* pre_w;    // [d], or NULL where no h, q are asked for
  float w_offset, eps;
  uint16_t* h;              // [t][ldh] or NULL
  int64_t ldh;
  uint8_t* q;               // [t][d] or NULL
  float* q_scales;          // [t][blocks]
};
// Waves of a row's workgroup and groups of 8 elements a lane, by width: eight waves,
// with as few groups a lane as hold the row (8192 rows of 4096: 52.3 us, 54.0 with four
// waves, 66.3 with sixteen; 7168: 95.5, 99.6, 97.9), but four where eight would leave
// lanes without work (8192 of 5120: 73.3, 75.1 with eight, 77.5 with sixteen), and
// sixteen for up to 256 rows, a row for each CU, whose loads are all in flight at once
// (by the kernel's own time 64 of 5120: 4.2 us, 4.4 with four; 256: 4.9, 5.2; 300: 6.6,
// 6.0).
struct NormShape {
  int waves, groups;
};
inline NormShape norm_shape(int64_t t, int d) {
  const int n8 = d / 8;
  if (n8 <= 64) return {1, 1};
  if (n8 <= 256) return {4, 1};
  if (n8 <= 512) return {8, 1};
  if (t <= 256 && n8 <= 1024) return {16, 1};
  if (n8 <= 768) return {4, 3};
  if (n8 <= 1024) return {8, 2};
  if (n8 <= 1536) return {8, 3};
  if (n8 <= 2048) return {8, 4};
  if (n8 <= 4096) return {16, 4};
  return {16, 8};
}
int launch_norm_residual(const NormArgs& a, void* stream);

}  // namespace qmm
