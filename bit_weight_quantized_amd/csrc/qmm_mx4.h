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
// few rows: weights straight to registers
int launch_mx4_rows(const Mx4GemmArgs& a, void* stream);
// the choice of kernel, and its launch
int launch_mx4_product(const Mx4GemmArgs& a, void* stream);

}  // namespace qmm
