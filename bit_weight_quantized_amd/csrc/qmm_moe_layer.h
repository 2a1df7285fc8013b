// A mixture-of-experts layer for a few tokens: launch arguments and limits.
#pragma once

#include <stdint.h>

#include "qmm_internal.h"

namespace qmm {

constexpr int kLayerMaxTokens = 16;    // columns of a matrix instruction
constexpr int kLayerMaxPairs = 256;    // tokens times choices

struct MoeLayerArgs {
  const uint8_t* gate_up;   // packed MXFP4 stacks: [n_experts] of [2·inter, d]
  int64_t gate_up_stride;
  const uint8_t* down;      // and of [d, inter]
  int64_t down_stride;
  int n_experts, d, inter;
  const uint16_t* x;        // [t][d] bf16
  int t;
  const void* logits;       // [t][ld], bf16 or fp32
  bool bf16;
  int64_t ld;
  bool sigmoid;
  const float* bias;        // [n_experts] or NULL
  int groups, keep;
  bool top2;
  int k;
  bool renorm;
  float scale;
  const uint16_t* shared;   // [t][d] or NULL
  int32_t* topk;            // [t][k]
  float* weights;           // [t][k]
  uint16_t* out;            // [t][d]
  uint16_t* h;              // the workspace, rows by expert, then token: [2][t·k][inter] two bf16 parts, or
  bool pairs;               // [t·k][inter] pairs with an exponent
  int cols;                 // columns of a workgroup in the second kernel, even, <= 16; set by the launch
};
int launch_moe_layer(const MoeLayerArgs& a, void* stream);

}  // namespace qmm
