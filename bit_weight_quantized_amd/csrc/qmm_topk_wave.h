// The choice of a token's experts by one wave, J experts a lane: scores, groups, top-k and
// weights, as the router has it for few tokens or many experts.
#pragma once

#include <hip/hip_runtime.h>

#include <math.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"

namespace qmm {

// Order-preserving map to an unsigned key; 0 marks an expert that cannot be
// chosen: masked (-inf), NaN, or taken.
__device__ __forceinline__ uint32_t choice_key(float c) {
  const uint32_t b = __float_as_uint(c) == 0x80000000u ? 0u : __float_as_uint(c);
  const uint32_t flip = uint32_t(int32_t(b) >> 31) | 0x80000000u;
  return c > -INFINITY ? (b ^ flip) : 0u;
}

__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp_f<0xB1>(v));
  v = fmaxf(v, dpp_f<0x4E>(v));
  v = fmaxf(v, dpp_f<0x141>(v));
  return fmaxf(v, dpp_f<0x140>(v));
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = group_umax<16>(v);
  const uint32_t r0 = __builtin_amdgcn_readlane(int(v), 0), r1 = __builtin_amdgcn_readlane(int(v), 16);
  const uint32_t r2 = __builtin_amdgcn_readlane(int(v), 32), r3 = __builtin_amdgcn_readlane(int(v), 48);
  return umax(umax(r0, r1), umax(r2, r3));
}

__device__ __forceinline__ float readlane_f(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  return (readlane_f(v, 0) + readlane_f(v, 16)) + (readlane_f(v, 32) + readlane_f(v, 48));
}

__device__ __forceinline__ float wave_max(float v) {
  v = row_max(v);
  return fmaxf(fmaxf(readlane_f(v, 0), readlane_f(v, 16)), fmaxf(readlane_f(v, 32), readlane_f(v, 48)));
}

// The two largest of a set, and of the sets of two lanes.
struct Two {
  float first, second;
};
__device__ __forceinline__ void take(Two& t, float v) {
  t.second = fmaxf(t.second, fminf(t.first, v));
  t.first = fmaxf(t.first, v);
}
__device__ __forceinline__ void merge(Two& t, float first, float second) {
  t.second = fmaxf(fmaxf(t.second, second), fminf(t.first, first));
  t.first = fmaxf(t.first, first);
}
template <int CTRL>
__device__ __forceinline__ void merge_dpp(Two& t) {
  merge(t, dpp_f<CTRL>(t.first), dpp_f<CTRL>(t.second));
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

template <bool BF16>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

struct TopkRule {
  int k, groups, keep, gs;   // gs: experts of a group
  // Lanes of a group.  Where a group is a power of two of whole lanes (2 .. 16, as
  // 256 experts in 8 groups) a lane's experts share its group, and the lanes of a
  // group exchange by DPP; otherwise `per` lanes go over a group's scores in LDS.
  bool aligned, by_logit, top2, renorm;
  int per;
};
template <int J, bool SIGMOID>
__device__ __forceinline__ TopkRule topk_rule(int ne, int k, bool bias, int groups, int keep, bool top2, bool renorm) {
  TopkRule r{k, groups, keep, ne / groups, false, !SIGMOID && !bias && (groups == 1 || !top2), top2, renorm, 64};
  const int own = r.gs % J == 0 ? r.gs / J : 0;
  r.aligned = own == 2 || own == 4 || own == 8 || own == 16;
  r.per = r.aligned ? own : 64;
  while (r.per * groups > 64) r.per >>= 1;
  return r;
}

// Lane r has the r-th choice (-1: nothing left, and past k) and its weight before the scale.
struct TopkChoice {
  int expert;
  float weight;
};
// l: the lane's logits, -inf past the experts; bias_of(j), first_lane(j): bias of the lane's j-th
// expert and the first lane of its group; mine: 64·J floats of the wave's own in LDS.
template <int J, bool SIGMOID, typename Bias, typename First>
__device__ __forceinline__ TopkChoice topk_wave(float* l, const TopkRule& rule, Bias bias_of, First first_lane, float* mine) {
  const int lane = threadIdx.x & 63, k = rule.k, gs = rule.gs, per = rule.per;
  float top = 0.f, total = 1.f;
  if constexpr (!SIGMOID) {
    float m = l[0];
#pragma unroll
    for (int j = 1; j < J; ++j) m = fmaxf(m, l[j]);
    m = wave_max(m);
    top = m > -INFINITY ? m : 0.f;              // nothing left: every e^(l - top) is 0
    float z = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) z += expf(l[j] - top);
    total = wave_sum(z);
  }
  auto prob = [&](float v) { return SIGMOID ? sigmoid(v) : total > 0.f ? expf(v - top) / total : total; };
  uint32_t key[J];
  float c[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float p = rule.by_logit ? l[j] : prob(l[j]);
    c[j] = rule.by_logit ? p : p + bias_of(j);
    if (l[j] == -INFINITY) c[j] = -INFINITY;
    key[j] = choice_key(c[j]);
    if (key[j] == 0u) c[j] = -INFINITY;         // NaN ranks with the masked
    l[j] = SIGMOID ? p : l[j];                  // what the weight is made from
  }

  if (rule.groups > 1) {
    Two two = {-INFINITY, -INFINITY};
    const int q = lane / per;                   // the lane's group
    if (rule.aligned) {
#pragma unroll
      for (int j = 0; j < J; ++j) take(two, c[j]);
      merge_dpp<0xB1>(two);
      if (per > 2) merge_dpp<0x4E>(two);
      if (per > 4) merge_dpp<0x141>(two);
      if (per > 8) merge_dpp<0x140>(two);
    } else {
#pragma unroll
      for (int j = 0; j < J; ++j) mine[J * lane + j] = c[j];
      __builtin_amdgcn_wave_barrier();
      if (q < rule.groups)
        for (int i = lane - q * per; i < gs; i += per) take(two, mine[q * gs + i]);
      for (int o = 1; o < per; o <<= 1) merge(two, __shfl_xor(two.first, o), __shfl_xor(two.second, o));
      __builtin_amdgcn_wave_barrier();
    }
    const float value = rule.top2 && two.second > -INFINITY ? two.first + two.second : two.first;
    // rank among the groups: larger values first, equal ones by index
    int rank = 0;
    for (int o = 0; o < rule.groups; ++o) {
      const float v = readlane_f(value, o * per);
      rank += v > value || (v == value && o < q) ? 1 : 0;
    }
    const bool keep = q < rule.groups && rank < rule.keep;
    const uint64_t kept = __ballot(keep);
#pragma unroll
    for (int j = 0; j < J; ++j) key[j] = (rule.aligned ? keep : (kept >> first_lane(j)) & 1) ? key[j] : 0u;
  }
  // probabilities (softmax: logits) by expert, for the weights of the chosen
#pragma unroll
  for (int j = 0; j < J; ++j) mine[J * lane + j] = l[j];

  int mine_e = -1;
  for (int r = 0; r < k; ++r) {
    uint32_t best = key[0];
#pragma unroll
    for (int j = 1; j < J; ++j) best = umax(best, key[j]);
    const uint32_t m = wave_umax(best);
    if (m == 0) break;                          // nothing left (uniform)
    // the lowest lane that holds it, and its lowest expert: scalar work on the
    // comparisons' masks
    uint64_t has[J], any = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      has[j] = __ballot(key[j] == m);
      any |= has[j];
    }
    const int at = __builtin_ctzll(any);
    int j0 = J - 1;
#pragma unroll
    for (int j = J - 2; j >= 0; --j) j0 = (has[j] >> at) & 1 ? j : j0;
    const bool here = lane == at;
#pragma unroll
    for (int j = 0; j < J; ++j) key[j] = here && j == j0 ? 0u : key[j];
    const int win = J * at + j0;
    mine_e = lane == r ? win : mine_e;
  }
  __builtin_amdgcn_wave_barrier();
  float w = 0.f;
  if (mine_e >= 0) w = SIGMOID ? mine[mine_e] : prob(mine[mine_e]);
  if (rule.renorm) {
    const float sum = wave_sum(w);
    w = sum == 0.f ? 0.f : w / sum;             // a NaN stays one
  }
  __builtin_amdgcn_wave_barrier();
  return {mine_e, w};
}

}  // namespace qmm
