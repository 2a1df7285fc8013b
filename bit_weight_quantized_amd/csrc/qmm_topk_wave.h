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
// The larger key, or of equal ones the lower expert, into the first.
__device__ __forceinline__ void order(uint32_t& ka, uint32_t& kb, int& ea, int& eb) {
  const bool swap = kb > ka || (kb == ka && eb < ea);
  const uint32_t k = ka;
  const int e = ea;
  ka = swap ? kb : ka;
  ea = swap ? eb : ea;
  kb = swap ? k : kb;
  eb = swap ? e : eb;
}

// N tokens at once, whose chains of operations fill each other's gaps.  l: the lane's logits of
// each, -inf past the experts; bias_of(j), first_lane(j): bias of the lane's j-th expert and the
// first lane of its group; mine: 64·J floats for each token, the wave's own in LDS.
template <int J, bool SIGMOID, bool SORTED, int N, typename Bias, typename First>
__device__ __forceinline__ void topk_wave(float (&l)[N][J], const TopkRule& rule, Bias bias_of, First first_lane, float* mine,
                                          TopkChoice (&out)[N]) {
  const int lane = threadIdx.x & 63, k = rule.k, gs = rule.gs, per = rule.per;
  float top[N], total[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    top[n] = 0.f;
    total[n] = 1.f;
    if constexpr (!SIGMOID) {
      float m = l[n][0];
#pragma unroll
      for (int j = 1; j < J; ++j) m = fmaxf(m, l[n][j]);
      m = wave_max(m);
      top[n] = m > -INFINITY ? m : 0.f;         // nothing left: every e^(l - top) is 0
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) z += expf(l[n][j] - top[n]);
      total[n] = wave_sum(z);
    }
  }
  auto prob = [&](int n, float v) { return SIGMOID ? sigmoid(v) : total[n] > 0.f ? expf(v - top[n]) / total[n] : total[n]; };
  uint32_t key[N][J];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float c[J], *at = mine + 64 * J * n;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float p = rule.by_logit ? l[n][j] : prob(n, l[n][j]);
      c[j] = rule.by_logit ? p : p + bias_of(j);
      if (l[n][j] == -INFINITY) c[j] = -INFINITY;
      key[n][j] = choice_key(c[j]);
      if (key[n][j] == 0u) c[j] = -INFINITY;    // NaN ranks with the masked
      l[n][j] = SIGMOID ? p : l[n][j];          // what the weight is made from
    }

    if (rule.groups > 1) {
      Two two = {-INFINITY, -INFINITY};
      const int q = lane / per;                 // the lane's group
      if (rule.aligned) {
#pragma unroll
        for (int j = 0; j < J; ++j) take(two, c[j]);
        merge_dpp<0xB1>(two);
        if (per > 2) merge_dpp<0x4E>(two);
        if (per > 4) merge_dpp<0x141>(two);
        if (per > 8) merge_dpp<0x140>(two);
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j) at[J * lane + j] = c[j];
        __builtin_amdgcn_wave_barrier();
        if (q < rule.groups)
          for (int i = lane - q * per; i < gs; i += per) take(two, at[q * gs + i]);
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
      for (int j = 0; j < J; ++j) key[n][j] = (rule.aligned ? keep : (kept >> first_lane(j)) & 1) ? key[n][j] : 0u;
    }
    // probabilities (softmax: logits) by expert, for the weights of the chosen
#pragma unroll
    for (int j = 0; j < J; ++j) at[J * lane + j] = l[n][j];
  }

  // A round takes the largest key, from the lowest lane that holds it and there the lowest
  // expert: SORTED from a lane's list in order, which is the shorter chain (one token, 256
  // experts, k = 8: 0.3 us), else by scalar work on the comparisons' masks, which is less work (100
  // tokens in 16 waves: 10.9 us, 11.1).
  int mine_e[N], e[N][J];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    mine_e[n] = -1;
    if constexpr (SORTED) {
#pragma unroll
      for (int j = 0; j < J; ++j) e[n][j] = J * lane + j;
#pragma unroll
      for (int a = J - 1; a > 0; --a)
#pragma unroll
        for (int j = 0; j < a; ++j) order(key[n][j], key[n][j + 1], e[n][j], e[n][j + 1]);
    }
  }
  for (int r = 0; r < k; ++r) {
    uint32_t m[N], left = 0;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      uint32_t best = key[n][0];
      if constexpr (!SORTED) {
#pragma unroll
        for (int j = 1; j < J; ++j) best = umax(best, key[n][j]);
      }
      m[n] = wave_umax(best);
      left |= m[n];
    }
    if (left == 0) break;                       // nothing left (uniform)
#pragma unroll
    for (int n = 0; n < N; ++n) {
      int win;
      if constexpr (SORTED) {
        const int at = __builtin_ctzll(__ballot(key[n][0] == m[n]));
        win = __builtin_amdgcn_readlane(e[n][0], at);
        const bool here = lane == at;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          key[n][j] = here ? (j + 1 < J ? key[n][j + 1] : 0u) : key[n][j];
          if (j + 1 < J) e[n][j] = here ? e[n][j + 1] : e[n][j];
        }
      } else {
        uint64_t has[J], any = 0;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          has[j] = __ballot(key[n][j] == m[n]);
          any |= has[j];
        }
        const int at = __builtin_ctzll(any);
        int j0 = J - 1;
#pragma unroll
        for (int j = J - 2; j >= 0; --j) j0 = (has[j] >> at) & 1 ? j : j0;
        const bool here = lane == at;
#pragma unroll
        for (int j = 0; j < J; ++j) key[n][j] = here && j == j0 ? 0u : key[n][j];
        win = J * at + j0;
      }
      mine_e[n] = lane == r && m[n] != 0 ? win : mine_e[n];
    }
  }
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float w = 0.f;
    if (mine_e[n] >= 0) w = SIGMOID ? mine[64 * J * n + mine_e[n]] : prob(n, mine[64 * J * n + mine_e[n]]);
    if (rule.renorm) {
      const float sum = wave_sum(w);
      w = sum == 0.f ? 0.f : w / sum;           // a NaN stays one
    }
    out[n] = {mine_e[n], w};
  }
  __builtin_amdgcn_wave_barrier();
}

}  // namespace qmm
