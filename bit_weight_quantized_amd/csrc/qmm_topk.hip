// Router from logits to grouped rows: softmax or sigmoid scores, a balance
// bias, the best groups of experts, top-k, renormalised weights, and the
// tables that the grouped matmuls and the gather read.
//
//   p = softmax(l) or 1 / (1 + e^-l);  a logit of -inf masks its expert (p = 0)
//   c = p + bias, or l itself (softmax, no bias, no sum over a group: the same
//       order, without the rounding of e^l)
//   groups ranked by their largest c or the sum of their two largest; the k
//   largest c of the kept groups; weight p (/ Σ p of the chosen) · scale
//
// One workgroup of 16 waves per chunk of tokens.  Up to 256 experts and k = 16, a
// row of 16 lanes has a token (four a wave), so that no step leaves the row's DPP:
// lane i holds experts n·i .. n·i + n-1, n = ceil(experts / 16).  A round takes the
// largest order-preserving integer key of the row, the lowest expert that has it (a
// second reduction) and drops it; 129 to 256 experts take a sort of each lane's 8
// largest and merges across the row instead where there are 5 to 8 rounds.  More
// experts: a wave has a token, and scalar instructions find the winner in the
// comparisons' masks.
// 16384 tokens x 256 experts in 8 groups, k = 8, are 2 us of bytes and take 24 (18.5
// router, 6.8 placing in a trace; a wave a token: 34).  Counters of the router: 1530
// vector instructions a wave, which has four tokens once; the vector units issue 64%
// of the time, the rest is what a wave's one pass waits for.  A sigmoid that rounds as
// the formula does is 35 instructions a score, 560 of those a wave, and scores that
// round otherwise would change choices; the sort is 360.  Placing waits for the counts
// and its LDS passes: its vector units issue half of a CU's busy time.
//
// Grouping counts the chunk's tokens per expert in LDS (integer atomics, order
// free).  One chunk: the same workgroup scans the counts and places its rows.
// More: the counts go to the workspace (a byte each, as a chunk of up to 128 tokens
// allows), and a second kernel, one workgroup per chunk, adds up every chunk's counts
// (at most 256 per expert) and places the chunk's rows.  Rows of an expert ascend
// with the token, found from a bitmap of the chunk's tokens per expert, so nothing
// depends on timing.
#include <hip/hip_runtime.h>

#include <math.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"
#include "qmm_launch.h"
#include "qmm_topk_wave.h"

namespace qmm {
namespace {

constexpr int kTkWords = kTopkChunk / 32;        // bitmap words of an expert and pass
constexpr int kTopkRowMaxK = 16;                 // lane r of a row holds the r-th choice
constexpr int kTopkRounds = 4;                   // more rounds of 84 instructions cost more than the sort's 360
static_assert(kRouteMaxExperts == 64 * kTopkWaves, "a thread of the workgroup owns an expert");

// Smallest of the 16 lanes of a row; every lane gets it.
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }
__device__ __forceinline__ uint32_t row_umin(uint32_t v) {
  v = umin(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));
  v = umin(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));
  v = umin(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 0xF, 0xF, false)));
  return umin(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x140, 0xF, 0xF, false)));
}
template <int WAVES>
struct TopkLds {
  static constexpr int kThreads = 64 * WAVES;    // a thread owns an expert
  int32_t count[kThreads];
  int32_t first[kThreads];                       // the next row of each expert
  uint32_t bits[kThreads][kTkWords];
  int32_t wsum[WAVES];
};

// Exclusive sum over the workgroup's threads; every thread gets the total too.
template <int WAVES>
__device__ __forceinline__ int block_scan(int c, int32_t* wsum, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = c;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int up = __shfl_up(incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    before += w < wave ? wsum[w] : 0;
    all += wsum[w];
  }
  *total = all;
  return before + incl - c;
}

// Writes the rows of tokens [t0, t1), whose ids are ids[0 ..] and whose first row
// of expert e is lds.first[e]: 128 tokens at a time, one bit per (expert, token).
template <int WAVES>
__device__ __forceinline__ void place_rows(TopkLds<WAVES>& lds, const int32_t* ids, int64_t t0, int64_t t1, int k,
                                           int32_t* row_index, int32_t* slot_row) {
  const int tid = threadIdx.x;
  for (int64_t b0 = t0; b0 < t1; b0 += kTopkChunk) {
    const int nb = int(min(int64_t(kTopkChunk), t1 - b0)) * k;
#pragma unroll
    for (int h = 0; h < kTkWords; ++h) lds.bits[tid][h] = 0u;
    __syncthreads();
    for (int i = tid; i < nb; i += 64 * WAVES) {
      const int e = ids[(b0 - t0) * k + i], tl = i / k;
      if (e >= 0) atomicOr(&lds.bits[e][tl >> 5], 1u << (tl & 31));
    }
    __syncthreads();
    for (int i = tid; i < nb; i += 64 * WAVES) {
      const int e = ids[(b0 - t0) * k + i], tl = i / k;
      int row = -1;
      if (e >= 0) {
        row = lds.first[e] + __builtin_popcount(lds.bits[e][tl >> 5] & ((1u << (tl & 31)) - 1u));
        for (int h = 0; h < tl >> 5; ++h) row += __builtin_popcount(lds.bits[e][h]);
        row_index[row] = int32_t(b0 + tl);
      }
      slot_row[b0 * k + i] = row;
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kTkWords; ++h) lds.first[tid] += __builtin_popcount(lds.bits[tid][h]);
  }
}

// The end of a chunk: its counts to the workspace, or (ONE: it is the only one) the
// tables themselves.
template <int WAVES, bool ONE>
__device__ __forceinline__ void finish(const TopkArgs& a, TopkLds<WAVES>& lds, const int32_t* chosen, int chunk,
                                       int64_t t0, int64_t t1) {
  const int tid = threadIdx.x;
  __syncthreads();                                // counts; the ids of the chunk
  if constexpr (!ONE) {
    if (a.t <= kTopkChunk) return;                // counted from the ids
    if (topk_bytes(chunk)) {
      for (int i = tid; i < topk_row(a.ne); i += 64 * WAVES)   // zeros at the end
        reinterpret_cast<uint8_t*>(a.ws)[int64_t(blockIdx.x) * topk_row(a.ne) + i] = uint8_t(lds.count[i]);
    } else if (tid < a.ne) {
      a.ws[int64_t(blockIdx.x) * a.ne + tid] = lds.count[tid];
    }
  } else {
    int total;
    const int at = block_scan<WAVES>(lds.count[tid], lds.wsum, &total);
    lds.first[tid] = at;
    if (tid < a.ne) {
      a.seg_expert[tid] = tid;
      a.seg_offsets[tid] = at;
    }
    if (tid == 0) a.seg_offsets[a.ne] = total;
    for (int64_t i = total + tid; i < a.t * a.k; i += 64 * WAVES) a.row_index[i] = -1;
    place_rows(lds, chosen, t0, t1, a.k, a.row_index, a.slot_row);
  }
}

// Logits of a row of 16 lanes: J a lane from e0 on; `whole`: the row has 16·J, read
// at any alignment.
template <int J, bool BF16>
__device__ __forceinline__ void load_row(const void* logits, int64_t at, int e0, int n, int ne, bool whole, float* v) {
  if (whole && J >= 4) {
    if constexpr (BF16) {
      typedef uint32_t word2_t __attribute__((ext_vector_type(2), aligned(2)));
      const uint16_t* p = static_cast<const uint16_t*>(logits) + at + e0;
#pragma unroll
      for (int j = 0; j < J / 4; ++j) {
        const word2_t w = reinterpret_cast<const word2_t*>(p)[j];
        v[4 * j] = bf16_lo(w[0]);
        v[4 * j + 1] = bf16_hi(w[0]);
        v[4 * j + 2] = bf16_lo(w[1]);
        v[4 * j + 3] = bf16_hi(w[1]);
      }
    } else {
      typedef float float4_at4_t __attribute__((ext_vector_type(4), aligned(4)));
      const float* p = static_cast<const float*>(logits) + at + e0;
#pragma unroll
      for (int j = 0; j < J / 4; ++j) {
        const float4_at4_t w = reinterpret_cast<const float4_at4_t*>(p)[j];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * j + i] = w[i];
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const float l = logit<BF16>(logits, at + min(e0 + j, ne - 1));
    v[j] = j < n && e0 + j < ne ? l : -INFINITY;
  }
}

// Sorting of keys that carry their expert: the 62 bits (key, 255 - code) as a positive
// double, whose order is theirs (the exponent stays below that of infinity), since a
// 64-bit maximum is one instruction on doubles.  In asm: fmax would quiet NaNs first.
__device__ __forceinline__ double wide_key(uint32_t key, uint32_t code) {
  return __hiloint2double(int(key >> 2), int(key << 30 | (255u - code)));
}
__device__ __forceinline__ double wide_max(double a, double b) {
  double r;
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ double wide_min(double a, double b) {
  double r;
  asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ void wide_order(double& a, double& b) {   // the larger first
  const double hi = wide_max(a, b);
  b = wide_min(a, b);
  a = hi;
}
// 8 values that rise and then fall (or the reverse), largest first: Batcher's bitonic merge
__device__ __forceinline__ void wide_merge(double* v) {
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) wide_order(v[i], v[i + d]);
}
// 8 values, largest first: Batcher's odd-even merge network (pairs, then merges of 2
// and 4)
__device__ __forceinline__ void wide_sort(double* v) {
  constexpr int pair[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                               {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
  for (int i = 0; i < 19; ++i) wide_order(v[pair[i][0]], v[pair[i][1]]);
}
// the 8 largest of this lane's and another's, both sorted
template <int CTRL>
__device__ __forceinline__ void wide_join(double* v) {
  double o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    o[i] = __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v[i]), CTRL, 0xF, 0xF, false),
                            __builtin_amdgcn_update_dpp(0, __double2loint(v[i]), CTRL, 0xF, 0xF, false));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = wide_max(v[i], o[7 - i]);
  wide_merge(v);
}

// A row of 16 lanes a token, J experts a lane at most.
template <int WAVES, int J, bool BF16, bool SIGMOID, bool ONE>
__global__ __launch_bounds__(64 * WAVES) void topk_row_kernel(TopkArgs a, int chunk) {
  __shared__ TopkLds<WAVES> lds;
  __shared__ float cs[WAVES][J][64];             // a token's scores, [j][lane]
  __shared__ __attribute__((aligned(16))) float group_value[WAVES][4][kRouteMaxK];   // at most 64 groups
  __shared__ uint32_t group_kept[WAVES][4][kRouteMaxK];
  __shared__ int32_t chosen[ONE ? kTopkChunk * kTopkRowMaxK : 1];
  const int tid = threadIdx.x;
  const int lane = tid & 63, rl = lane & 15, rt = lane >> 4;   // lane of the row, row of the wave
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = int(blockIdx.x) * chunk, t1 = min(int(a.t), t0 + chunk);   // at most 2^24 tokens
  const int ne = a.ne, k = a.k, groups = a.groups;
  const int n = (ne + 15) >> 4, e0 = n * rl;      // the lane's experts
  const int gs = ne / groups;                     // experts of a group
  const bool by_logit = !SIGMOID && !a.bias && (groups == 1 || !a.top2);
  // Where a group is a power of two of whole lanes (as 256 experts in 8 groups: 2) a
  // lane's experts share its group, and its lanes exchange by DPP; otherwise each
  // lane goes over the scores of its groups in LDS.
  const int own = gs % n == 0 ? gs / n : 0;
  const bool aligned = own == 1 || own == 2 || own == 4 || own == 8 || own == 16;
  const int own_shift = aligned ? __builtin_ctz(own) : 0;
  const int g0 = min(e0, ne - 1) / gs, g0_at = min(e0, ne - 1) - g0 * gs;   // the first expert's group, and its place there
  const bool whole = ne == 16 * J;

  lds.count[tid] = 0;
  float bias[J];
#pragma unroll
  for (int j = 0; j < J; ++j) bias[j] = a.bias ? a.bias[min(e0 + j, ne - 1)] : 0.f;
  float* value_of = group_value[wave][rt];
  uint32_t* kept_of = group_kept[wave][rt];
#pragma unroll
  for (int i = 0; i < kRouteMaxK / 16; ++i) value_of[16 * i + rl] = -INFINITY;
  __syncthreads();

  for (int first = t0 + 4 * wave; first < t1; first += 4 * WAVES) {
    const int tok = first + rt;
    const bool live = tok < t1;
    float l[J];
    uint32_t key[J];
    int from = e0;
    asm volatile("" : "+v"(from));                // what hangs on it is not kept from token to token
    load_row<J, BF16>(a.logits, int64_t(min(tok, t1 - 1)) * a.ld, from, n, ne, whole, l);
    float top = 0.f, total = 1.f;
    if constexpr (!SIGMOID) {
      float m = l[0];
#pragma unroll
      for (int j = 1; j < J; ++j) m = fmaxf(m, l[j]);
      m = row_max(m);
      top = m > -INFINITY ? m : 0.f;              // nothing left: every e^(l - top) is 0
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) z += expf(l[j] - top);
      total = sum16(z);
    }
    auto prob = [&](float v) { return SIGMOID ? sigmoid(v) : total > 0.f ? expf(v - top) / total : total; };
    Two two = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float p = by_logit ? l[j] : prob(l[j]);
      float c = by_logit ? p : p + bias[j];
      if (l[j] == -INFINITY) c = -INFINITY;
      key[j] = choice_key(c);
      if (key[j] == 0u) c = -INFINITY;            // NaN ranks with the masked
      l[j] = SIGMOID ? p : l[j];                  // what the weight is made from
      take(two, c);
      if (groups > 1 && !aligned) cs[wave][j][lane] = c;
    }
    if (groups > 1) {
      auto worth = [&](const Two& v) { return a.top2 && v.second > -INFINITY ? v.first + v.second : v.first; };
      // rank among the groups: larger values first, equal ones by index
      auto kept = [&](float v, int q) {
        int rank = 0;
        for (int o = 0; o < groups; o += 4) {
          const f32x4_t u = *reinterpret_cast<const f32x4_t*>(value_of + o);
#pragma unroll
          for (int i = 0; i < 4; ++i) rank += u[i] > v || (u[i] == v && o + i < q) ? 1 : 0;
        }
        return rank < a.keep;
      };
      if (aligned) {
        if (own > 1) merge_dpp<0xB1>(two);
        if (own > 2) merge_dpp<0x4E>(two);
        if (own > 4) merge_dpp<0x141>(two);
        if (own > 8) merge_dpp<0x140>(two);
        const int q = rl >> own_shift;
        const float v = worth(two);
        if (q < groups) value_of[q] = v;
        __builtin_amdgcn_wave_barrier();
        const bool keep = q < groups && kept(v, q);
#pragma unroll
        for (int j = 0; j < J; ++j) key[j] = keep ? key[j] : 0u;
      } else {
        __builtin_amdgcn_wave_barrier();
        for (int q = rl; q < groups; q += 16) {
          Two best = {-INFINITY, -INFINITY};
          int at = q * gs / n, j = q * gs - at * n;
          for (int i = 0; i < gs; ++i) {
            take(best, cs[wave][j][16 * rt + at]);
            if (++j == n) {
              j = 0;
              ++at;
            }
          }
          value_of[q] = worth(best);
        }
        __builtin_amdgcn_wave_barrier();
        for (int q = rl; q < groups; q += 16) kept_of[q] = kept(value_of[q], q) ? 1u : 0u;
        __builtin_amdgcn_wave_barrier();
        int q = g0, i = g0_at;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          key[j] = kept_of[min(q, groups - 1)] ? key[j] : 0u;
          if (++i == gs) {
            i = 0;
            ++q;
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
    // probabilities (softmax: logits) for the weights of the chosen
#pragma unroll
    for (int j = 0; j < J; ++j) cs[wave][j][lane] = l[j];

    // an expert's code, 16·lane + j, has the experts' order
    uint32_t mine = ~0u;
    const bool sorted = J == 16 && k > kTopkRounds && k <= 8;
    if (J == 16 && sorted) {
      double v[J];
#pragma unroll
      for (int j = 0; j < J; ++j) v[j] = wide_key(key[j], uint32_t(16 * rl + j));
      wide_sort(v);
      wide_sort(v + J / 2);
#pragma unroll
      for (int i = 0; i < J / 2; ++i) v[i] = wide_max(v[i], v[J - 1 - i]);
      wide_merge(v);
      wide_join<0xB1>(v);
      wide_join<0x4E>(v);
      wide_join<0x141>(v);
      wide_join<0x140>(v);
      double pick = v[0];
#pragma unroll
      for (int i = 1; i < J / 2; ++i) pick = rl == i ? v[i] : pick;
      const uint32_t lo = uint32_t(__double2loint(pick));
      if (rl < k && (__double2hiint(pick) != 0 || lo >> 30 != 0)) mine = 255u - (lo & 255u);
    }
    for (int r = sorted ? k : 0; r < k; ++r) {
      uint32_t best = key[0];
#pragma unroll
      for (int j = 1; j < J; ++j) best = umax(best, key[j]);
      const uint32_t m = group_umax<16>(best);
      if (!__any(m != 0u)) break;                 // nothing left in any row
      uint32_t at = 255u;
#pragma unroll
      for (int j = J - 1; j >= 0; --j) at = key[j] == m ? uint32_t(j) : at;
      const uint32_t win = row_umin(at + 16u * uint32_t(rl));
      const uint32_t drop = win - 16u * uint32_t(rl);
#pragma unroll
      for (int j = 0; j < J; ++j) key[j] = drop == uint32_t(j) ? 0u : key[j];
      mine = rl == r && m != 0u ? win : mine;
    }
    __builtin_amdgcn_wave_barrier();
    const int e = mine != ~0u ? int(mine >> 4) * n + int(mine & 15u) : -1;
    float w = 0.f;
    if (e >= 0) {
      w = cs[wave][mine & 15u][16 * rt + int(mine >> 4)];
      if constexpr (!SIGMOID) w = prob(w);
    }
    if (a.renorm) {
      const float sum = sum16(w);
      w = sum == 0.f ? 0.f : w / sum;             // a NaN stays one
    }
    __builtin_amdgcn_wave_barrier();
    if (rl < k && live) {
      a.topk[tok * k + rl] = e;   // t·k is below 2^30
      a.weights[tok * k + rl] = w * a.scale;
      if (e >= 0) atomicAdd(&lds.count[e], 1);
      if constexpr (ONE) chosen[(tok - t0) * k + rl] = e;
    }
  }
  finish<WAVES, ONE>(a, lds, chosen, chunk, t0, t1);
}

// A wave a token, J experts a lane; ONE: all tokens are one chunk, and the workgroup
// groups them itself.
template <int WAVES, int J, bool BF16, bool SIGMOID, bool ONE>
__global__ __launch_bounds__(64 * WAVES) void topk_kernel(TopkArgs a, int chunk) {
  __shared__ TopkLds<WAVES> lds;
  __shared__ float cs[WAVES][64 * J];            // a wave's scores by expert
  __shared__ int32_t chosen[ONE ? kTopkChunk * kRouteMaxK : 1];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = int64_t(blockIdx.x) * chunk, t1 = min(a.t, t0 + chunk);
  const int ne = a.ne, k = a.k;
  const TopkRule rule = topk_rule<J, SIGMOID>(ne, k, a.bias != nullptr, a.groups, a.keep, a.top2, a.renorm);
  const int gs = rule.gs, per = rule.per;

  lds.count[tid] = 0;
  // What a lane's experts need for every token is kept where the registers allow it.
  constexpr bool kKeep = J <= 8;
  int base = J * lane;                            // the lane's first expert
  auto bias_of = [&](int j) { return a.bias ? a.bias[min(base + j, ne - 1)] : 0.f; };
  auto first_lane = [&](int j) { return min(base + j, ne - 1) / gs * per; };   // of the expert's group
  float bias[J];
  int gid[J];
  if constexpr (kKeep) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      bias[j] = bias_of(j);
      gid[j] = first_lane(j);
    }
  }
  float next[J];
  auto load = [&](int64_t tok) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = base + j;
      const float v = logit<BF16>(a.logits, tok * a.ld + min(e, ne - 1));
      next[j] = e < ne ? v : -INFINITY;
    }
  };
  if (kKeep && t0 + wave < t1) load(t0 + wave);
  __syncthreads();

  for (int64_t tok = t0 + wave; tok < t1; tok += WAVES) {
    float l[1][J];
    if constexpr (!kKeep) {
      asm volatile("" : "+v"(base));              // what hangs on it is not kept from token to token
      load(tok);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) l[0][j] = next[j];
    if (kKeep && tok + WAVES < t1) load(tok + WAVES);
    TopkChoice choice[1];
    topk_wave<J, SIGMOID, false>(l, rule, [&](int j) { return kKeep ? bias[j] : bias_of(j); },
                                 [&](int j) { return kKeep ? gid[j] : first_lane(j); }, cs[wave], choice);
    const int mine_e = choice[0].expert;
    if (lane < k) {
      a.topk[tok * k + lane] = mine_e;
      a.weights[tok * k + lane] = choice[0].weight * a.scale;
      if (mine_e >= 0) atomicAdd(&lds.count[mine_e], 1);
      if constexpr (ONE) chosen[(tok - t0) * k + lane] = mine_e;
    }
  }
  finish<WAVES, ONE>(a, lds, chosen, chunk, t0, t1);
}

__global__ __launch_bounds__(64 * kTopkWaves) void topk_place_kernel(
    const int32_t* __restrict__ topk, int64_t t, int ne, int k, int chunk, const int32_t* __restrict__ counts,
    int32_t* __restrict__ seg_expert, int32_t* __restrict__ seg_offsets, int32_t* __restrict__ row_index,
    int32_t* __restrict__ slot_row) {
  constexpr int kThreads = 64 * kTopkWaves;
  __shared__ TopkLds<kTopkWaves> lds;
  const int tid = threadIdx.x, chunks = gridDim.x, me = blockIdx.x;
  // counts of all chunks and of those before this one; the threads go over the
  // chunks in as many parts as the experts leave room for, 8 loads in flight
  lds.count[tid] = 0;
  lds.first[tid] = 0;
  __syncthreads();
  if (!counts) {
    for (int i = tid; i < int(t) * k; i += kThreads)
      if (topk[i] >= 0) atomicAdd(&lds.count[topk[i]], 1);
  } else if (topk_bytes(chunk)) {
    // four experts a thread, in sums of 16 bits (256 chunks of at most 128)
    const int words = (ne + 3) / 4, parts = kThreads / words;
    const int e = tid % words, part = tid / words;
    const uint32_t* row = reinterpret_cast<const uint32_t*>(counts) + e;
    if (part < parts) {
      uint32_t before[2] = {0, 0}, all[2] = {0, 0};
      for (int c0 = part; c0 < chunks; c0 += 16 * parts) {
        uint32_t v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) v[u] = row[int64_t(min(c0 + u * parts, chunks - 1)) * words];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int c = c0 + u * parts;
          const uint32_t lo = c < chunks ? v[u] & 0x00FF00FFu : 0u, hi = c < chunks ? v[u] >> 8 & 0x00FF00FFu : 0u;
          all[0] += lo;
          all[1] += hi;
          before[0] += c < me ? lo : 0u;
          before[1] += c < me ? hi : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        atomicAdd(&lds.count[4 * e + i], int(all[i & 1] >> (8 * (i & 2)) & 0xFFFFu));
        atomicAdd(&lds.first[4 * e + i], int(before[i & 1] >> (8 * (i & 2)) & 0xFFFFu));
      }
    }
  } else {
    const int span = (ne + 63) / 64 * 64, parts = kThreads / span;
    const int e = tid % span, part = tid / span;
    if (e < ne && part < parts) {
      int before = 0, all = 0;
      for (int c0 = part; c0 < chunks; c0 += 8 * parts) {
        int v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = counts[int64_t(min(c0 + u * parts, chunks - 1)) * ne + e];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int c = c0 + u * parts;
          before += c < me ? v[u] : 0;
          all += c < chunks ? v[u] : 0;
        }
      }
      atomicAdd(&lds.count[e], all);
      atomicAdd(&lds.first[e], before);
    }
  }
  __syncthreads();
  int total;
  const int at = block_scan<kTopkWaves>(lds.count[tid], lds.wsum, &total);
  lds.first[tid] += at;
  if (me == 0) {
    if (tid < ne) {
      seg_expert[tid] = tid;
      seg_offsets[tid] = at;
    }
    if (tid == 0) seg_offsets[ne] = total;
  }
  for (int64_t i = total + int64_t(me) * kThreads + tid; i < t * k; i += int64_t(chunks) * kThreads)
    row_index[i] = -1;
  const int64_t t0 = int64_t(me) * chunk;
  place_rows(lds, topk + t0 * k, t0, min(t, t0 + chunk), k, row_index, slot_row);
}

// `one` (with its waves) for a single chunk.  Otherwise `more` for every chunk, and a
// second kernel places the rows; up to kTopkChunk tokens it counts the ids itself.
using TopkKernel = void (*)(TopkArgs, int);
struct TopkLaunch {
  TopkKernel kernel;
  int waves;
};
int go(const TopkArgs& a, TopkLaunch one, TopkLaunch more, int64_t chunk, hipStream_t s) {
  const unsigned chunks = a.t <= chunk ? 1u : unsigned((a.t + chunk - 1) / chunk);   // no tokens: the tables alone
  const ProfileEvents pe = take_profile_events();
  const hipEvent_t ev0 = static_cast<hipEvent_t>(pe.start), ev1 = static_cast<hipEvent_t>(pe.stop);
  if (chunks == 1) {
    hipExtLaunchKernelGGL(one.kernel, dim3(1), dim3(64 * one.waves), 0, s, ev0, ev1, 0, a, int(chunk));
    return int(hipGetLastError());
  }
  hipExtLaunchKernelGGL(more.kernel, dim3(chunks), dim3(64 * more.waves), 0, s, ev0, nullptr, 0, a, int(chunk));
  const int err = int(hipGetLastError());
  if (err) return err;
  const bool count = a.t <= kTopkChunk;
  hipExtLaunchKernelGGL(topk_place_kernel, dim3(count ? 1u : chunks), dim3(64 * kTopkWaves), 0, s, nullptr, ev1, 0,
                        static_cast<const int32_t*>(a.topk), a.t, a.ne, a.k, int(count ? kTopkChunk : chunk),
                        static_cast<const int32_t*>(count ? nullptr : a.ws), a.seg_expert, a.seg_offsets, a.row_index,
                        a.slot_row);
  return int(hipGetLastError());
}

// J experts a lane of a row.  Chunks of 16 tokens take four waves (256 experts, 32
// tokens: 11 us, 15 with sixteen), longer ones sixteen.
template <int J, bool BF16, bool SIGMOID>
int go_row(const TopkArgs& a, int64_t chunk, hipStream_t s) {
  constexpr int W = kTopkWaves;
  const TopkLaunch one = a.t <= 16 ? TopkLaunch{topk_row_kernel<4, J, BF16, SIGMOID, true>, 4}
                                   : TopkLaunch{topk_row_kernel<W, J, BF16, SIGMOID, true>, W};
  const TopkLaunch more = chunk <= 16 ? TopkLaunch{topk_row_kernel<4, J, BF16, SIGMOID, false>, 4}
                                      : TopkLaunch{topk_row_kernel<W, J, BF16, SIGMOID, false>, W};
  return go(a, one, more, chunk, s);
}

template <bool BF16, bool SIGMOID>
int go(const TopkArgs& a, hipStream_t s) {
  constexpr int W = kTopkWaves;
  int64_t chunk = topk_chunk(a.t, a.ne);
  // One workgroup for up to 128 tokens, or more of them and a second launch where
  // its passes take longer than that (256 experts, 32 tokens: 15.1 us in one, 10.6 in
  // two, 128 tokens 26.9 and 11.1; 896 experts, 75 tokens, k = 3, 64 and 15; 60
  // experts, 128 tokens 9.6 and 9.5).
  if (a.t <= kTopkChunk && a.t * a.ne >= 8192) chunk = 16;
  if (a.ne <= 256 && a.k <= kTopkRowMaxK) {
    // Few tokens of many experts: a wave each (256 experts, 1 token: 5.8 us, 7.6 with
    // rows; 8 tokens: 8.9, 7.7).
    if (a.ne > 128 && a.t <= 4) {
      const TopkLaunch wave{topk_kernel<4, 4, BF16, SIGMOID, true>, 4};
      return go(a, wave, wave, chunk, s);
    }
    if (a.ne <= 64) return go_row<4, BF16, SIGMOID>(a, chunk, s);
    if (a.ne <= 128) return go_row<8, BF16, SIGMOID>(a, chunk, s);
    return go_row<16, BF16, SIGMOID>(a, chunk, s);
  }
  if (a.ne <= 512)
    return go(a, {topk_kernel<W, 8, BF16, SIGMOID, true>, W}, {topk_kernel<W, 8, BF16, SIGMOID, false>, W}, chunk, s);
  return go(a, {topk_kernel<W, 16, BF16, SIGMOID, true>, W}, {topk_kernel<W, 16, BF16, SIGMOID, false>, W}, chunk, s);
}

// Weighted sum of the chosen experts' rows, one workgroup per token and 2048
// columns: out = Σ_j weights[j]·o[slot_row[j]] (+ shared), in slot order, fp32,
// rounded once.  Bound by the reads of o; the rows are known before the first
// load, so all of a token's loads are in flight together (8 slots at a time).  4096
// tokens, 8 slots of 3584: 40 us by itself (6.6 TB/s, a part of o from the Infinity
// Cache), 46 after the product that writes o (5.7).
__global__ __launch_bounds__(256) void gather_kernel(GatherArgs a, int64_t first) {
  const int64_t tok = first + blockIdx.x;
  const int c8 = blockIdx.y * 256 + threadIdx.x;
  if (c8 >= a.d / 8) return;
  const int32_t* rows = a.slot_row + tok * a.k;
  const float* ws = a.weights + tok * a.k;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  bool bad = false;
  for (int j0 = 0; j0 < a.k; j0 += 8) {
    u32x4_t v[8];
    float w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int r = j0 + u < a.k ? rows[j0 + u] : -1;
      bad |= r >= a.m_total;
      const bool live = r >= 0 && r < a.m_total;
      w[u] = live ? ws[j0 + u] : 0.f;
      v[u] = live ? load16(a.o + int64_t(r) * a.d + 8 * c8) : u32x4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        acc[2 * q] = __builtin_fmaf(w[u], bf16_lo(v[u][q]), acc[2 * q]);
        acc[2 * q + 1] = __builtin_fmaf(w[u], bf16_hi(v[u][q]), acc[2 * q + 1]);
      }
  }
  if (a.shared) {
    const u32x4_t v = load16(a.shared + tok * a.d + 8 * c8);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      acc[2 * q] += bf16_lo(v[q]);
      acc[2 * q + 1] += bf16_hi(v[q]);
    }
  }
  u32x4_t o;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = bad ? 0x7FC07FC0u : pack_bf16x2(acc[2 * q], acc[2 * q + 1]);
  *reinterpret_cast<u32x4_t*>(a.out + tok * a.d + 8 * c8) = o;
}

}  // namespace

int launch_topk(const TopkArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.sigmoid) return a.bf16 ? go<true, true>(a, s) : go<false, true>(a, s);
  return a.bf16 ? go<true, false>(a, s) : go<false, false>(a, s);
}

int launch_gather(const GatherArgs& a, void* stream) {
  return launch_rows(gather_kernel, a, a.t, unsigned((a.d / 8 + 255) / 256), 256, static_cast<hipStream_t>(stream));
}

}  // namespace qmm
