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
// One workgroup of 16 waves per chunk of tokens, one wave per token: lane i
// holds experts J·i .. J·i + J-1 as order-preserving integer keys, so the
// lowest lane and the lowest j among equal keys is the lowest expert.  A round
// takes the largest key of the wave (DPP, then scalar registers) and the
// winning lane looks for its next best.
//
// Grouping counts the chunk's tokens per expert in LDS (integer atomics, order
// free).  One chunk: the same workgroup scans the counts and places its rows.
// More: the counts go to the workspace, and a second kernel, one workgroup per
// chunk, adds up every chunk's counts (at most 128 per expert) and places the
// chunk's rows.  Rows of an expert ascend with the token, found from a bitmap
// of the chunk's tokens per expert, so nothing depends on timing.
#include <hip/hip_runtime.h>

#include <math.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"
#include "qmm_launch.h"

namespace qmm {
namespace {

constexpr int kTkThreads = 64 * kTopkWaves;
constexpr int kTkWords = kTopkChunk / 32;        // bitmap words of an expert and pass
constexpr int kTkMaxExperts = kRouteMaxExperts;  // one per thread of the workgroup
static_assert(kTkMaxExperts == kTkThreads, "a thread owns an expert");

// Order-preserving map to an unsigned key; 0 marks an expert that cannot be
// chosen: masked (-inf), NaN, or taken.
__device__ __forceinline__ uint32_t choice_key(float c) {
  const uint32_t b = __float_as_uint(c) == 0x80000000u ? 0u : __float_as_uint(c);
  const uint32_t flip = uint32_t(int32_t(b) >> 31) | 0x80000000u;
  return c > -INFINITY ? (b ^ flip) : 0u;
}

__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = group_umax<16>(v);
  const uint32_t r0 = __builtin_amdgcn_readlane(int(v), 0), r1 = __builtin_amdgcn_readlane(int(v), 16);
  const uint32_t r2 = __builtin_amdgcn_readlane(int(v), 32), r3 = __builtin_amdgcn_readlane(int(v), 48);
  return umax(umax(r0, r1), umax(r2, r3));
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

template <bool BF16>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

struct TopkLds {
  int32_t count[kTkMaxExperts];
  uint32_t bits[kTkMaxExperts][kTkWords];
  int32_t first[kTkMaxExperts];      // the next row of each expert
  int32_t wsum[kTopkWaves];
};

// Exclusive sum over the workgroup's threads; every thread gets the total too.
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
  for (int w = 0; w < kTopkWaves; ++w) {
    before += w < wave ? wsum[w] : 0;
    all += wsum[w];
  }
  *total = all;
  return before + incl - c;
}

// Writes the rows of tokens [t0, t1), whose first row of expert e is
// lds.first[e]: 128 tokens at a time, one bit per (expert, token).
__device__ void place_rows(TopkLds& lds, const int32_t* topk, int64_t t0, int64_t t1, int k,
                           int32_t* row_index, int32_t* slot_row) {
  const int tid = threadIdx.x;
  for (int64_t b0 = t0; b0 < t1; b0 += kTopkChunk) {
    const int nb = int(min(int64_t(kTopkChunk), t1 - b0)) * k;
#pragma unroll
    for (int h = 0; h < kTkWords; ++h) lds.bits[tid][h] = 0u;
    __syncthreads();
    for (int i = tid; i < nb; i += kTkThreads) {
      const int e = topk[b0 * k + i], tl = i / k;
      if (e >= 0) atomicOr(&lds.bits[e][tl >> 5], 1u << (tl & 31));
    }
    __syncthreads();
    for (int i = tid; i < nb; i += kTkThreads) {
      const int e = topk[b0 * k + i], tl = i / k;
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

// J experts a lane; ONE: all tokens are one chunk, and the workgroup groups
// them itself.
template <int J, bool BF16, bool ONE>
__global__ __launch_bounds__(kTkThreads) void topk_kernel(TopkArgs a, int chunk) {
  __shared__ TopkLds lds;
  __shared__ float cs[kTopkWaves][64 * J];       // a wave's c, for the groups' values
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t0 = int64_t(blockIdx.x) * chunk, t1 = min(a.t, t0 + chunk);
  const int ne = a.ne, k = a.k, groups = a.groups;
  const int gs = ne / groups;                     // experts of a group
  int per = 64;                                   // lanes that share a group's experts
  while (per * groups > 64) per >>= 1;
  const bool by_logit = !a.sigmoid && !a.bias && (groups == 1 || !a.top2);

  lds.count[tid] = 0;
  __syncthreads();
  float bias[J];
  int gid[J];                                     // first lane of the expert's group
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = J * lane + j;
    bias[j] = a.bias && e < ne ? a.bias[e] : 0.f;
    gid[j] = e < ne ? e / gs * per : 0;
  }

  for (int64_t tok = t0 + wave; tok < t1; tok += kTopkWaves) {
    float l[J], c[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = J * lane + j;
      l[j] = e < ne ? logit<BF16>(a.logits, tok * a.ld + e) : -INFINITY;
    }
    float top = 0.f, total = 1.f;
    if (!a.sigmoid) {
      float m = l[0];
#pragma unroll
      for (int j = 1; j < J; ++j) m = fmaxf(m, l[j]);
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o));
      top = m > -INFINITY ? m : 0.f;              // nothing left: every e^(l - top) is 0
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) z += expf(l[j] - top);
      total = wave_sum(z);
    }
    auto prob = [&](float v) { return a.sigmoid ? sigmoid(v) : total > 0.f ? expf(v - top) / total : total; };
#pragma unroll
    for (int j = 0; j < J; ++j) {
      c[j] = by_logit ? l[j] : prob(l[j]) + bias[j];
      if (l[j] == -INFINITY) c[j] = -INFINITY;
    }
    uint32_t key[J];
#pragma unroll
    for (int j = 0; j < J; ++j) key[j] = choice_key(c[j]);

    if (groups > 1) {
      // the groups' values: `per` lanes each, their best (two) merged
      float* mine = cs[wave];
#pragma unroll
      for (int j = 0; j < J; ++j) mine[J * lane + j] = key[j] ? c[j] : -INFINITY;
      __builtin_amdgcn_wave_barrier();
      const int q = lane / per;
      float b1 = -INFINITY, b2 = -INFINITY;
      if (q < groups)
        for (int i = lane - q * per; i < gs; i += per) {
          const float v = mine[q * gs + i];
          b2 = fmaxf(b2, fminf(b1, v));
          b1 = fmaxf(b1, v);
        }
      for (int o = 1; o < per; o <<= 1) {
        const float o1 = __shfl_xor(b1, o), o2 = __shfl_xor(b2, o);
        b2 = fmaxf(fmaxf(b2, o2), fminf(b1, o1));
        b1 = fmaxf(b1, o1);
      }
      const float value = a.top2 && b2 > -INFINITY ? b1 + b2 : b1;
      // rank among the groups: larger values first, equal ones by index
      int rank = 0;
      for (int o = 0; o < groups; ++o) {
        const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(value), o * per));
        rank += v > value || (v == value && o < q) ? 1 : 0;
      }
      const uint64_t kept = __ballot(q < groups && rank < a.keep);
#pragma unroll
      for (int j = 0; j < J; ++j) key[j] = (kept >> gid[j]) & 1 ? key[j] : 0u;
      __builtin_amdgcn_wave_barrier();
    }

    int mine_e = -1;
    for (int r = 0; r < k; ++r) {
      uint32_t bk = key[0];
      int be = J * lane;
#pragma unroll
      for (int j = 1; j < J; ++j) {
        const bool gt = key[j] > bk;
        bk = gt ? key[j] : bk;
        be = gt ? J * lane + j : be;
      }
      const uint32_t m = wave_umax(bk);
      if (m == 0) break;                          // nothing left (uniform)
      const int first = __builtin_ctzll(__ballot(bk == m));
      const int win = __builtin_amdgcn_readlane(be, first);
#pragma unroll
      for (int j = 0; j < J; ++j) key[j] = J * lane + j == win ? 0u : key[j];
      mine_e = lane == r ? win : mine_e;
    }
    // the weights, from the logits of the chosen
    float w = 0.f;
    if (mine_e >= 0) w = prob(logit<BF16>(a.logits, tok * a.ld + mine_e));
    if (a.renorm) {
      const float sum = wave_sum(w);
      w = sum == 0.f ? 0.f : w / sum;             // a NaN stays one
    }
    if (lane < k) {
      a.topk[tok * k + lane] = mine_e;
      a.weights[tok * k + lane] = w * a.scale;
      if (mine_e >= 0) atomicAdd(&lds.count[mine_e], 1);
    }
  }
  __syncthreads();                                // counts; the ids of the chunk
  if constexpr (!ONE) {
    if (tid < ne) a.ws[int64_t(blockIdx.x) * ne + tid] = lds.count[tid];
  } else {
    int total;
    const int at = block_scan(lds.count[tid], lds.wsum, &total);
    lds.first[tid] = at;
    if (tid < ne) {
      a.seg_expert[tid] = tid;
      a.seg_offsets[tid] = at;
    }
    if (tid == 0) a.seg_offsets[ne] = total;
    for (int64_t i = total + tid; i < a.t * k; i += kTkThreads) a.row_index[i] = -1;
    place_rows(lds, a.topk, t0, t1, k, a.row_index, a.slot_row);
  }
}

__global__ __launch_bounds__(kTkThreads) void topk_place_kernel(const int32_t* __restrict__ topk, int64_t t, int ne,
                                                                int k, int chunk, const int32_t* __restrict__ counts,
                                                                int32_t* __restrict__ seg_expert,
                                                                int32_t* __restrict__ seg_offsets,
                                                                int32_t* __restrict__ row_index,
                                                                int32_t* __restrict__ slot_row) {
  __shared__ TopkLds lds;
  const int tid = threadIdx.x, chunks = gridDim.x, me = blockIdx.x;
  int before = 0, all = 0;
  if (tid < ne) {
    // 8 loads in flight
    int c0 = 0;
    for (; c0 + 8 <= chunks; c0 += 8) {
      int v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = counts[int64_t(c0 + u) * ne + tid];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        before += c0 + u < me ? v[u] : 0;
        all += v[u];
      }
    }
    for (; c0 < chunks; ++c0) {
      const int v = counts[int64_t(c0) * ne + tid];
      before += c0 < me ? v : 0;
      all += v;
    }
  }
  int total;
  const int at = block_scan(all, lds.wsum, &total);
  lds.first[tid] = at + before;
  if (me == 0) {
    if (tid < ne) {
      seg_expert[tid] = tid;
      seg_offsets[tid] = at;
    }
    if (tid == 0) seg_offsets[ne] = total;
  }
  for (int64_t i = total + int64_t(me) * kTkThreads + tid; i < t * k; i += int64_t(chunks) * kTkThreads)
    row_index[i] = -1;
  const int64_t t0 = int64_t(me) * chunk;
  place_rows(lds, topk, t0, min(t, t0 + chunk), k, row_index, slot_row);
}

template <int J, bool BF16>
int go(const TopkArgs& a, hipStream_t s) {
  const int64_t chunk = topk_chunk(a.t);
  const unsigned chunks = a.t <= chunk ? 1u : unsigned((a.t + chunk - 1) / chunk);   // no tokens: the tables alone
  const ProfileEvents pe = take_profile_events();
  const hipEvent_t ev0 = static_cast<hipEvent_t>(pe.start), ev1 = static_cast<hipEvent_t>(pe.stop);
  if (chunks == 1) {
    hipExtLaunchKernelGGL((topk_kernel<J, BF16, true>), dim3(1), dim3(kTkThreads), 0, s, ev0, ev1, 0, a, int(chunk));
    return int(hipGetLastError());
  }
  hipExtLaunchKernelGGL((topk_kernel<J, BF16, false>), dim3(chunks), dim3(kTkThreads), 0, s, ev0, nullptr, 0, a,
                        int(chunk));
  const int err = int(hipGetLastError());
  if (err) return err;
  hipExtLaunchKernelGGL(topk_place_kernel, dim3(chunks), dim3(kTkThreads), 0, s, nullptr, ev1, 0,
                        static_cast<const int32_t*>(a.topk), a.t, a.ne, a.k, int(chunk),
                        static_cast<const int32_t*>(a.ws), a.seg_expert, a.seg_offsets, a.row_index, a.slot_row);
  return int(hipGetLastError());
}

template <int J>
int go(const TopkArgs& a, hipStream_t s) {
  return a.bf16 ? go<J, true>(a, s) : go<J, false>(a, s);
}

// Weighted sum of the chosen experts' rows, one workgroup per token and 2048
// columns: out = Σ_j weights[j]·o[slot_row[j]] (+ shared), in slot order, fp32,
// rounded once.  Bound by the reads of o; the rows are known before the first
// load, so all of a token's loads are in flight together (8 slots at a time).
__global__ __launch_bounds__(256) void gather_kernel(GatherArgs a) {
  const int64_t tok = blockIdx.x;
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
    o[q] = bad ? 0x7FC07FC0u
               : uint32_t(f32_to_bf16(acc[2 * q])) | uint32_t(f32_to_bf16(acc[2 * q + 1])) << 16;
  *reinterpret_cast<u32x4_t*>(a.out + tok * a.d + 8 * c8) = o;
}

}  // namespace

int launch_topk(const TopkArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.ne <= 64) return go<1>(a, s);
  if (a.ne <= 128) return go<2>(a, s);
  if (a.ne <= 256) return go<4>(a, s);
  if (a.ne <= 512) return go<8>(a, s);
  return go<16>(a, s);
}

int launch_gather(const GatherArgs& a, void* stream) {
  launch_kernel(gather_kernel, dim3(unsigned(a.t), unsigned((a.d / 8 + 255) / 256)), dim3(256),
                static_cast<hipStream_t>(stream), a);
  return int(hipGetLastError());
}

}  // namespace qmm
