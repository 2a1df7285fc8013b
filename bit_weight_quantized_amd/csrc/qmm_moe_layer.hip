// A mixture-of-experts layer for up to 16 tokens in two launches, MXFP4 weights and bf16
// activations:
//
//   1  logits -> k experts a token and their weights;  h[t,j] = silu(G_e x_t)·(U_e x_t)
//   2  out[t] = Σ_j weight[t,j]·D_e h[t,j] (+ shared[t])
//
// Bound by the chosen experts' bytes, read once each whatever the tokens.  Every workgroup
// (one a CU) makes the choice itself, a wave a token: a launch of its own would take as long
// as the layer's start.  The second kernel reads the choice that the first one's workgroup 0
// has written.  From the choice follows a table of the chosen experts, ascending, and of each
// one's tokens.
//
// Work is dealt out to waves in tasks of 16 weight rows of an expert: 8 gate rows and the 8 up
// rows of the same outputs in the first kernel, whose sums meet in registers; 16 output columns
// in the second, where a workgroup has all experts of its columns (and, where they are few, parts
// of the reduction axis), its waves' weighted sums meet in LDS in the waves' order, and nothing
// depends on timing.
//
// A wave goes through its tasks as one sequence of steps of 128 codes: weights, exponents and
// the expert's activation rows of a step come through a private LDS ring (global -> LDS, no
// registers, no barriers), the copies a whole ring ahead, across the borders of tasks.  A
// lane's 16-byte piece of weights is a block of 32 codes, converted exactly to bf16 for four
// v_mfma_f32_16x16x32_bf16 with 16 weight rows (A operand) and the tokens (B operand).
#include <hip/hip_runtime.h>

#include "qmm_device.h"
#include "qmm_fp8_device.h"
#include "qmm_fp8_tile.h"
#include "qmm_launch.h"
#include "qmm_lds_copy.h"
#include "qmm_moe_layer.h"
#include "qmm_topk_wave.h"

#include <algorithm>

namespace qmm {
namespace {

constexpr int kLayerWaves = 8;
constexpr int kLayerRing = 18 * 1024;     // a wave's ring

struct LayerTables {
  int32_t ids[kLayerMaxPairs];            // experts of the pairs (token, choice), -1: none
  float weights[kLayerMaxPairs];
  uint32_t bits[kRouteMaxExperts / 32];   // chosen experts
  uint16_t pairs[kLayerMaxPairs];         // by expert, then token
  uint16_t expert[kLayerMaxPairs];        // the chosen ones, ascending
  uint16_t first[kLayerMaxPairs + 2];     // where an expert's pairs begin
  int32_t count, most;                    // chosen experts; most tokens of one
};
constexpr int kLayerRed = kLayerWaves * kLayerRing;                    // the waves' sums
constexpr int kLayerTables = kLayerRed + kLayerWaves * 1024;
constexpr int kLayerLds = kLayerTables + int(sizeof(LayerTables));
static_assert(kLayerLds <= 160 * 1024, "LDS");

// The tables from ids, by a thread for each pair; every thread of the workgroup calls it.
__device__ __forceinline__ void make_tables(LayerTables& T, int pairs) {
  const int tid = threadIdx.x;
  if (tid < kRouteMaxExperts / 32) T.bits[tid] = 0u;
  if (tid == 0) T.most = 0;
  __syncthreads();
  const int e = tid < pairs ? T.ids[tid] : -1;
  if (e >= 0) atomicOr(&T.bits[e >> 5], 1u << (e & 31));
  __syncthreads();
  int before = 0, same = 0, all = 0, valid = 0;   // pairs that come before, of this expert before and at all
  for (int q = 0; q < pairs; ++q) {
    const int o = T.ids[q];
    before += o >= 0 && (o < e || (o == e && q < tid)) ? 1 : 0;
    same += o == e && q < tid ? 1 : 0;
    all += o == e ? 1 : 0;
    valid += o >= 0 ? 1 : 0;
  }
  int rank = 0, count = 0;
  for (int w = 0; w < kRouteMaxExperts / 32; ++w) {
    const uint32_t b = T.bits[w];
    count += __builtin_popcount(b);
    rank += w < e >> 5 ? __builtin_popcount(b) : w == e >> 5 ? __builtin_popcount(b & ((1u << (e & 31)) - 1u)) : 0;
  }
  if (e >= 0) {
    T.pairs[before] = uint16_t(tid);
    if (same == 0) {
      T.expert[rank] = uint16_t(e);
      T.first[rank] = uint16_t(before);
      atomicMax(&T.most, all);
    }
  }
  if (tid == 0) {
    T.count = count;
    T.first[count] = uint16_t(valid);
  }
  __syncthreads();
}

// One wave's choice for one token.
template <int J, bool SIGMOID>
__device__ __forceinline__ void choose(const MoeLayerArgs& a, int tok, float* mine, LayerTables& T) {
  const int lane = threadIdx.x & 63;
  const TopkRule rule = topk_rule<J, SIGMOID>(a.n_experts, a.k, a.bias != nullptr, a.groups, a.keep, a.top2, a.renorm);
  float l[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int e = J * lane + j;
    const int64_t at = int64_t(tok) * a.ld + min(e, a.n_experts - 1);
    const float v = a.bf16 ? logit<true>(a.logits, at) : logit<false>(a.logits, at);
    l[j] = e < a.n_experts ? v : -INFINITY;
  }
  const TopkChoice c = topk_wave<J, SIGMOID>(
      l, rule, [&](int j) { return a.bias ? a.bias[min(J * lane + j, a.n_experts - 1)] : 0.f; },
      [&](int j) { return min(J * lane + j, a.n_experts - 1) / rule.gs * rule.per; }, mine);
  if (lane < a.k) {
    T.ids[tok * a.k + lane] = c.expert;
    T.weights[tok * a.k + lane] = c.weight * a.scale;
  }
}

// 16-byte pieces of a row of 128 activations lie in LDS at piece ^ spread(row): 16 lanes that
// an LDS read serves at once (rows 0..3, 12..15 of one piece, 4..11 of the fourth after it)
// are then in different banks.
__device__ __forceinline__ int spread(int row) { return (row & 7) | ((row >> 3 ^ row >> 2) & 1) << 3; }

// The steps of a wave.  AC copies of 4 activation rows a step.
template <bool DOWN, int AC>
__device__ __forceinline__ void stream(const MoeLayerArgs& a, unsigned char* lds, LayerTables& T) {
  constexpr int kStage = 1024 + 1024 * AC + 256, D = kLayerRing / kStage, kOps = 2 + AC;
  static_assert((D - 1) * kOps <= 63, "the waits count the copies in flight");
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int axis = DOWN ? a.inter : a.d, n = DOWN ? a.d : 2 * a.inter;
  const int steps = (axis + 127) / 128, nd = __builtin_amdgcn_readfirstlane(T.count);
  const Slabs L{n, axis, QMM_MXFP4_G32};
  const int last = L.count() - 1;
  const uint32_t width = uint32_t(L.width(0) / 2), width_last = uint32_t(L.width(last) / 2);
  const uint32_t mrow = uint32_t(L.meta_row(0)), mrow_last = uint32_t(L.meta_row(last)), mquad = uint32_t(L.meta_quad());
  const uint32_t slab_bytes = uint32_t(n) * (kSlabCodes / 2);   // of a slab that another follows
  const uint32_t codes_bytes = uint32_t(n) * (uint32_t(axis) / 2), meta_bytes = (uint32_t(n) + 3) / 4 * mquad;
  const int64_t meta_offset = (kHeaderBytes + int64_t(codes_bytes) + 255) / 256 * 256;
  const uint8_t* stack = DOWN ? a.down : a.gate_up;
  const int64_t stride = DOWN ? a.down_stride : a.gate_up_stride;
  const uint32_t row_bytes = uint32_t(axis) * 2u;
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(DOWN ? a.h : a.x, uint32_t(DOWN ? a.t * a.k : a.t) * row_bytes);
  unsigned char* ring = lds + wave * kLayerRing;
  const uint32_t ring_at = lds_addr(ring);

  // Tasks.  First kernel: an expert and 8 outputs, dealt out to all waves of the grid, those of
  // a CU far apart.  Second: for each block of 16 columns of the workgroup all experts, each in
  // `parts` parts, so that the waves have like shares.
  const int blocks = DOWN ? a.d / 16 : a.inter / 8;
  int parts = 1;
  if (DOWN)
    while (2 * parts <= min(8, steps) && (nd * parts + 7) / 8 * 8 * 20 > 23 * nd * parts) parts *= 2;
  const int rounds = DOWN ? (blocks - int(blockIdx.x) + int(gridDim.x) - 1) / int(gridDim.x) : 1;
  const int of_round = DOWN ? nd * parts : nd * blocks, stride_of = DOWN ? kLayerWaves : kLayerWaves * int(gridDim.x);
  const int begin = DOWN ? wave : wave * int(gridDim.x) + int(blockIdx.x);
  struct Task {
    int j, block, from, to;
  };
  auto task_of = [&](int round, int i) {
    if (DOWN) {
      const int j = i / parts, p = i - j * parts;
      return Task{j, int(blockIdx.x) + round * int(gridDim.x), steps * p / parts, steps * (p + 1) / parts};
    }
    const int j = i / blocks;
    return Task{j, i - j * blocks, 0, steps};
  };

  // ---- the copies' place in the sequence
  const int wrow = lane >> 2, wpiece = (lane & 3) ^ (wrow >> 1 & 3);
  int c_round = 0, c_task = begin, c_h = 0, c_to = 0;
  __amdgpu_buffer_rsrc_t cr = make_rsrc(stack, 0), mr = cr;
  uint32_t w_full = 0, w_last = 0, m_full = 0, m_last = 0, aoff[AC];
#pragma unroll
  for (int i = 0; i < AC; ++i) aoff[i] = kOOB8;
  auto packed_row = [&](int block, int row) {
    return DOWN ? 16 * block + row : 8 * block + (row & 7) + (row >= 8 ? a.inter : 0);
  };
  auto open = [&]() {
    const Task t = task_of(c_round, c_task);
    int e = __builtin_amdgcn_readfirstlane(T.expert[t.j]), at = __builtin_amdgcn_readfirstlane(T.first[t.j]);
    int end = __builtin_amdgcn_readfirstlane(T.first[t.j + 1]);
    // wait states between these, which vector instructions write, and the copies that read what follows from them
    asm volatile("s_nop 4" : "+s"(e), "+s"(at), "+s"(end));
    const uint8_t* blob = stack + int64_t(e) * stride;
    cr = make_rsrc(blob + kHeaderBytes, codes_bytes);
    mr = make_rsrc(blob + meta_offset, meta_bytes);
    const uint32_t row = uint32_t(packed_row(t.block, wrow)), row_m = uint32_t(packed_row(t.block, c));
    w_full = row * width + 16u * uint32_t(wpiece);
    w_last = row * width_last + 16u * uint32_t(wpiece);
    m_full = lane < 16 ? (row_m >> 2) * mquad + (row_m & 3u) * mrow : kOOB8;
    m_last = lane < 16 ? (row_m >> 2) * mquad + (row_m & 3u) * mrow_last : kOOB8;
#pragma unroll
    for (int i = 0; i < AC; ++i) {
      const int r = 4 * i + (lane >> 4), p = T.pairs[min(at + r, kLayerMaxPairs - 1)];
      aoff[i] = at + r < end ? uint32_t(DOWN ? p : p / a.k) * row_bytes + 16u * uint32_t((lane & 15) ^ spread(r)) : kOOB8;
    }
    c_h = t.from;
    c_to = t.to;
  };
  auto copies = [&](int stage) {
    const bool in = c_round < rounds && c_task < of_round;
    const int h = c_h, s = h >> 2;
    const uint32_t at = ring_at + uint32_t(stage * kStage), none = in ? 0u : kOOB8;
    copy16_to_lds_from(cr, (s == last ? w_last : w_full) | none | (128 * h + 32 * wpiece < axis ? 0u : kOOB8),
                       in ? uint32_t(s) * slab_bytes + 64u * uint32_t(h & 3) : 0u, at);
#pragma unroll
    for (int i = 0; i < AC; ++i)
      copy16_to_lds_from(ar, aoff[i] | none | (128 * h + 8 * ((lane & 15) ^ spread(4 * i + (lane >> 4))) < axis ? 0u : kOOB8),
                         in ? 256u * uint32_t(h) : 0u, at + 1024u + 1024u * uint32_t(i));
    copy4_to_lds(mr, ((s == last ? m_last : m_full) + 64u * uint32_t(s) + 4u * uint32_t(h & 3)) | none,
                 at + 1024u + 1024u * AC);
    if (in && ++c_h == c_to) {
      c_task += stride_of;
      if (c_task >= of_round) {
        c_task = begin;
        ++c_round;
      }
      if (c_round < rounds && c_task < of_round) open();
    }
  };
  if (rounds > 0 && begin < of_round) open();
#pragma unroll 1
  for (int i = 0; i < D; ++i) copies(i);

  int stage = 0;
  f32x4_t* red = reinterpret_cast<f32x4_t*>(lds + kLayerRed);
  for (int round = 0; round < rounds; ++round) {
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};           // token c, columns 4g .. 4g + 3
    for (int i = begin; i < of_round; i += stride_of) {
      const Task t = task_of(round, i);
      const int at = T.first[t.j], rows = T.first[t.j + 1] - at;
      // the lane's pair, and its row in LDS: the c-th of the expert's, or token c's
      int row = min(c, rows - 1), pair = -1;
      if (DOWN) {
        row = 0;
        for (int r = 0; r < rows; ++r) {
          const int p = T.pairs[at + r];
          if (p / a.k == c) {
            row = r;
            pair = p;
          }
        }
      } else if (c < rows) {
        pair = T.pairs[at + c];
      }
      const uint32_t a_at = 1024u + 256u * uint32_t(row);
      const int x0 = spread(row);
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      for (int h = t.from; h < t.to; ++h) {
        wait_copies<(D - 1) * kOps>();
        const unsigned char* st = ring + stage * kStage;
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(st + 64 * c + 16 * (g ^ (c >> 1 & 3)));
        const uint32_t e8 = st[1024 + 1024 * AC + 4 * c + g];
        u32x4_t b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const u32x4_t*>(st + a_at + 16 * ((4 * g + j) ^ x0));
        wait_reads();                             // ... and is in registers: its stage is free
        copies(stage);
        stage = stage + 1 == D ? 0 : stage + 1;
        const float scale = e8m0_scale(e8);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, mxfp4_word_to_bf16x8(w[j], scale)),
                                                        __builtin_bit_cast(bf16x8_t, b[j]), acc, 0, 0, 0);
      }
      if (DOWN) {
        const float weight = pair >= 0 ? T.weights[pair] : 0.f;
        if (pair >= 0)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = __builtin_fmaf(weight, acc[e], sum[e]);
      } else {
        // gate rows in the lanes with g < 2, the same outputs' up rows 32 lanes on
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = silu(acc[e]) * __shfl_xor(acc[e], 32);
        if (g < 2 && pair >= 0)
          *reinterpret_cast<u32x2_t*>(a.h + int64_t(pair) * a.inter + 8 * t.block + 4 * g) =
              u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      }
    }
    if (DOWN) {
      red[64 * wave + lane] = sum;
      wait_reads();
      phase_end();
      if (wave == 0 && c < a.t) {
#pragma unroll
        for (int w = 1; w < kLayerWaves; ++w) sum += red[64 * w + lane];
        const int64_t o = int64_t(c) * a.d + 16 * (int(blockIdx.x) + round * int(gridDim.x)) + 4 * g;
        if (a.shared) {
          const u32x2_t v = *reinterpret_cast<const u32x2_t*>(a.shared + o);
          sum += f32x4_t{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
        }
        *reinterpret_cast<u32x2_t*>(a.out + o) = u32x2_t{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
      }
      wait_reads();
      phase_end();                                // the next columns' sums take the place
    }
  }
  wait_copies<0>();
}

template <bool DOWN>
__device__ __forceinline__ void stream_any(const MoeLayerArgs& a, unsigned char* lds, LayerTables& T) {
  const int most = __builtin_amdgcn_readfirstlane(T.most);
  if (most <= 4) stream<DOWN, 1>(a, lds, T);
  else if (most <= 8) stream<DOWN, 2>(a, lds, T);
  else stream<DOWN, 4>(a, lds, T);
}

__global__ __launch_bounds__(64 * kLayerWaves) void layer_gate_up_kernel(MoeLayerArgs a) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  LayerTables& T = *reinterpret_cast<LayerTables*>(lds + kLayerTables);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* mine = reinterpret_cast<float*>(lds + wave * kLayerRing);
  for (int tok = wave; tok < a.t; tok += kLayerWaves) {
    if (a.n_experts <= 256) {
      if (a.sigmoid) choose<4, true>(a, tok, mine, T);
      else choose<4, false>(a, tok, mine, T);
    } else {
      if (a.sigmoid) choose<16, true>(a, tok, mine, T);
      else choose<16, false>(a, tok, mine, T);
    }
  }
  __syncthreads();
  const int pairs = a.t * a.k, tid = threadIdx.x;
  if (blockIdx.x == 0 && tid < pairs) {
    a.topk[tid] = T.ids[tid];
    a.weights[tid] = T.weights[tid];
  }
  make_tables(T, pairs);
  stream_any<false>(a, lds, T);
}

__global__ __launch_bounds__(64 * kLayerWaves) void layer_down_kernel(MoeLayerArgs a) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  LayerTables& T = *reinterpret_cast<LayerTables*>(lds + kLayerTables);
  const int pairs = a.t * a.k, tid = threadIdx.x;
  if (tid < pairs) {
    const int e = a.topk[tid];
    T.ids[tid] = e >= 0 && e < a.n_experts ? e : -1;
    T.weights[tid] = a.weights[tid];
  }
  make_tables(T, pairs);
  stream_any<true>(a, lds, T);
}

}  // namespace

int launch_moe_layer(const MoeLayerArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  DevInfo di{};
  const int cus = device_info(&di) == 0 && di.cus > 0 ? di.cus : 256;
  const ProfileEvents pe = take_profile_events();
  const dim3 block(64 * kLayerWaves);
  const int64_t tasks = int64_t(std::min(a.n_experts, a.t * a.k)) * (a.inter / 8);
  hipExtLaunchKernelGGL(layer_gate_up_kernel, dim3(unsigned(std::min<int64_t>(cus, tasks))), block, kLayerLds, s,
                        static_cast<hipEvent_t>(pe.start), nullptr, 0, a);
  const int err = int(hipGetLastError());
  if (err) return err;
  hipExtLaunchKernelGGL(layer_down_kernel, dim3(unsigned(std::min(cus, a.d / 16))), block, kLayerLds, s, nullptr,
                        static_cast<hipEvent_t>(pe.stop), 0, a);
  return int(hipGetLastError());
}

}  // namespace qmm
