// Norms before and after a block, with the block's gate and the residual scale,
// in one pass over the rows:
//
//   u = o·rsqrt(mean(o²) + eps)·(w_offset + post_w)     (u = o without post_w)
//   v = res_scale·r + gate·u                            (the new residual row)
//   h = v·rsqrt(mean(v²) + eps)·(w_offset + pre_w)      (the next block's input)
//
// A workgroup holds one row in registers (8 elements a lane and step), so o and
// r are read once and v and h are written once: bound by memory for many rows,
// by the two sums over the row for a few.  Everything between the loads and the
// stores is fp32; h is made from v before v is rounded for the store, and the
// e4m3 codes from h before h is rounded.  8192 x 5120 with gate and both outputs: 76.7 us
// (74 us for its bytes at the rate of a copy); 1 x 5120: 4.1 us.  At most 128 registers,
// for four waves on a SIMD (1000 x 13824: 26.7 us, 32.9 with the 130 of three waves).
#include <hip/hip_runtime.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"
#include "qmm_launch.h"

namespace qmm {
namespace {

struct F8 {
  float f[8];
};

__device__ __forceinline__ F8 widen(const u32x4_t v) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.f[2 * i] = bf16_lo(v[i]);
    r.f[2 * i + 1] = bf16_hi(v[i]);
  }
  return r;
}

__device__ __forceinline__ u32x4_t narrow(const F8& v) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = pack_bf16x2(v.f[2 * i], v.f[2 * i + 1]);
  return r;
}

__device__ __forceinline__ F8 load_f32x8(const float* p) {
  const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(p + 4);
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.f[i] = a[i];
    r.f[4 + i] = b[i];
  }
  return r;
}

// Sum over the workgroup, the same in every lane: a tree in each wave, then
// the waves' sums in wave order.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = sum16(v);
  const int i = __float_as_int(v);
  float s = (__int_as_float(__builtin_amdgcn_readlane(i, 0)) + __int_as_float(__builtin_amdgcn_readlane(i, 16))) +
            (__int_as_float(__builtin_amdgcn_readlane(i, 32)) + __int_as_float(__builtin_amdgcn_readlane(i, 48)));
  if constexpr (WAVES == 1) return s;
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) s += lds[w];
  return s;
}

// One row a workgroup, V groups of 8 elements a lane.  Up to 16384 columns every
// load of the row is issued before the first sum, so a row waits for memory once
// (beyond, the registers do not hold them).
template <int WAVES, int V, bool RF32>
__global__ __launch_bounds__(64 * WAVES, 4) void norm_kernel(NormArgs a, int64_t first) {
  __shared__ float sums[2][WAVES];
  constexpr bool kEarly = WAVES * V <= 32;
  const int64_t row = first + blockIdx.x;
  const int n8 = a.d >> 3;
  const float inv_d = 1.0f / float(a.d);
  const u32x4_t zero = {0, 0, 0, 0};
  const uint16_t* o = a.o ? a.o + row * a.ldo : nullptr;
  const uint16_t* g = a.gate ? a.gate + row / a.gate_rows * a.ldg : nullptr;
  auto at = [&](int j) { return int(threadIdx.x) + 64 * WAVES * j; };
  auto load = [&](const uint16_t* p, int j) { return p && at(j) < n8 ? load16(p + 8 * at(j)) : zero; };
  auto load_r = [&](int j) {
    F8 r = widen(zero);
    if (at(j) < n8) {
      if constexpr (RF32)
        r = load_f32x8(static_cast<const float*>(a.r) + row * a.ldr + 8 * at(j));
      else
        r = widen(load16(static_cast<const uint16_t*>(a.r) + row * a.ldr + 8 * at(j)));
    }
    return r;
  };
  u32x4_t ov[V], wv[V], gv[V], pv[V];
  F8 rv[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    ov[j] = load(o, j);
    if constexpr (kEarly) {
      rv[j] = load_r(j);
      wv[j] = load(a.post_w, j);
      gv[j] = load(g, j);
      pv[j] = load(a.pre_w, j);
    }
  }
  // the block's output, its norm and its gate
  F8 v[V];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    v[j] = widen(ov[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[j].f[e], v[j].f[e], ss);
  }
  if (a.post_w) {
    const float k = 1.0f / sqrtf(block_sum<WAVES>(ss, sums[0]) * inv_d + a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const F8 w = widen(kEarly ? wv[j] : load(a.post_w, j));
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j].f[e] = v[j].f[e] * k * (a.w_offset + w.f[e]);
    }
  }
  if (g) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const F8 w = widen(kEarly ? gv[j] : load(g, j));
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j].f[e] *= w.f[e];
    }
  }
  // the residual
  ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const F8 r = kEarly ? rv[j] : load_r(j);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[j].f[e] = __builtin_fmaf(a.res_scale, r.f[e], v[j].f[e]);
      ss = __builtin_fmaf(v[j].f[e], v[j].f[e], ss);
    }
    if (a.r_out && at(j) < n8) {
      if constexpr (RF32) {
        float* to = static_cast<float*>(a.r_out) + row * a.ldr_out + 8 * at(j);
        *reinterpret_cast<f32x4_t*>(to) = f32x4_t{v[j].f[0], v[j].f[1], v[j].f[2], v[j].f[3]};
        *reinterpret_cast<f32x4_t*>(to + 4) = f32x4_t{v[j].f[4], v[j].f[5], v[j].f[6], v[j].f[7]};
      } else {
        *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.r_out) + row * a.ldr_out + 8 * at(j)) = narrow(v[j]);
      }
    }
  }
  if (!a.h && !a.q) return;
  // the next block's norm
  const float k = 1.0f / sqrtf(block_sum<WAVES>(ss, sums[1]) * inv_d + a.eps);
  const int nb = (a.d + kFp8Block - 1) / kFp8Block;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = at(j);
    const F8 w = widen(kEarly ? pv[j] : load(a.pre_w, j));
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j].f[e] = v[j].f[e] * k * (a.w_offset + w.f[e]);
    if (a.h && i < n8) *reinterpret_cast<u32x4_t*>(a.h + row * a.ldh + 8 * i) = narrow(v[j]);
    if (a.q) {
      // a scale block is 16 lanes; lanes past the row hold zeros
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = umax(m, __float_as_uint(v[j].f[e]) & 0x7FFFFFFFu);
      m = group_umax<16>(m);
      const BlockScale s = block_scale(m);
      if (i < n8) {
        const float f = s.factor;
        *reinterpret_cast<u32x2_t*>(a.q + row * a.d + 8 * i) =
            u32x2_t{pack_e4m3x4(v[j].f[0] * f, v[j].f[1] * f, v[j].f[2] * f, v[j].f[3] * f),
                    pack_e4m3x4(v[j].f[4] * f, v[j].f[5] * f, v[j].f[6] * f, v[j].f[7] * f)};
        if ((i & 15) == 0) a.q_scales[row * nb + (i >> 4)] = s.scale;
      }
    }
  }
}

template <int WAVES, int V>
int go(const NormArgs& a, hipStream_t s) {
  return launch_rows(a.r_f32 ? norm_kernel<WAVES, V, true> : norm_kernel<WAVES, V, false>, a, a.t, 1, 64 * WAVES, s);
}

}  // namespace

int launch_norm_residual(const NormArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const NormShape p = norm_shape(a.t, a.d);
  switch (100 * p.groups + p.waves) {
    case 101: return go<1, 1>(a, s);
    case 104: return go<4, 1>(a, s);
    case 108: return go<8, 1>(a, s);
    case 116: return go<16, 1>(a, s);
    case 304: return go<4, 3>(a, s);
    case 208: return go<8, 2>(a, s);
    case 308: return go<8, 3>(a, s);
    case 408: return go<8, 4>(a, s);
    case 416: return go<16, 4>(a, s);
    case 816: return go<16, 8>(a, s);
  }
  return int(hipErrorInvalidValue);
}

}  // namespace qmm
