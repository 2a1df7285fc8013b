// bf16 rows -> E2M1 codes with one E8M0 exponent for each block of 32.
//
//   m = max_b |x|;  E = floor(log2 m) - 2 + 127, or the smallest E with m <= 6·2^(E-127);
//   q = E2M1(x·2^(127-E)), nearest, ties to even, at most 6
//
// Scaling by a power of two is exact, so codes follow from x alone, bit for bit; the
// conversion instruction does scaling, rounding and saturation of a pair at once.
// Bound by memory: 2 bytes read and 1/2 + 1/32 written for each element.  A lane takes 16
// elements (two 16-byte loads, one 8-byte store): a block is two lanes, a slab of 512 half
// a wave.
#include <hip/hip_runtime.h>

#include "qmm_launch.h"
#include "qmm_mx4.h"
#include "qmm_mx4_device.h"

namespace qmm {
namespace {

constexpr int64_t kMaxBlocks = int64_t(1) << 22;   // workgroups of a launch; more slabs take further passes

__device__ __forceinline__ bf16x2_t pair(uint32_t v) { return __builtin_bit_cast(bf16x2_t, v); }

__global__ __launch_bounds__(256) void mx4_quant_kernel(Mx4QuantArgs a, uint32_t slabs, int64_t total) {
  // slab `id` of the [t][slabs], lane `c` of its 32
  const int c = threadIdx.x & 31;
  for (int64_t id = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); id < total; id += int64_t(gridDim.x) * 8) {
    const int64_t row = int64_t(uint64_t(id) / slabs);
    const int s = int(id - row * slabs);
    const int k = kSlabCodes * s + 16 * c;
    const bool live = k < a.d;
    u32x4_t v[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if (live) {
      v[0] = load16(a.x + row * a.ldx + k);
      v[1] = load16(a.x + row * a.ldx + k + 8);
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t u = v[i >> 2][i & 3];
      m = umax(m, umax((u << 16) & 0x7FFFFFFFu, u & 0x7FFF0000u));
    }
    m = umax(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0xB1, 0xF, 0xF, false)));   // the other lane of the block
    const uint32_t e = mx_exponent(m, a.fit);
    const float scale = mx_scale(e);
    if (live) {
      u32x2_t o = {0, 0};
      if (e != 255u) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          o[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o[i], pair(v[i][0]), scale, 0);
          o[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o[i], pair(v[i][1]), scale, 1);
          o[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o[i], pair(v[i][2]), scale, 2);
          o[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(o[i], pair(v[i][3]), scale, 3);
        }
      }
      *reinterpret_cast<u32x2_t*>(a.q + row * (a.d / 2) + k / 2) = o;
    }
    if (!(c & 1)) a.scales[id * 16 + (c >> 1)] = live ? uint8_t(e) : uint8_t(0);
  }
}

}  // namespace

int launch_mx4_quant(const Mx4QuantArgs& a, void* stream) {
  const int64_t slabs = mx_slabs(a.d), total = a.t * slabs;
  const int64_t blocks = std::min((total + 7) / 8, kMaxBlocks);
  launch_kernel(mx4_quant_kernel, dim3(unsigned(blocks)), dim3(256), static_cast<hipStream_t>(stream), a, uint32_t(slabs),
                total);
  return int(hipGetLastError());
}

}  // namespace qmm
