// Device helpers of the microscaled 4-bit path.
#pragma once

#include "qmm_device.h"
#include "qmm_fp8_device.h"
#include "qmm_mx4.h"

namespace qmm {

__device__ __forceinline__ i32x8_t fp4_operand(const u32x4_t v) {
  return i32x8_t{int(v[0]), int(v[1]), int(v[2]), int(v[3]), 0, 0, 0, 0};
}

// 16 x 16 block sums over 128 codes: lane (c, g) holds 32 neighbouring codes of row c of
// either side, and byte BA (BB) of sa (sb) is the exponent of those 32.  Format 4: E2M1.
// The products of two codes are whole quarters up to 36, so nothing is lost within a block.
template <int BA, int BB>
__device__ __forceinline__ f32x4_t mfma_fp4(const u32x4_t a, const u32x4_t b, f32x4_t acc, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(a), fp4_operand(b), acc, 4, 4, BA, int(sa), BB,
                                                          int(sb));
}

// E8M0 of a block whose largest |x| has the fp32 bits m (sign clear): the exponent that puts
// it into [4, 8), from where codes over 6 saturate, or (fit) into (3, 6]: one more where the
// mantissa is over 1.5.  255, which stands for NaN, where m is not finite.
__device__ __forceinline__ uint32_t mx_exponent(uint32_t m, bool fit) {
  if (m >= 0x7F800000u) return 255u;
  const uint32_t e = (m + (fit ? 0x3FFFFFu : 0u)) >> 23;
  return e > 2u ? e - 2u : 0u;
}

// 2^(e - 127) as the conversions take it: they read the exponent bits alone.
__device__ __forceinline__ float mx_scale(uint32_t e) { return __uint_as_float(e << 23); }

}  // namespace qmm
