// Device helpers of the block-scaled e4m3 path.
#pragma once

#include "qmm_device.h"

namespace qmm {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Smallest block maximum a scale is made from: keeps m / 448 and 448 / m
// normal fp32 numbers, and gives a block of zeros a scale like any other.
constexpr float kFp8Floor = 0x1p-96f;

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest |v| of fp32 bit patterns with the sign cleared, compared as integers:
// the order of the numbers, with NaN above infinity, so a NaN is kept.
template <int LANES>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
  v = umax(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0xB1, 0xF, 0xF, false)));    // xor 1
  v = umax(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x4E, 0xF, 0xF, false)));    // xor 2
  v = umax(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x141, 0xF, 0xF, false)));   // mirror in 8
  if constexpr (LANES == 16)
    v = umax(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x140, 0xF, 0xF, false))); // mirror in 16
  return v;
}

struct BlockScale {
  float scale, factor;   // m / 448 and 448 / m
};
// m: bits of the block's largest |x|.  Two IEEE divisions, so the codes are
// the ones the formula gives, whatever the order of anything else.
__device__ __forceinline__ BlockScale block_scale(uint32_t m) {
  const float f = __uint_as_float(umax(m, __float_as_uint(kFp8Floor)));
  return {f / 448.0f, 448.0f / f};
}

// four fp32 -> four e4m3 codes, round to nearest even; |v| <= 448·(1 + 2^-23),
// which still rounds to 448
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return uint32_t(v);
}

// A value at a uniform address of memory that the kernel does not write, as a
// scalar load (a vector load would count among the copies in flight).
__device__ __forceinline__ float scalar_load(const float* p, int i) {
  typedef const __attribute__((address_space(4))) float* constant_ptr;
  return reinterpret_cast<constant_ptr>(reinterpret_cast<uintptr_t>(p))[i];
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + expf(-v)); }

// The same from the hardware's exponential and reciprocal, for tiles of many values:
// the precise form is 35 instructions a value.  The product with log2(e) is rounded
// before the exponential, so e^-v is off by 1.22·|v|·2^-24 of its value and what
// follows by a few 2^-24 more: 2^-18 of silu at v = -40, 2^-9 of what the rounding to
// bf16 takes.  Below v = -87, where silu is under 2^-119, either form may give zero.
__device__ __forceinline__ float quick_silu(float v) {
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504f));
}

}  // namespace qmm
