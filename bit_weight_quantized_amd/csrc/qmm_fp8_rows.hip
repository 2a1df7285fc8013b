// Block-scaled e4m3 product for a few activation rows (a decode batch, routed
// segments): every weight is read once from memory for up to 64 rows.
//
//   y[t,n] = Σ_b xs[t,b]·ws[n/128,b] · Σ_{k in b} x[t,k]·w[n,k]
//
// Bound by the weights' bytes, so the kernel is built to keep reads in flight:
// a workgroup takes 16·R weight rows, its waves split the reduction axis into
// equal runs of blocks, and every wave streams its blocks through a private LDS
// ring of D stages (weights, activations and activation scales of one block,
// global -> LDS, no registers, no barriers): while one block is used, the next
// D - 1 are on their way.  Each wave keeps fp32 accumulators, and the waves'
// sums are added in wave order through LDS: nothing depends on timing.
//
// Weights are the A operand, activations the B operand: a lane's four results
// share one activation row (its xs) and one weight block (ws), and a block sum
// takes its two scales in one multiply-add.  Up to 16 rows convert the codes
// to bf16 (exact) for four v_mfma_f32_16x16x32_bf16, which sum in fp32; the e4m3
// instruction, used beyond, aligns the products of 8 neighbouring codes to the
// largest and cuts what lies 13 binary places below it (measured).  Few rows
// feed the next layer's rounding directly and have the time; with more rows the
// conversions would cost more than the reads.
#include <hip/hip_runtime.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"
#include "qmm_launch.h"
#include "qmm_lds_copy.h"

#include <algorithm>

namespace qmm {
namespace {

// Waits for the ring, as asm so that no LDS read is moved across them: at most N
// copies of this wave in flight; every LDS read of this wave done.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds_reads() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

struct Fp8Grouped {
  const int32_t* row_index;
  const int32_t* seg_expert;
  const int32_t* seg_offsets;
  int n_experts, m_total;
  int t_x;
  int max_rows;   // longer segments are left out (0: none)
};

// eight codes -> eight bf16
__device__ __forceinline__ bf16x8_t e4m3x8_to_bf16(uint32_t lo, uint32_t hi) {
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true));
  return __builtin_bit_cast(bf16x8_t, r);
}

__device__ __forceinline__ i32x8_t join(const u32x4_t a, const u32x4_t b) {
  i32x8_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[i] = int(a[i]);
    r[4 + i] = int(b[i]);
  }
  return r;
}

// WAVES waves split the reduction axis; R blocks of 16 weight rows, X8 groups of
// 8 activation rows, D ring stages.  GLU: the upper half of the R blocks are the
// up rows of the same outputs.
template <int WAVES, int R, int X8, int D, bool GROUPED, bool GLU>
struct Fp8Rows {
  static constexpr int C = (X8 + 1) / 2;                 // blocks of 16 activation rows
  static constexpr int RO = GLU ? R / 2 : R;             // blocks of output columns
  static constexpr bool kExact = C == 1;
  static constexpr int kSc = (X8 * 8 + 63) / 64;         // scale copies of a stage
  static constexpr int kOps = 2 * R + X8 + kSc;          // copies of a stage
  static constexpr int kX = 2048 * R, kS = kX + 2048 * C; // stage: weights, activations, scales
  static constexpr int kStage = kS + 256 * kSc;
  static constexpr int kRing = WAVES * D * kStage, kPart = WAVES * R * C * 1024;
  static constexpr int kLds = kRing > kPart ? kRing : kPart;
  static_assert(!GLU || R % 2 == 0, "gate and up blocks come in pairs");
  static_assert((D - 1) * kOps <= 63, "the waits count the copies in flight");
  static_assert(kLds <= 160 * 1024, "LDS");
};

template <int WAVES, int R, int X8, int D, bool GROUPED, bool GLU>
__global__ __launch_bounds__(64 * WAVES) void fp8_rows_kernel(
    const uint8_t* __restrict__ w, const float* __restrict__ ws, int n, int d, int nb,
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t t, uint16_t* __restrict__ y, int64_t ldy,
    Fp8Grouped grp) {
  using T = Fp8Rows<WAVES, R, X8, D, GROUPED, GLU>;
  constexpr int C = T::C, RO = T::RO, kRows = 8 * X8;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int nout = GLU ? n / 2 : n;
  const int n0 = blockIdx.x * 16 * RO;             // first output column

  int64_t m_begin, m_end;
  bool bad_expert = false;
  const uint8_t* wm = w;
  const float* wsm = ws;
  const int sb = GLU ? (nout + kFp8Block - 1) / kFp8Block : 0;   // scale rows of the gate half
  if constexpr (GROUPED) {
    const int s = blockIdx.y;
    m_begin = min(max(grp.seg_offsets[s], 0), grp.m_total);
    m_end = min(max(grp.seg_offsets[s + 1], int(m_begin)), grp.m_total);
    if (m_begin == m_end || (grp.max_rows && m_end - m_begin > grp.max_rows)) return;
    const int e = grp.seg_expert[s];
    bad_expert = e < 0 || e >= grp.n_experts;
    if (!bad_expert) {
      wm += int64_t(e) * n * d;
      wsm += int64_t(e) * (GLU ? 2 * sb : (n + kFp8Block - 1) / kFp8Block) * nb;
    }
  } else {
    m_begin = int64_t(blockIdx.y) * kRows;
    m_end = min(t, m_begin + kRows);
  }
  const float* ws0 = wsm + int64_t(n0 / kFp8Block) * nb;
  const float* ws1 = wsm + int64_t(sb + n0 / kFp8Block) * nb;

  // Copies: lane / 8 is the row of a copy's eight, LDS chunk lane % 8 holds the
  // row's 16-byte chunk (lane % 8) ^ (row % 8), so that the operand reads of
  // eight neighbouring rows fall into different banks.
  // Weight rows: one buffer per half, based at the tile's first row, so the
  // 32-bit offsets stay small; rows past the matrix read zero.
  const int crow = lane >> 3, cchunk = 16 * ((lane & 7) ^ crow);
  const int live = min(16 * RO, nout - n0);
  const __amdgpu_buffer_rsrc_t wr0 = make_rsrc(wm + int64_t(n0) * d, uint32_t(live) * uint32_t(d));
  const __amdgpu_buffer_rsrc_t wr1 =
      GLU ? make_rsrc(wm + int64_t(nout + n0) * d, uint32_t(live) * uint32_t(d)) : wr0;
  uint32_t woff[2 * RO];
#pragma unroll
  for (int i = 0; i < 2 * RO; ++i) woff[i] = 8 * i + crow < live ? uint32_t(8 * i + crow) * uint32_t(d) : kOOB8;

  // the wave's share of the reduction axis, and its ring
  const int b_begin = nb * wave / WAVES, b_end = nb * (wave + 1) / WAVES;
  const unsigned char* ring = lds + wave * D * T::kStage;
  const uint32_t ring_at = lds_addr(ring);
  const int o0 = 128 * col + 16 * (g ^ (col & 7));       // operand chunks g and g + 4 of row col

  for (int64_t m0 = m_begin; m0 < m_end; m0 += kRows) {
    // activation rows: dense rows are based at the pass's first row; grouped
    // rows can be anywhere in x (below 2 GiB, checked by the caller)
    __amdgpu_buffer_rsrc_t xr, sr;
    if constexpr (GROUPED) {
      xr = make_rsrc(x, uint32_t(grp.t_x) * uint32_t(d));
      sr = make_rsrc(xs, uint32_t(grp.t_x) * uint32_t(nb) * 4u);
    } else {
      const uint32_t rows = uint32_t(min(int64_t(kRows), m_end - m0));
      xr = make_rsrc(x + m0 * d, rows * uint32_t(d));
      sr = make_rsrc(xs + m0 * nb, rows * uint32_t(nb) * 4u);
    }
    auto source = [&](int row) -> int {            // the row of x (dense: of the pass), or -1
      if (m0 + row >= m_end) return -1;
      if constexpr (!GROUPED) return row;
      const int src = grp.row_index ? grp.row_index[m0 + row] : int(m0 + row);
      return bad_expert || src < 0 || src >= grp.t_x ? -1 : src;
    };
    uint32_t xoff[X8], soff[T::kSc];
#pragma unroll
    for (int i = 0; i < X8; ++i) {
      const int src = source(8 * i + crow);
      xoff[i] = src >= 0 ? uint32_t(src) * uint32_t(d) : kOOB8;
    }
#pragma unroll
    for (int i = 0; i < T::kSc; ++i) {
      const int src = 64 * i + lane < kRows ? source(64 * i + lane) : -1;
      soff[i] = src >= 0 ? uint32_t(src) * uint32_t(nb) * 4u : kOOB8;
    }
    auto copy = [&](int b, int stage) {
      const uint32_t at = ring_at + uint32_t(stage * T::kStage);
      const uint32_t k = uint32_t(kFp8Block * b + cchunk);
      const uint32_t ko = b < b_end && k < uint32_t(d) ? k : kOOB8;   // past the wave's share: zeros, no reads
#pragma unroll
      for (int i = 0; i < 2 * R; ++i) {
        const uint32_t o = woff[i % (2 * RO)];
        copy16_to_lds(i < 2 * RO ? wr0 : wr1, (o + ko) | ((o | ko) & kOOB8), at + 1024u * i);
      }
#pragma unroll
      for (int i = 0; i < X8; ++i)
        copy16_to_lds(xr, (xoff[i] + ko) | ((xoff[i] | ko) & kOOB8), at + T::kX + 1024u * i);
#pragma unroll
      for (int i = 0; i < T::kSc; ++i)
        copy4_to_lds(sr, b < b_end ? soff[i] + 4u * uint32_t(b) : kOOB8, at + T::kS + 256u * i);
    };

    f32x4_t acc[R][C];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) acc[r][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll
    for (int i = 0; i < D; ++i) copy(b_begin + i, i);
    float w0 = ws0[min(b_begin, nb - 1)], w1 = GLU ? ws1[min(b_begin, nb - 1)] : 0.f;
    int stage = 0;
    for (int b = b_begin; b < b_end; ++b) {
      const int next = min(b + 1, nb - 1);
      const float w0n = ws0[next], w1n = GLU ? ws1[next] : 0.f;
      wait_copies<(D - 1) * T::kOps>();   // block b has landed
      const unsigned char* st = ring + stage * T::kStage;
      u32x4_t a[R][2], x2[C][2];
      float s[C];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int h = 0; h < 2; ++h) a[r][h] = *reinterpret_cast<const u32x4_t*>(st + 2048 * r + (o0 ^ (64 * h)));
#pragma unroll
      for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int h = 0; h < 2; ++h) x2[c][h] = *reinterpret_cast<const u32x4_t*>(st + T::kX + 2048 * c + (o0 ^ (64 * h)));
        s[c] = *reinterpret_cast<const float*>(st + T::kS + 4 * (16 * c + col));
      }
      wait_lds_reads();                   // ... and is in registers: its stage is free
      copy(b + D, stage);
      stage = stage + 1 == D ? 0 : stage + 1;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float s0 = s[c] * w0, s1 = GLU ? s[c] * w1 : 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          f32x4_t p = {0.f, 0.f, 0.f, 0.f};
          if constexpr (T::kExact) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  e4m3x8_to_bf16(a[r][q >> 1][2 * (q & 1)], a[r][q >> 1][2 * (q & 1) + 1]),
                  e4m3x8_to_bf16(x2[c][q >> 1][2 * (q & 1)], x2[c][q >> 1][2 * (q & 1) + 1]), p, 0, 0, 0);
          } else {
            // formats 0: e4m3; block exponents 0 select the unscaled instruction
            p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(a[r][0], a[r][1]), join(x2[c][0], x2[c][1]), p,
                                                                 0, 0, 0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][c][i] = __builtin_fmaf(p[i], r < RO ? s0 : s1, acc[r][c][i]);
        }
      }
      w0 = w0n;
      w1 = w1n;
    }

    // the ring becomes the waves' sums: [wave][R·C][64]
    wait_copies<0>();
    __syncthreads();
    f32x4_t* part = reinterpret_cast<f32x4_t*>(lds);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) part[(wave * R * C + r * C + c) * 64 + lane] = acc[r][c];
    __syncthreads();
    const bool wide = (ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(y) & 7) == 0;
    auto summed = [&](int u) {
      f32x4_t v = part[u * 64 + lane];
#pragma unroll
      for (int p = 1; p < WAVES; ++p) {
        const f32x4_t o = part[(p * R * C + u) * 64 + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += o[i];
      }
      return v;
    };
    // unit u: output block (r, c), a lane's four columns of one row
    for (int u = wave; u < RO * C; u += WAVES) {
      const int r = u / C, c = u % C;
      const int64_t row = m0 + 16 * c + col;
      const int j = n0 + 16 * r + 4 * g;
      f32x4_t v = summed(u);
      if constexpr (GLU) {
        const f32x4_t up = summed(u + RO * C);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * up[i];
      }
      if (16 * c + col < kRows && row < m_end) {
        const bool bad = GROUPED && source(16 * c + col) < 0;
        uint16_t* to = y + row * ldy + j;
        uint16_t b16[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b16[i] = bad ? uint16_t(0x7FC0) : f32_to_bf16(v[i]);
        if (wide && j + 4 <= nout) {
          *reinterpret_cast<u32x2_t*>(to) =
              u32x2_t{uint32_t(b16[0]) | uint32_t(b16[1]) << 16, uint32_t(b16[2]) | uint32_t(b16[3]) << 16};
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (j + i < nout) to[i] = b16[i];
        }
      }
    }
    __syncthreads();   // the next pass fills the ring again
  }
}

template <int WAVES, int R, int X8, int D, bool GROUPED, bool GLU>
int go(const Fp8GemmArgs& a, int max_rows, hipStream_t s) {
  using T = Fp8Rows<WAVES, R, X8, D, GROUPED, GLU>;
  const int nout = GLU ? a.n / 2 : a.n, per = 16 * T::RO;
  const Fp8Grouped grp{a.row_index, a.seg_expert, a.seg_offsets, a.n_experts, a.m_total, int(a.t_x), max_rows};
  const unsigned gy = GROUPED ? unsigned(a.n_seg) : unsigned((a.t + 8 * X8 - 1) / (8 * X8));
  launch_kernel_lds(fp8_rows_kernel<WAVES, R, X8, D, GROUPED, GLU>, dim3(unsigned((nout + per - 1) / per), gy),
                    dim3(64 * WAVES), T::kLds, s, a.w, a.ws, a.n, a.d, fp8_blocks(a.d), a.x, a.xs, a.t, a.y, a.ldy, grp);
  return int(hipGetLastError());
}

}  // namespace

int launch_fp8_rows(const Fp8GemmArgs& a, int max_rows, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t rows = a.n_seg > 0 ? (max_rows ? std::min(max_rows, a.max_seg_rows) : a.max_seg_rows) : a.t;
  if (a.n_seg > 0) {
    if (a.glu) {
      if (rows <= 8) return go<4, 2, 1, 4, true, true>(a, max_rows, s);
      if (rows <= 16) return go<4, 2, 2, 4, true, true>(a, max_rows, s);
      if (rows <= 32) return go<4, 2, 4, 3, true, true>(a, max_rows, s);
      return go<4, 2, 8, 3, true, true>(a, max_rows, s);
    }
    if (rows <= 8) return go<4, 2, 1, 4, true, false>(a, max_rows, s);
    if (rows <= 16) return go<4, 2, 2, 4, true, false>(a, max_rows, s);
    if (rows <= 32) return go<4, 2, 4, 3, true, false>(a, max_rows, s);
    return go<4, 2, 8, 3, true, false>(a, max_rows, s);
  }
  if (rows <= 8) return go<4, 2, 1, 4, false, false>(a, 0, s);
  if (rows <= 16) return go<4, 2, 2, 4, false, false>(a, 0, s);
  if (rows <= 32) return go<4, 2, 4, 3, false, false>(a, 0, s);
  return go<4, 2, 8, 3, false, false>(a, 0, s);
}

}  // namespace qmm
