// Block-scaled e4m3 product for a few activation rows (a decode batch, routed
// segments): every weight is read once from memory for up to 64 rows.
//
//   y[t,n] = Σ_b xs[t,b]·ws[n/128,b] · Σ_{k in b} x[t,k]·w[n,k]
//
// Codes are converted to bf16 (exact) and multiplied by four
// v_mfma_f32_16x16x32_bf16 per scale block: these sum in fp32, where the e4m3
// instruction aligns the products of 8 neighbouring codes to the largest and
// cuts what lies 13 binary places below (measured); reading the weights takes
// several times longer than either.  Weights are the A operand, activations the
// B operand, so a lane's four results share one activation row (its xs) and one
// weight block (ws), and a block sum takes its scales in one multiply-add.
//
// A workgroup takes 16·R weight rows; its waves split the reduction axis in
// runs of U blocks (U·128 consecutive bytes of each weight row), each keeps
// fp32 accumulators, and the waves' sums are added in wave order through LDS:
// the result does not depend on timing.
#include <hip/hip_runtime.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"
#include "qmm_launch.h"

#include <algorithm>

namespace qmm {
namespace {

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

// WAVES waves split the reduction axis; R (C) blocks of 16 weight (activation)
// rows; U scale blocks a wave loads at once.  GLU: the upper half of the R
// blocks are the up rows of the same outputs.
template <int WAVES, int R, int C, int U, bool GROUPED, bool GLU>
__global__ __launch_bounds__(64 * WAVES) void fp8_rows_kernel(
    const uint8_t* __restrict__ w, const float* __restrict__ ws, int n, int d, int nb,
    const uint8_t* __restrict__ x, const float* __restrict__ xs, int64_t t, uint16_t* __restrict__ y, int64_t ldy,
    Fp8Grouped grp) {
  static_assert(!GLU || R % 2 == 0, "gate and up blocks come in pairs");
  constexpr int RO = GLU ? R / 2 : R;              // blocks of output columns
  __shared__ __attribute__((aligned(16))) f32x4_t part[WAVES][R * C][64];

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
    m_begin = int64_t(blockIdx.y) * 16 * C;
    m_end = min(t, m_begin + 16 * C);
  }

  // weight rows: one buffer per half, based at the tile's first row, so the
  // 32-bit offsets stay small; rows past the matrix read zero
  const int live = min(16 * RO, nout - n0);
  const __amdgpu_buffer_rsrc_t wr0 = make_rsrc(wm + int64_t(n0) * d, uint32_t(live) * uint32_t(d));
  const __amdgpu_buffer_rsrc_t wr1 =
      GLU ? make_rsrc(wm + int64_t(nout + n0) * d, uint32_t(live) * uint32_t(d)) : wr0;
  const float* ws0 = wsm + int64_t(n0 / kFp8Block) * nb;
  const float* ws1 = wsm + int64_t(sb + n0 / kFp8Block) * nb;

  for (int64_t m0 = m_begin; m0 < m_end; m0 += 16 * C) {
    // activation rows: dense rows are based at the pass's first row; grouped
    // rows can be anywhere in x (below 2 GiB, checked by the caller)
    __amdgpu_buffer_rsrc_t xr, sr;
    uint32_t xoff[C], soff[C];
    bool bad_row[C];
    if constexpr (GROUPED) {
      xr = make_rsrc(x, uint32_t(grp.t_x) * uint32_t(d));
      sr = make_rsrc(xs, uint32_t(grp.t_x) * uint32_t(nb) * 4u);
    } else {
      const uint32_t rows = uint32_t(min(int64_t(16 * C), m_end - m0));
      xr = make_rsrc(x + m0 * d, rows * uint32_t(d));
      sr = make_rsrc(xs + m0 * nb, rows * uint32_t(nb) * 4u);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      uint32_t row = uint32_t(16 * c + col);
      bool ok = m0 + row < m_end;
      bad_row[c] = false;
      if constexpr (GROUPED) {
        const int64_t at = m0 + row;
        const int src = ok ? (grp.row_index ? grp.row_index[at] : int(at)) : 0;
        bad_row[c] = bad_expert || src < 0 || src >= grp.t_x;
        ok = ok && !bad_row[c];
        row = uint32_t(src);
      }
      xoff[c] = ok ? row * uint32_t(d) : kOOB8;
      soff[c] = ok ? row * uint32_t(nb) * 4u : kOOB8;
    }

    f32x4_t acc[R][C];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) acc[r][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    struct Block {
      u32x4_t a[R][2], b[C][2];
      float s[C], w0, w1;
    };
    auto load = [&](Block& v, int b) {
      const bool in = b < nb;                      // uniform
      const int bs = in ? b : 0;
      v.w0 = ws0[bs];
      v.w1 = GLU ? ws1[bs] : 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = kFp8Block * b + 64 * h + 16 * g;
        const uint32_t ko = k < d ? uint32_t(k) : kOOB8;   // also past the last block
#pragma unroll
        for (int r = 0; r < R; ++r)
          v.a[r][h] = buf_load16(r < RO ? wr0 : wr1, (uint32_t(16 * (r % RO) + col) * uint32_t(d) + ko) | (ko & kOOB8));
#pragma unroll
        for (int c = 0; c < C; ++c) v.b[c][h] = buf_load16(xr, (xoff[c] + ko) | ((xoff[c] | ko) & kOOB8));
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
        v.s[c] = __uint_as_float(buf_load4(sr, in ? (soff[c] + 4u * uint32_t(b)) | (soff[c] & kOOB8) : kOOB8));
    };
    auto use = [&](const Block& v) {
      f32x4_t p[R][C];
#pragma unroll
      for (int h = 0; h < 4; ++h) {   // codes 16·g + 8·(h & 1) .. + 7 of half h >> 1
        bf16x8_t a[R];
#pragma unroll
        for (int r = 0; r < R; ++r) a[r] = e4m3x8_to_bf16(v.a[r][h >> 1][2 * (h & 1)], v.a[r][h >> 1][2 * (h & 1) + 1]);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const bf16x8_t b = e4m3x8_to_bf16(v.b[c][h >> 1][2 * (h & 1)], v.b[c][h >> 1][2 * (h & 1) + 1]);
#pragma unroll
          for (int r = 0; r < R; ++r)
            p[r][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[r], b, h ? p[r][c] : f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float s0 = v.s[c] * v.w0, s1 = GLU ? v.s[c] * v.w1 : 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[r][c][i] = __builtin_fmaf(p[r][c][i], r < RO ? s0 : s1, acc[r][c][i]);
      }
    };

    // runs of U blocks, the next run loaded while the present one is used; a
    // run past the end reads zeros
    Block v0[U], v1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load(v0[u], wave * U + u);
    for (int b = wave * U; b < nb; b += 2 * WAVES * U) {
#pragma unroll
      for (int u = 0; u < U; ++u) load(v1[u], b + WAVES * U + u);
#pragma unroll
      for (int u = 0; u < U; ++u) use(v0[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) load(v0[u], b + 2 * WAVES * U + u);
#pragma unroll
      for (int u = 0; u < U; ++u) use(v1[u]);
    }

#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < C; ++c) part[wave][r * C + c][lane] = acc[r][c];
    __syncthreads();
    // unit u: block (r, c) of the outputs, a lane's four values
    const bool wide = (ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(y) & 7) == 0;
    for (int u = wave; u < RO * C; u += WAVES) {
      const int r = u / C, c = u % C;
      f32x4_t v = part[0][u][lane];
      for (int p = 1; p < WAVES; ++p) {
        const f32x4_t o = part[p][u][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += o[i];
      }
      if constexpr (GLU) {
        f32x4_t up = part[0][u + RO * C][lane];
        for (int p = 1; p < WAVES; ++p) {
          const f32x4_t o = part[p][u + RO * C][lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) up[i] += o[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * up[i];
      }
      const int64_t row = m0 + 16 * c + col;
      const int j = n0 + 16 * r + 4 * g;
      bool bad = false;
#pragma unroll
      for (int cc = 0; cc < C; ++cc) bad = cc == c ? bad_row[cc] : bad;
      if (row < m_end) {
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
    __syncthreads();   // part is written again by the next pass
  }
}

template <int WAVES, int R, int C, int U, bool GROUPED, bool GLU>
int go(const Fp8GemmArgs& a, int max_rows, hipStream_t s) {
  const int nout = GLU ? a.n / 2 : a.n, per = 16 * (GLU ? R / 2 : R);
  const Fp8Grouped grp{a.row_index, a.seg_expert, a.seg_offsets, a.n_experts, a.m_total, int(a.t_x), max_rows};
  const unsigned gy = GROUPED ? unsigned(a.n_seg) : unsigned((a.t + 16 * C - 1) / (16 * C));
  launch_kernel(fp8_rows_kernel<WAVES, R, C, U, GROUPED, GLU>, dim3(unsigned((nout + per - 1) / per), gy),
                dim3(64 * WAVES), s, a.w, a.ws, a.n, a.d, fp8_blocks(a.d), a.x, a.xs, a.t, a.y, a.ldy, grp);
  return int(hipGetLastError());
}

}  // namespace

int launch_fp8_rows(const Fp8GemmArgs& a, int max_rows, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t rows = a.n_seg > 0 ? (max_rows ? std::min(max_rows, a.max_seg_rows) : a.max_seg_rows) : a.t;
  if (a.n_seg > 0) {
    if (a.glu) {
      if (rows <= 16) return go<4, 2, 1, 2, true, true>(a, max_rows, s);
      if (rows <= 32) return go<4, 2, 2, 2, true, true>(a, max_rows, s);
      return go<4, 4, 4, 1, true, true>(a, max_rows, s);
    }
    if (rows <= 16) return go<4, 1, 1, 4, true, false>(a, max_rows, s);
    if (rows <= 32) return go<4, 2, 2, 2, true, false>(a, max_rows, s);
    return go<4, 4, 4, 1, true, false>(a, max_rows, s);
  }
  if (rows <= 16) return go<4, 1, 1, 4, false, false>(a, 0, s);
  if (rows <= 32) return go<4, 2, 2, 2, false, false>(a, 0, s);
  return go<4, 4, 4, 1, false, false>(a, 0, s);
}

}  // namespace qmm
