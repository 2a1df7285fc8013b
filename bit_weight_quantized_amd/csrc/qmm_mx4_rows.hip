// Microscaled 4-bit product for few activation rows: both sides straight from memory to the
// registers of the fp4 matrix instruction, nothing shared but the sums at the end.
//
//   y[t,n] = Σ_b 2^(Ex[t,b] + Ew[n,b] - 254) · Σ_{k in b} x[t,k]·w[n,k]
//
// A workgroup has 16·R weight rows (the A operand) and passes of 16·X activation rows (the B
// operand); its W waves take the steps of 256 codes in turn, each summing all rows, and the
// W sums meet in LDS in the waves' order.  In a step lane (c, g) loads of each of its rows c
// the 16-byte pieces g and 4 + g, which are whole blocks, and the row's 8 exponents; every
// load is issued without a branch (an offset past the buffer reads zeros) and kRing steps
// ahead.  Weight rows of a slab lie one behind the other in the packed layout, so a wave's
// loads of 16 rows cover whole lines.
//
// Bound by the weights' bytes: every weight is read once for up to 16·X activation rows.
#include <hip/hip_runtime.h>

#include "qmm_launch.h"
#include "qmm_mx4.h"
#include "qmm_mx4_device.h"

namespace qmm {
namespace {

constexpr uint32_t kOOB = 0x80000000u;   // OR-ed into a buffer offset: past every range
constexpr int64_t kMaxPasses = 65535;    // of a dense launch's grid; more rows take further turns

struct Mx4RowsArgs {
  const uint8_t* codes;
  const uint8_t* meta;
  uint32_t codes_bytes, meta_bytes;
  Mx4GemmArgs g;
};

__device__ __forceinline__ u32x2_t buf_load8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, int(off), 0, 0));
}

template <int R, int X, int W, bool GROUPED, bool GLU>
__global__ __launch_bounds__(64 * W) void mx4_rows_kernel(Mx4RowsArgs A) {
  constexpr int kOut = GLU ? 8 * R : 16 * R;        // output columns of a workgroup
  constexpr int kRing = R + X <= 3 ? 3 : 2;         // steps in flight
  static_assert(!GLU || R % 2 == 0, "gate blocks, then as many up blocks");
  __shared__ f32x4_t red[W][X][R][64];
  const Mx4GemmArgs& a = A.g;
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Slabs L{a.n, a.d, QMM_MXFP4_G32};
  const int steps = mx_steps(a.d), nout = GLU ? a.n / 2 : a.n, n0 = blockIdx.x * kOut;
  const uint32_t sstride = uint32_t(mx_scale_bytes(a.d)), xstride = uint32_t(a.d) / 2;

  int64_t r_begin = 0, r_end = a.t;
  bool bad_expert = false;
  const uint8_t *codes = A.codes, *meta = A.meta;
  int turn = blockIdx.y, turns = gridDim.y;
  if constexpr (GROUPED) {
    const int s = blockIdx.y;
    r_begin = min(max(a.seg_offsets[s], 0), a.m_total);
    r_end = min(max(a.seg_offsets[s + 1], int(r_begin)), a.m_total);
    const int e = a.seg_expert[s];
    bad_expert = e < 0 || e >= a.n_experts;
    const int64_t off = bad_expert ? 0 : int64_t(e) * a.expert_stride;
    codes += off;
    meta += off;
    turn = 0;
    turns = 1;
  }
  const __amdgpu_buffer_rsrc_t cr = make_rsrc(codes, A.codes_bytes), mr = make_rsrc(meta, A.meta_bytes);
  // the lane's weight rows; one past the end reads the last and is dropped
  int wrow[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int o = GLU ? n0 + 16 * (j % (R / 2 > 0 ? R / 2 : 1)) + c : n0 + 16 * j + c;
    wrow[j] = min(o, nout - 1) + (GLU && j >= R / 2 ? nout : 0);
  }

  for (int64_t r0 = r_begin + int64_t(turn) * 16 * X; r0 < r_end; r0 += int64_t(turns) * 16 * X) {
    const int rows = int(min(int64_t(16 * X), r_end - r0));
    // activation rows of the pass: dense ones from its first, grouped ones anywhere
    uint32_t xoff[X], soff[X];
    bool bad[X];
#pragma unroll
    for (int i = 0; i < X; ++i) {
      int row = min(16 * i + c, rows - 1);
      bad[i] = false;
      if constexpr (GROUPED) {
        row = a.row_index ? a.row_index[r0 + row] : int(r0) + row;
        bad[i] = bad_expert || row < 0 || row >= a.t_x;
        row = bad[i] ? 0 : row;
      }
      xoff[i] = uint32_t(row) * xstride;
      soff[i] = uint32_t(row) * sstride;
    }
    const int64_t first = GROUPED ? 0 : r0;
    const uint32_t held = GROUPED ? uint32_t(a.t_x) : uint32_t(rows);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x + first * xstride, held * xstride);
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(a.xs + first * sstride, held * sstride);

    u32x4_t wq[kRing][R][2], xq[kRing][X][2];
    u32x2_t we[kRing][R], xe[kRing][X];
    auto issue = [&](int slot, int b) {
      const bool in = b < steps;
      const int s = in ? b >> 1 : 0, half = b & 1, w = L.width(s);
      uint32_t piece[2];
#pragma unroll
      for (int m = 0; m < 2; ++m) piece[m] = in && 256 * half + 128 * m + 32 * g < w ? 0u : kOOB;
      const uint32_t at = uint32_t(128 * half + 16 * g), all = in ? 0u : kOOB;
      const uint32_t cs = uint32_t(L.codes(s, 0)), mrow = uint32_t(L.meta_row(s)), mq = uint32_t(L.meta_quad());
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const uint32_t off = cs + uint32_t(wrow[j]) * uint32_t(w / 2) + at;
        wq[slot][j][0] = buf_load16(cr, off | piece[0]);
        wq[slot][j][1] = buf_load16(cr, (off + 64u) | piece[1]);
        we[slot][j] = buf_load8(mr, (uint32_t(wrow[j] >> 2) * mq + 64u * uint32_t(s) + uint32_t(wrow[j] & 3) * mrow +
                                     8u * uint32_t(half)) | all);
      }
#pragma unroll
      for (int i = 0; i < X; ++i) {
        const uint32_t off = xoff[i] + 256u * uint32_t(s) + at;
        xq[slot][i][0] = buf_load16(xr, off | piece[0]);
        xq[slot][i][1] = buf_load16(xr, (off + 64u) | piece[1]);
        xe[slot][i] = buf_load8(sr, (soff[i] + 16u * uint32_t(s) + 8u * uint32_t(half)) | all);
      }
    };
    f32x4_t acc[X][R];
#pragma unroll
    for (int i = 0; i < X; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < kRing; ++u) issue(u, wave + W * u);
    for (int b0 = wave; b0 < steps; b0 += W * kRing) {
#pragma unroll
      for (int u = 0; u < kRing; ++u) {
        // a step past the last one adds zeros
        uint32_t se[X][2];
#pragma unroll
        for (int i = 0; i < X; ++i)
#pragma unroll
          for (int m = 0; m < 2; ++m) se[i][m] = xe[u][i][m] >> (8 * g);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int j = 0; j < R; ++j) {
            const uint32_t we8 = we[u][j][m] >> (8 * g);
#pragma unroll
            for (int i = 0; i < X; ++i) acc[i][j] = mfma_fp4<0, 0>(wq[u][j][m], xq[u][i][m], acc[i][j], we8, se[i][m]);
          }
        issue(u, b0 + W * (u + kRing));
      }
    }

    // the waves' sums, in their order; a wave finishes the activation blocks i % W == wave
    if constexpr (W > 1) {
#pragma unroll
      for (int i = 0; i < X; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) red[wave][i][j][lane] = acc[i][j];
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < X; ++i) {
      if (i % W != wave) continue;
      f32x4_t v[R];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        v[j] = W > 1 ? red[0][i][j][lane] : acc[i][j];
#pragma unroll
        for (int w = 1; w < W; ++w) v[j] += red[w][i][j][lane];
      }
      // lane (c, g): row c of the block, columns 4g .. 4g + 3 of each weight block
      const int row = 16 * i + c;
      if constexpr (GLU) {
#pragma unroll
        for (int j = 0; j < R / 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] = silu(v[j][e]) * v[R / 2 + j][e];
      }
      constexpr int kBlocks = GLU ? R / 2 : R;
      if constexpr (GLU && kBlocks == 2) {
        if (a.hq) {
          // 32 neighbouring columns are a block: 8 here, the rest in the lanes of the same row
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) m = umax(m, __float_as_uint(v[j][e]) & 0x7FFFFFFFu);
          m = umax(m, uint32_t(__shfl_xor(int(m), 16)));
          m = umax(m, uint32_t(__shfl_xor(int(m), 32)));
          if (bad[i]) m = 0x7FC00000u;
          const uint32_t ex = mx_exponent(m, a.fit);
          const float scale = mx_scale(ex);
          if (row < rows) {
            const int64_t out = r0 + row;
            uint8_t* hs = a.hs + out * mx_scale_bytes(nout);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t q = 0;
              if (ex != 255u) {
                q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[j][0], v[j][1], scale, 0);
                q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[j][2], v[j][3], scale, 1);
              }
              *reinterpret_cast<uint16_t*>(a.hq + out * (nout / 2) + (n0 + 16 * j + 4 * g) / 2) = uint16_t(q);
            }
            if (g == 0) hs[n0 / 32] = uint8_t(ex);
            if (n0 + 32 == nout)   // zeros past the row's blocks
              for (int b = nout / 32 + g; b < mx_scale_bytes(nout); b += 4) hs[b] = 0;
          }
          continue;
        }
      }
      if (row < rows) {
        uint16_t* y = a.y + (r0 + row) * a.ldy;
#pragma unroll
        for (int j = 0; j < kBlocks; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int o = n0 + 16 * j + 4 * g + e;
            if (o < nout) y[o] = f32_to_bf16(bad[i] ? __builtin_nanf("") : v[j][e]);
          }
      }
    }
    if constexpr (W > 1) __syncthreads();   // the next pass writes the sums again
  }
}

template <int R, int X, int W, bool GROUPED, bool GLU>
int go(const Mx4GemmArgs& a, hipStream_t s) {
  Layout l;
  if (!layout_of(QMM_MXFP4_G32, a.n, a.d, &l)) return int(hipErrorInvalidValue);
  const int out = GLU ? 8 * R : 16 * R, nout = GLU ? a.n / 2 : a.n;
  const int64_t passes = GROUPED ? a.n_seg : std::min((a.t + 16 * X - 1) / (16 * X), kMaxPasses);
  const Mx4RowsArgs k{a.packed + l.codes_offset, a.packed + l.meta_offset, uint32_t(int64_t(a.n) * (a.d / 2)),
                      uint32_t(l.meta_bytes), a};
  launch_kernel((mx4_rows_kernel<R, X, W, GROUPED, GLU>), dim3(unsigned((nout + out - 1) / out), unsigned(passes)),
                dim3(64 * W), s, k);
  return int(hipGetLastError());
}

}  // namespace

int launch_mx4_rows(const Mx4GemmArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.n_seg > 0) return a.glu ? go<4, 1, 4, true, true>(a, s) : go<2, 1, 4, true, false>(a, s);
  if (a.t <= 16) return go<2, 1, 4, false, false>(a, s);
  return a.t <= 32 ? go<2, 2, 4, false, false>(a, s) : go<4, 4, 4, false, false>(a, s);
}

int launch_mx4_product(const Mx4GemmArgs& a, void* stream) { return launch_mx4_rows(a, stream); }

}  // namespace qmm
