// Block-scaled e4m3 product for many activation rows: tiles of activations and
// weights in LDS, e4m3 matrix instructions.
//
//   y[t,n] = Σ_b xs[t,b]·ws[n/128,b] · Σ_{k in b} x[t,k]·w[n,k]
//
// A K step is one scale block (128 codes, 128 bytes of every row).  One
// v_mfma_f32_16x16x128_f8f6f4 sums a whole block for 16 weight rows (A operand)
// and 16 activation rows (B operand); its four results of a lane share one
// activation row and one weight block, so a block's two scales are one fp32
// product and the sum over the blocks is one fp32 multiply-add per value, which
// the vector unit does while the matrix unit works on the next block sums.
//
// Both tiles go global -> LDS without passing registers, double-buffered: the
// copies of step k + 1 are in flight during the whole of step k, one barrier a
// step.  A row's eight 16-byte chunks are stored at chunk ^ (row mod 8), done on
// the global side of the copy, so the operand reads of eight neighbouring rows
// fall into different banks.
#include <hip/hip_runtime.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"
#include "qmm_launch.h"
#include "qmm_lds_copy.h"

#include <algorithm>

namespace qmm {
namespace {

// TS (WS) blocks of 16 activation (weight) rows a wave, WT × WN waves.
// GLU: the lower half of a wave's weight blocks are gate rows, the upper half
// the up rows of the same outputs.
template <int TS, int WS, int WT, int WN, bool GROUPED, bool GLU>
struct Fp8Tile {
  static constexpr int kWaves = WT * WN;
  static constexpr int kT = 16 * TS * WT;              // activation rows
  static constexpr int kN = 16 * WS * WN;              // weight rows
  static constexpr int kOut = GLU ? kN / 2 : kN;       // output columns
  static constexpr int kStage = (kT + kN) * 128 + kT * 4;
  static_assert((kT + kN) / 8 % kWaves == 0 && kT % 64 == 0, "whole copies per wave");
  static constexpr int kXCopies = kT / 8 / kWaves, kWCopies = kN / 8 / kWaves;
};

template <int TS, int WS, int WT, int WN, bool GROUPED, bool GLU>
__global__ __launch_bounds__(64 * WT * WN) void fp8_tile_kernel(
    const uint8_t* __restrict__ w, const float* __restrict__ ws, int n, int d, int nb, const uint8_t* __restrict__ x,
    const float* __restrict__ xs, int64_t t, uint16_t* __restrict__ y, int64_t ldy, int tiles_n,
    const int32_t* __restrict__ row_index, const int32_t* __restrict__ seg_expert,
    const int32_t* __restrict__ seg_offsets, int n_experts, int n_seg, int m_total, int t_x, int skip_rows) {
  using T = Fp8Tile<TS, WS, WT, WN, GROUPED, GLU>;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int wt = wave % WT, wn = wave / WT;
  const int nout = GLU ? n / 2 : n;

  // tile: XCD id mod 8 takes a contiguous run of tiles, activation tiles
  // fastest, so the workgroups of an XCD share weight rows in its L2
  const int total = gridDim.x;
  const int xcd = blockIdx.x & 7, share = total >> 3, extra = total & 7;
  const int id = xcd * share + min(xcd, extra) + (blockIdx.x >> 3);
  const int tiles_t = total / tiles_n;
  const int tn = id / tiles_t, tt = id % tiles_t;
  const int n0 = tn * T::kOut;

  int64_t m0, m_end;
  bool bad_expert = false;
  const uint8_t* wm = w;
  const float* wsm = ws;
  const int sb = GLU ? (nout + kFp8Block - 1) / kFp8Block : 0;
  if constexpr (GROUPED) {
    // the tt-th row tile of the segments longer than skip_rows
    __shared__ int32_t found[3];
    if (threadIdx.x < 64) {
      int before = 0, hit = -1, first = 0, end = 0;
      for (int s0 = 0; s0 < n_seg; s0 += 64) {
        const int s = s0 + lane;
        int lo = 0, hi = 0;
        if (s < n_seg) {
          lo = min(max(seg_offsets[s], 0), m_total);
          hi = min(max(seg_offsets[s + 1], lo), m_total);
        }
        const int tiles = hi - lo > skip_rows ? (hi - lo + T::kT - 1) / T::kT : 0;
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int up = __shfl_up(incl, o);
          if (lane >= o) incl += up;
        }
        const int at = before + incl - tiles;
        const bool mine = tt >= at && tt < at + tiles;
        const uint64_t who = __ballot(mine);
        if (who) {
          const int src = __builtin_ctzll(who);
          hit = s0 + src;
          first = __shfl(lo + (tt - at) * T::kT, src);
          end = __shfl(hi, src);
          break;
        }
        before += __shfl(incl, 63);
      }
      if (lane == 0) {
        found[0] = hit;
        found[1] = first;
        found[2] = end;
      }
    }
    __syncthreads();
    const int s = found[0];
    if (s < 0) return;                                  // fewer tiles than the grid's bound
    m0 = found[1];
    m_end = found[2];
    const int e = seg_expert[s];
    bad_expert = e < 0 || e >= n_experts;
    if (!bad_expert) {
      wm += int64_t(e) * n * d;
      wsm += int64_t(e) * (GLU ? 2 * sb : (n + kFp8Block - 1) / kFp8Block) * nb;
    }
  } else {
    m0 = int64_t(tt) * T::kT;
    m_end = min(t, m0 + T::kT);
  }

  // ---- copies: row 8·i + lane / 8 of a copy, LDS chunk lane % 8 holding the
  // global chunk (lane % 8) ^ (row % 8)
  const int crow = lane >> 3, cchunk = (lane & 7) ^ crow;
  uint32_t xoff[T::kXCopies], woff[T::kWCopies], soff = kOOB8;
  __amdgpu_buffer_rsrc_t xr, sr;
  auto source = [&](int64_t at) -> int {                // grouped: the row of x, or -1
    if (at >= m_end || bad_expert) return -1;
    const int src = row_index ? row_index[at] : int(at);
    return src < 0 || src >= t_x ? -1 : src;
  };
  if constexpr (GROUPED) {
    xr = make_rsrc(x, uint32_t(t_x) * uint32_t(d));
    sr = make_rsrc(xs, uint32_t(t_x) * uint32_t(nb) * 4u);
  } else {
    const uint32_t rows = uint32_t(m_end - m0);
    xr = make_rsrc(x + m0 * d, rows * uint32_t(d));
    sr = make_rsrc(xs + m0 * nb, rows * uint32_t(nb) * 4u);
  }
#pragma unroll
  for (int i = 0; i < T::kXCopies; ++i) {
    const int row = 8 * (wave * T::kXCopies + i) + crow;
    if constexpr (GROUPED) {
      const int src = source(m0 + row);
      xoff[i] = src >= 0 ? uint32_t(src) * uint32_t(d) : kOOB8;
    } else {
      xoff[i] = m0 + row < m_end ? uint32_t(row) * uint32_t(d) : kOOB8;
    }
  }
  if (wave < T::kT / 64) {                              // scales of 64 rows a wave
    const int row = 64 * wave + lane;
    if constexpr (GROUPED) {
      const int src = source(m0 + row);
      soff = src >= 0 ? uint32_t(src) * uint32_t(nb) * 4u : kOOB8;
    } else {
      soff = m0 + row < m_end ? uint32_t(row) * uint32_t(nb) * 4u : kOOB8;
    }
  }
  // weight rows: a wave's WS blocks are consecutive LDS rows; with the
  // activation their upper half comes from the up rows (8·WS rows are whole
  // copies, so a copy reads one of the two halves)
  const int live = min(T::kOut, nout - n0);
  const __amdgpu_buffer_rsrc_t wr0 = make_rsrc(wm + int64_t(n0) * d, uint32_t(live) * uint32_t(d));
  const __amdgpu_buffer_rsrc_t wr1 =
      GLU ? make_rsrc(wm + int64_t(nout + n0) * d, uint32_t(live) * uint32_t(d)) : wr0;
#pragma unroll
  for (int i = 0; i < T::kWCopies; ++i) {
    int row = 8 * (wave * T::kWCopies + i) + crow;
    if constexpr (GLU) row = row / (16 * WS) * (8 * WS) + row % (8 * WS);   // output column
    woff[i] = row < live ? uint32_t(row) * uint32_t(d) : kOOB8;
  }
  const uint32_t base = lds_addr(lds);
  auto copy = [&](int b, int stage) {
    const uint32_t at = base + uint32_t(stage) * T::kStage;
    const uint32_t k = uint32_t(kFp8Block * b + 16 * cchunk);
    const uint32_t ko = k < uint32_t(d) ? k : kOOB8;
#pragma unroll
    for (int i = 0; i < T::kXCopies; ++i)
      copy16_to_lds(xr, (xoff[i] + ko) | ((xoff[i] | ko) & kOOB8), at + 1024u * uint32_t(wave * T::kXCopies + i));
#pragma unroll
    for (int i = 0; i < T::kWCopies; ++i)
      copy16_to_lds(GLU && ((wave * T::kWCopies + i) / WS & 1) ? wr1 : wr0, (woff[i] + ko) | ((woff[i] | ko) & kOOB8),
                    at + 128u * T::kT + 1024u * uint32_t(wave * T::kWCopies + i));
    if (wave < T::kT / 64)
      copy4_to_lds(sr, soff + 4u * uint32_t(b), at + 128u * (T::kT + T::kN) + 256u * uint32_t(wave));
  };

  // ---- operands
  const float* ws0 = wsm + int64_t((n0 + (GLU ? 8 : 16) * WS * wn) / kFp8Block) * nb;
  const float* ws1 = wsm + int64_t(sb + (n0 + 8 * WS * wn) / kFp8Block) * nb;
  const int o0 = 16 * (g ^ (col & 7));
  f32x4_t acc[TS][WS];
#pragma unroll
  for (int i = 0; i < TS; ++i)
#pragma unroll
    for (int j = 0; j < WS; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  copy(0, 0);
  float w0 = ws0[0], w1 = GLU ? ws1[0] : 0.f;
  for (int b = 0; b < nb; ++b) {
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();                                    // step b copied; step b - 1 read by every wave
    const int next = min(b + 1, nb - 1);
    if (b + 1 < nb) copy(b + 1, (b + 1) & 1);
    const float w0n = ws0[next], w1n = GLU ? ws1[next] : 0.f;
    const unsigned char* st = lds + (b & 1) * T::kStage;
    const unsigned char* xt = st + 128 * (16 * TS * wt + col);
    const unsigned char* wt_ = st + 128 * (T::kT + 16 * WS * wn + col);
    const float* sc = reinterpret_cast<const float*>(st + 128 * (T::kT + T::kN)) + 16 * TS * wt + col;
    auto operand = [&](const unsigned char* p) {
      const u32x4_t lo = *reinterpret_cast<const u32x4_t*>(p + o0);
      const u32x4_t hi = *reinterpret_cast<const u32x4_t*>(p + (o0 ^ 64));
      i32x8_t r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[i] = int(lo[i]);
        r[4 + i] = int(hi[i]);
      }
      return r;
    };
    i32x8_t a[WS];
#pragma unroll
    for (int j = 0; j < WS; ++j) a[j] = operand(wt_ + 2048 * j);
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      const i32x8_t bx = operand(xt + 2048 * i);
      const float s = sc[16 * i];
      const float s0 = s * w0, s1 = GLU ? s * w1 : 0.f;
#pragma unroll
      for (int j = 0; j < WS; ++j) {
        const f32x4_t p = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a[j], bx, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                                           0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_fmaf(p[e], GLU && j >= WS / 2 ? s1 : s0, acc[i][j][e]);
      }
    }
    w0 = w0n;
    w1 = w1n;
  }

  // ---- epilogue: lane (col, g) holds output columns 4g .. 4g + 3 of activation row col
  const bool wide = (ldy & 3) == 0 && (reinterpret_cast<uintptr_t>(y) & 7) == 0;
  constexpr int WO = GLU ? WS / 2 : WS;
#pragma unroll
  for (int i = 0; i < TS; ++i) {
    const int64_t row = m0 + 16 * (TS * wt + i) + col;
    if (row >= m_end) continue;
    const bool bad = GROUPED && source(row) < 0;
#pragma unroll
    for (int j = 0; j < WO; ++j) {
      const int c = n0 + 16 * (WO * wn + j) + 4 * g;
      uint16_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float f = acc[i][j][e];
        if constexpr (GLU) f = silu(f) * acc[i][WO + j][e];
        v[e] = bad ? uint16_t(0x7FC0) : f32_to_bf16(f);
      }
      uint16_t* to = y + row * ldy + c;
      if (wide && c + 4 <= nout) {
        *reinterpret_cast<u32x2_t*>(to) =
            u32x2_t{uint32_t(v[0]) | uint32_t(v[1]) << 16, uint32_t(v[2]) | uint32_t(v[3]) << 16};
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < nout) to[e] = v[e];
      }
    }
  }
}

template <int TS, int WS, int WT, int WN, bool GROUPED, bool GLU>
int go(const Fp8GemmArgs& a, int skip_rows, hipStream_t s) {
  using T = Fp8Tile<TS, WS, WT, WN, GROUPED, GLU>;
  auto kernel = fp8_tile_kernel<TS, WS, WT, WN, GROUPED, GLU>;
  const size_t bytes = 2 * size_t(T::kStage);
  const int nout = GLU ? a.n / 2 : a.n;
  const int64_t tiles_n = (int64_t(nout) + T::kOut - 1) / T::kOut;
  // grouped: no more row tiles than whole tiles of rows and one part tile a segment
  const int64_t tiles_t = GROUPED ? int64_t(a.m_total) / T::kT + std::min<int64_t>(a.n_seg, a.m_total / (skip_rows + 1))
                                  : (a.t + T::kT - 1) / T::kT;
  if (tiles_t == 0) return 0;
  if (tiles_n * tiles_t >= (int64_t(1) << 22)) return int(hipErrorInvalidValue);
  launch_kernel_lds(kernel, dim3(unsigned(tiles_n * tiles_t)), dim3(64 * T::kWaves), bytes, s, a.w, a.ws, a.n, a.d,
                    fp8_blocks(a.d), a.x, a.xs, a.t, a.y, a.ldy, int(tiles_n), a.row_index, a.seg_expert,
                    a.seg_offsets, a.n_experts, a.n_seg, a.m_total, int(a.t_x), skip_rows);
  return int(hipGetLastError());
}

}  // namespace

int launch_fp8_tile(const Fp8GemmArgs& a, int skip_rows, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.n_seg > 0) return a.glu ? go<8, 4, 2, 4, true, true>(a, skip_rows, s) : go<8, 4, 2, 4, true, false>(a, skip_rows, s);
  return go<8, 4, 2, 4, false, false>(a, 0, s);
}

int launch_fp8_product(const Fp8GemmArgs& a, void* stream) {
  if (a.n_seg == 0) return a.t <= kFp8RowsMax ? launch_fp8_rows(a, 0, stream) : launch_fp8_tile(a, 0, stream);
  if (a.max_seg_rows <= kFp8RowsMax) return launch_fp8_rows(a, 0, stream);
  // two launches that split the segments on the device; armed events: the
  // start with the first, the stop with the second
  const ProfileEvents pe = take_profile_events();
  arm_profile_events({pe.start, nullptr});
  const int err = launch_fp8_rows(a, kFp8RowsMax, stream);
  arm_profile_events({nullptr, err ? nullptr : pe.stop});
  return err ? err : launch_fp8_tile(a, kFp8RowsMax, stream);
}

}  // namespace qmm
