// Microscaled 4-bit product for a few activation rows (a decode batch, routed segments): passes of
// up to 64 rows, 8 or 16 of a segment, each of which reads the weights once.
//
//   y[t,n] = Σ_b 2^(Ex[t,b] + Ew[n,b] - 254) · Σ_{k in b} x[t,k]·w[n,k]
//
// Bound by the weights' bytes, so the kernel is built to keep reads in flight: a workgroup
// takes 16·R weight rows, its waves split the reduction axis into equal runs of steps of 256
// codes, and every wave streams its steps through a private LDS ring of D stages (weights and
// activations, global -> LDS, no registers, no barriers): while one step is used, the next
// D - 1 are on their way.  A copy takes 8 rows of 128 bytes, whole cache lines; loads straight
// into the matrix instruction's operands have neighbouring lanes in different rows, which
// the memory pipeline takes one line at a time (47 x 5120 x 13824: 20.8 us so).  Exponents are copied
// a slab (two steps, 16 bytes a row) at a time into slots of their own.  The waves' sums are
// added in wave order through LDS: nothing depends on timing.
//
// Measured, weights of three matrices in turn, which the Infinity Cache holds, and of over 1.2 GB, from
// memory: 1 x 13824 x 5120 8.4 and 9.6 us (3.9 TB/s), 16 rows of it 8.8 and 10.3, 47 x 5120 x 13824
// 11.9 and 17.3, 64 x 4096 x 7168 6.7 and 8.8; SwiGLU 4096 x 3584 of 67 of 128 experts with a row or
// two 94 us (5.5 TB/s).
#include <hip/hip_runtime.h>

#include "qmm_fp8_tile.h"
#include "qmm_launch.h"
#include "qmm_lds_copy.h"
#include "qmm_mx4.h"
#include "qmm_mx4_device.h"
#include "qmm_segments.h"

#include <algorithm>

namespace qmm {
namespace {

struct Mx4RowsArgs {
  const uint8_t* codes;     // of the first matrix
  const uint8_t* meta;
  uint32_t codes_bytes, meta_bytes;
  int64_t expert_stride;
  int n, d;
  const uint8_t* x;
  const uint8_t* xs;
  int64_t t, ldy;
  uint16_t* y;
  bool fit;
  uint8_t* hq;
  uint8_t* hs;
  Fp8Grouped grp;
};

// WAVES waves split the reduction axis; R blocks of 16 weight rows, X8 groups of
// 8 activation rows, D ring stages.  GLU: the upper half of the R blocks are the
// up rows of the same outputs.
template <int WAVES, int R, int X8, int D, bool GROUPED, bool GLU>
struct Mx4Rows {
  static constexpr int C = (X8 + 1) / 2;                 // blocks of 16 activation rows
  static constexpr int RO = GLU ? R / 2 : R;             // blocks of output columns
  static constexpr int kOps = 2 * R + X8;                // copies of a stage
  static constexpr int kX = 2048 * R;                    // stage: weights, activations
  static constexpr int kStage = kX + 2048 * C;
  static constexpr int kChunk = 2048, kChunks = (D + 1) / 2;   // exponents of a slab: weights, activations
  static constexpr int kWave = D * kStage + kChunks * kChunk;
  static constexpr int kRing = WAVES * kWave, kPart = WAVES * R * C * 1024;
  static constexpr int kLds = kRing > kPart ? kRing : kPart;
  static_assert(!GLU || R % 2 == 0, "gate and up blocks come in pairs");
  static_assert(R <= 4 && X8 <= 8, "the exponents of either side are one copy");
  // of the D - 1 steps behind one, (D - 1) / 2 begin a slab and bring its exponents
  static_assert(D % 2 == 1 && (D - 1) * (kOps + 1) <= 63, "the waits count the copies in flight");
  static_assert(kRing == mx4_rows_lds(R, X8, WAVES) || D != kMxRing, "the host's count");
  static_assert(kLds <= 160 * 1024, "LDS");
};

template <int WAVES, int R, int X8, int D, bool GROUPED, bool GLU>
__global__ __launch_bounds__(64 * WAVES, 2) void mx4_rows_kernel(Mx4RowsArgs A) {
  using T = Mx4Rows<WAVES, R, X8, D, GROUPED, GLU>;
  constexpr int C = T::C, RO = T::RO, kRows = 8 * X8;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int n = A.n, d = A.d, nout = GLU ? n / 2 : n;
  const int n0 = blockIdx.x * 16 * RO;             // first output column
  const Slabs L{n, d, QMM_MXFP4_G32};
  const int steps = mx_steps(d), last = L.count() - 1;
  const int width = L.width(0) / 2, width_last = L.width(last) / 2;
  const int meta_row = L.meta_row(0), meta_last = L.meta_row(last);
  const uint32_t slab_bytes = uint32_t(n) * (kSlabCodes / 2);   // of a slab that another follows
  const uint32_t xstride = uint32_t(d) / 2, sstride = uint32_t(mx_scale_bytes(d));

  // grouped: the workgroups of a column share out the segments
  Fp8Segments segments;
  for (int turn = blockIdx.y;; turn += gridDim.y) {
    int64_t m_begin, m_end;
    bool bad_expert = false;
    const uint8_t *codes = A.codes, *meta = A.meta;
    if constexpr (GROUPED) {
      const int s = segments.find(turn, A.grp, A.grp.n_seg);
      if (s < 0) return;
      m_begin = min(max(A.grp.seg_offsets[s], 0), A.grp.m_total);
      m_end = min(max(A.grp.seg_offsets[s + 1], int(m_begin)), A.grp.m_total);
      const int e = A.grp.seg_expert[s];
      bad_expert = e < 0 || e >= A.grp.n_experts;
      if (!bad_expert) {
        codes += int64_t(e) * A.expert_stride;
        meta += int64_t(e) * A.expert_stride;
      }
    } else {
      m_begin = int64_t(turn) * kRows;
      if (m_begin >= A.t) return;
      m_end = min(A.t, m_begin + kRows);
    }

    // Copies: lane / 8 is the row of a copy's eight, LDS piece lane % 8 holds the row's
    // 16-byte piece (lane % 8) ^ (row % 8), so that the operand reads of eight neighbouring
    // rows fall into different banks.
    const int crow = lane >> 3, cpiece = (lane & 7) ^ crow;
    const int live = min(16 * RO, nout - n0);
    // packed row of row `row` of the workgroup's 16·R; -1 past the matrix
    auto w_row = [&](int row) {
      const int up = GLU && row >= 16 * RO ? nout : 0;
      if constexpr (GLU) row %= 16 * RO;
      return row < live ? up + n0 + row : -1;
    };
    // Offsets in slab 0; later slabs and the second half of one are a scalar offset further.
    // The last slab's rows may be narrower: theirs are worked out again.
    auto w_offset = [&](int i, int in_copy, int bytes) {
      const int row = w_row(8 * i + in_copy);
      return row >= 0 ? uint32_t(row) * uint32_t(bytes) + 16u * uint32_t(cpiece) : kOOB8;
    };
    auto m_offset = [&](int row_of, int bytes) {
      const int row = row_of < 16 * R ? w_row(row_of) : -1;
      return row >= 0 ? uint32_t(row >> 2) * uint32_t(L.meta_quad()) + uint32_t(row & 3) * uint32_t(bytes) : kOOB8;
    };
    uint32_t woff[2 * R];
#pragma unroll
    for (int i = 0; i < 2 * R; ++i) woff[i] = w_offset(i, crow, width);
    const uint32_t moff = m_offset(lane, meta_row);

    // the wave's share of the reduction axis, and its ring
    const int b_begin = steps * wave / WAVES, b_end = steps * (wave + 1) / WAVES;
    const unsigned char* ring = lds + wave * T::kWave;
    const uint32_t ring_at = lds_addr(ring);
    const int o0 = 128 * col + 16 * ((2 * g) ^ (col & 7)), o1 = 128 * col + 16 * ((2 * g + 1) ^ (col & 7));

    for (int64_t m0 = m_begin; m0 < m_end; m0 += kRows) {
      // activation rows: dense rows are based at the pass's first row; grouped
      // rows can be anywhere in x (below 2 GiB, checked by the caller)
      const int64_t x_first = GROUPED ? 0 : m0;
      const uint32_t x_rows = GROUPED ? uint32_t(A.grp.t_x) : uint32_t(min(int64_t(kRows), m_end - m0));
      const uint8_t* xp = A.x + x_first * xstride;
      const uint8_t* sp = A.xs + x_first * sstride;
      auto source = [&](int row) -> int {            // the row of x (dense: of the pass), or -1
        if (m0 + row >= m_end) return -1;
        if constexpr (!GROUPED) return row;
        const int src = A.grp.row_index ? A.grp.row_index[m0 + row] : int(m0 + row);
        return bad_expert || src < 0 || src >= A.grp.t_x ? -1 : src;
      };
      uint32_t xoff[X8];
#pragma unroll
      for (int i = 0; i < X8; ++i) {
        const int src = source(8 * i + crow);
        xoff[i] = src >= 0 ? uint32_t(src) * xstride + 16u * uint32_t(cpiece) : kOOB8;
      }
      const int mine = lane < kRows ? source(lane) : -1;
      const uint32_t soff = mine >= 0 ? uint32_t(mine) * sstride : kOOB8;
      const __amdgpu_buffer_rsrc_t cr = make_rsrc(codes, A.codes_bytes), mr = make_rsrc(meta, A.meta_bytes);
      const __amdgpu_buffer_rsrc_t xr = make_rsrc(xp, x_rows * xstride), sr = make_rsrc(sp, x_rows * sstride);
      // The copies of step b into a stage; past the wave's share, and for pieces past d, the
      // lanes' offsets are out of range (zeros, no reads, the same count of copies).  The same
      // four buffers throughout: more scalar registers would be spilled, and a copy must not
      // follow a scalar's way back from a vector register too closely.
      auto copy = [&](int b, int stage) {
        const bool in = b < b_end;
        const int s = b >> 1;
        const uint32_t at = ring_at + uint32_t(stage * T::kStage);
        const uint32_t past = in && kMxStep * b + kMxBlock * cpiece < d ? 0u : kOOB8;
        const uint32_t from = in ? uint32_t(s) * slab_bytes + 128u * uint32_t(b & 1) : 0u;
        if (s == last && width_last != width) {
          int in_copy = crow;
          asm volatile("" : "+v"(in_copy));               // not worked out before the loop: registers
#pragma unroll
          for (int i = 0; i < 2 * R; ++i)
            copy16_to_lds_from(cr, w_offset(i, in_copy, width_last) | past, from, at + 1024u * i);
        } else {
#pragma unroll
          for (int i = 0; i < 2 * R; ++i) copy16_to_lds_from(cr, woff[i] | past, from, at + 1024u * i);
        }
#pragma unroll
        for (int i = 0; i < X8; ++i)
          copy16_to_lds_from(xr, xoff[i] | past, in ? 128u * uint32_t(b) : 0u, at + T::kX + 1024u * i);
      };
      // the exponents of a slab, before its first step of the wave's
      auto slot = [&](int b) { return uint32_t(D * T::kStage + ((b >> 1) - (b_begin >> 1)) % T::kChunks * T::kChunk); };
      auto copy_scales = [&](int b) {
        const bool in = b < b_end;
        const int s = b >> 1;
        const uint32_t past = in ? 0u : kOOB8, at = ring_at + slot(b);
        uint32_t off = moff;
        if (s == last && meta_last != meta_row) {
          int row = lane;
          asm volatile("" : "+v"(row));
          off = m_offset(row, meta_last);
        }
        copy16_to_lds_from(mr, off | past, in ? 64u * uint32_t(s) : 0u, at);
        copy16_to_lds_from(sr, soff | past, in ? 16u * uint32_t(s) : 0u, at + 1024u);
      };

      f32x4_t acc[R][C];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};

      // D steps ahead of the first use; the same code fills the ring and refills it
      int stage = 0;
      int from_step = b_begin - D;
      asm volatile("" : "+s"(from_step));   // the filling is not taken apart: scalar registers
      for (int b = from_step; b < b_end; ++b) {
        const bool use = b >= b_begin;
        u32x4_t a[R][2], x2[C][2];
        uint32_t sa[R], sx[C];
        if (use) {
          // step b has landed: D - 1 steps are in flight behind it, every other with exponents
          wait_copies<(D - 1) * T::kOps + (D - 1) / 2 * 2>();
          const unsigned char* st = ring + stage * T::kStage;
          const unsigned char* sc = ring + slot(b) + 16 * col + 8 * (b & 1) + 2 * g;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            a[r][0] = *reinterpret_cast<const u32x4_t*>(st + 2048 * r + o0);
            a[r][1] = *reinterpret_cast<const u32x4_t*>(st + 2048 * r + o1);
            sa[r] = *reinterpret_cast<const uint16_t*>(sc + 256 * r);
          }
#pragma unroll
          for (int c = 0; c < C; ++c) {
            x2[c][0] = *reinterpret_cast<const u32x4_t*>(st + T::kX + 2048 * c + o0);
            x2[c][1] = *reinterpret_cast<const u32x4_t*>(st + T::kX + 2048 * c + o1);
            sx[c] = *reinterpret_cast<const uint16_t*>(sc + 1024 + 256 * c);
          }
          wait_reads();                     // ... and is in registers: its stage is free
        }
        if (((b + D) & 1) == 0 || b + D == b_begin) copy_scales(b + D);
        copy(b + D, stage);
        stage = stage + 1 == D ? 0 : stage + 1;
        if (use) {
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              acc[r][c] = mfma_fp4<0, 0>(a[r][0], x2[c][0], acc[r][c], sa[r], sx[c]);
              acc[r][c] = mfma_fp4<1, 1>(a[r][1], x2[c][1], acc[r][c], sa[r], sx[c]);
            }
        }
      }

      // the ring becomes the waves' sums: [wave][R·C][64], a lane's place changed so
      // that the eight lanes of a row read different banks
      wait_copies<0>();
      __syncthreads();
      f32x4_t* part = reinterpret_cast<f32x4_t*>(lds);
      auto place = [](int r, int l) { return l ^ r ^ (l >> 5 << 2); };
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) part[(wave * R * C + r * C + c) * 64 + place(r, lane)] = acc[r][c];
      __syncthreads();
      auto summed = [&](int r, int c, int l) {
        f32x4_t v = part[(r * C + c) * 64 + place(r, l)];
#pragma unroll
        for (int p = 1; p < WAVES; ++p) {
          const f32x4_t o = part[((p * R + r) * C + c) * 64 + place(r, l)];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += o[i];
        }
        return v;
      };
      // eight columns of a row a thread: a row's stores are next to each other
      const uint64_t no_source = __ballot(soff == kOOB8);
      for (int q = threadIdx.x; q < kRows * 2 * RO; q += 64 * WAVES) {
        const int row = q / (2 * RO), chunk = q % (2 * RO), r = chunk >> 1, l = 32 * (chunk & 1) + (row & 15);
        if (m0 + row >= m_end) break;
        const bool bad = GROUPED && (no_source >> row & 1);
        f32x4_t v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v[h] = summed(r, row >> 4, l + 16 * h);
          if constexpr (GLU) {
            const f32x4_t up = summed(r + RO, row >> 4, l + 16 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[h][i] = silu(v[h][i]) * up[i];
          }
        }
        if constexpr (GLU && RO == 2) {
          if (A.hq) {
            // the four threads of a row have a block of 32 columns
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = umax(m, __float_as_uint(v[i >> 2][i & 3]) & 0x7FFFFFFFu);
            m = umax(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0xB1, 0xF, 0xF, false)));
            m = umax(m, uint32_t(__builtin_amdgcn_update_dpp(0, int(m), 0x4E, 0xF, 0xF, false)));
            const uint32_t ex = mx_exponent(bad ? 0x7FC00000u : m, A.fit);
            uint32_t o = 0;
            if (ex != 255u) {
              const float scale = mx_scale(ex);
              o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[0][0], v[0][1], scale, 0);
              o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[0][2], v[0][3], scale, 1);
              o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[1][0], v[1][1], scale, 2);
              o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[1][2], v[1][3], scale, 3);
            }
            const int64_t out = m0 + row;
            *reinterpret_cast<uint32_t*>(A.hq + out * (nout / 2) + n0 / 2 + 4 * chunk) = o;
            uint8_t* hs = A.hs + out * mx_scale_bytes(nout);
            if (chunk == 0) hs[n0 / 32] = uint8_t(ex);
            if (n0 + 32 == nout)           // zeros past the row's blocks
              for (int b = nout / 32 + chunk; b < mx_scale_bytes(nout); b += 4) hs[b] = 0;
            continue;
          }
        }
        u32x4_t v16{pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]), pack_bf16x2(v[1][0], v[1][1]),
                    pack_bf16x2(v[1][2], v[1][3])};
        if (bad) v16 = u32x4_t{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
        store8(A.y + (m0 + row) * A.ldy, n0 + 8 * chunk, nout, v16);
      }
      __syncthreads();   // the next pass fills the ring again
    }
  }
}

template <int WAVES, int R, int X8, bool GROUPED, bool GLU>
int go(const Mx4GemmArgs& a, hipStream_t s) {
  using T = Mx4Rows<WAVES, R, X8, kMxRing, GROUPED, GLU>;
  Layout l;
  if (!layout_of(QMM_MXFP4_G32, a.n, a.d, &l)) return int(hipErrorInvalidValue);
  const int nout = GLU ? a.n / 2 : a.n, per = 16 * T::RO;
  const int64_t tiles = (nout + per - 1) / per;
  int64_t gy = std::min<int64_t>((a.t + 8 * X8 - 1) / (8 * X8), 65535);   // the grid's limit: more take turns
  if (GROUPED) {
    // no more segments than rows have any; two rounds of the workgroups that the LDS lets
    // 256 CUs hold, each taking several segments
    const int64_t resident = 2 * 256 * (160 * 1024 / T::kLds);
    gy = std::max<int64_t>(1, std::min<int64_t>(std::min(a.n_seg, a.m_total), resident / tiles));
  }
  const Mx4RowsArgs k{a.packed + l.codes_offset, a.packed + l.meta_offset, uint32_t(int64_t(a.n) * (a.d / 2)),
                      uint32_t(l.meta_bytes), a.expert_stride, a.n, a.d, a.x, a.xs, a.t, a.ldy, a.y, a.fit, a.hq, a.hs,
                      Fp8Grouped{a.row_index, a.seg_expert, a.seg_offsets, a.n_experts, a.m_total, int(a.t_x), a.n_seg}};
  launch_kernel_lds((mx4_rows_kernel<WAVES, R, X8, kMxRing, GROUPED, GLU>), dim3(unsigned(tiles), unsigned(gy)),
                    dim3(64 * WAVES), T::kLds, s, k);
  return int(hipGetLastError());
}

template <int R>
int dense(int x8, const Mx4GemmArgs& a, hipStream_t s) {
  switch (x8) {
    case 1: return go<mx4_rows_waves(R, 1), R, 1, false, false>(a, s);
    case 2: return go<mx4_rows_waves(R, 2), R, 2, false, false>(a, s);
    case 4: return go<mx4_rows_waves(R, 4), R, 4, false, false>(a, s);
    case 6: return go<mx4_rows_waves(R, 6), R, 6, false, false>(a, s);
    default: break;
  }
  if constexpr (R > 1) return go<mx4_rows_waves(R, 8), R, 8, false, false>(a, s);
  return int(hipErrorInvalidValue);
}

}  // namespace

int launch_mx4_rows(const Mx4GemmArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.n_seg > 0) {
    const Mx4GroupedShape p = mx4_grouped_shape(a);
    if (!a.glu) return p.x8 == 1 ? go<2, 2, 1, true, false>(a, s) : go<2, 2, 2, true, false>(a, s);
    if (p.waves == 4) return go<4, 4, 1, true, true>(a, s);
    return p.x8 == 1 ? go<2, 4, 1, true, true>(a, s) : go<2, 4, 2, true, true>(a, s);
  }
  const Mx4RowsShape p = mx4_rows_shape(a.t, a.n, a.d);
  return p.r == 1 ? dense<1>(p.x8, a, s) : p.r == 2 ? dense<2>(p.x8, a, s) : dense<4>(p.x8, a, s);
}

}  // namespace qmm
