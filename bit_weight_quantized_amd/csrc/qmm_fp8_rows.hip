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
//
// Measured: 1 x 13824 x 5120 12.6 us (5.6 TB/s), 16 rows of it 13.3; 37 x 5120 x 13824
// 16.4 to 16.8 us (4.3), 64 rows 19.9 (3.7; the activations come again from L2 for every 32
// weight rows); SwiGLU, 25 of 128 experts with a row or two, 4096 x 3584 65.4 us (5.6);
// all with a part of the weights in the Infinity Cache.
#include <hip/hip_runtime.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"
#include "qmm_fp8_tile.h"
#include "qmm_launch.h"
#include "qmm_lds_copy.h"

#include <algorithm>

namespace qmm {
namespace {

struct Fp8Grouped {
  const int32_t* row_index;
  const int32_t* seg_expert;
  const int32_t* seg_offsets;
  int n_experts, m_total;
  int t_x;
  int n_seg;
};

// The i-th segment that has rows, for ascending i:
// 256 segments at a time, one bit each.
struct Fp8Segments {
  int s0 = -256, before = 0;
  uint64_t m[4] = {0, 0, 0, 0};

  __device__ __forceinline__ int find(int i, const Fp8Grouped& grp, int n_seg) {
    const int lane = threadIdx.x & 63;
    for (;;) {
      int r = i - before, found = -1;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = __builtin_popcountll(m[u]);
        if (found < 0 && r < c) {
          const int rank = __builtin_amdgcn_mbcnt_hi(uint32_t(m[u] >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(m[u]), 0));
          found = s0 + 64 * u + __builtin_ctzll(__ballot(((m[u] >> lane) & 1) && rank == r));
        }
        r -= c;
      }
      if (found >= 0) return found;
      before = i - r;
      s0 += 256;
      if (s0 >= n_seg) return -1;
      int rows[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int s = min(s0 + 64 * u + lane, n_seg - 1);
        const int lo = min(max(grp.seg_offsets[s], 0), grp.m_total);
        rows[u] = min(max(grp.seg_offsets[s + 1], lo), grp.m_total) - lo;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        m[u] = __ballot(s0 + 64 * u + lane < n_seg && rows[u] > 0);
    }
  }
};

// WAVES waves split the reduction axis; R blocks of 16 weight rows, X8 groups of
// 8 activation rows, D ring stages.  GLU: the upper half of the R blocks are the
// up rows of the same outputs.
template <int WAVES, int R, int X8, int D, bool GROUPED, bool GLU>
struct Fp8Rows {
  static constexpr int C = (X8 + 1) / 2;                 // blocks of 16 activation rows
  static constexpr int RO = GLU ? R / 2 : R;             // blocks of output columns
  static constexpr bool kExact = C == 1;
  static constexpr int kOps = 2 * R + X8;                // copies of a stage
  static constexpr int kX = 2048 * R;                    // stage: weights, activations
  static constexpr int kStage = kX + 2048 * C;
  static constexpr int kSc = (X8 * 8 + 63) / 64;         // copies of the scales of four blocks
  static constexpr int kChunk = 1024 * kSc, kChunks = (D + 3) / 4 + 1;
  static constexpr int kWave = D * kStage + kChunks * kChunk;
  static constexpr int kRing = WAVES * kWave, kPart = WAVES * R * C * 1024;
  static constexpr int kLds = kRing > kPart ? kRing : kPart;
  static_assert(!GLU || R % 2 == 0, "gate and up blocks come in pairs");
  static_assert(kSc == 1 && D <= 4 && (D - 1) * kOps + kSc <= 63, "the waits count the copies in flight");
  static_assert(kLds <= 160 * 1024, "LDS");
};

template <int WAVES, int R, int X8, int D, bool GROUPED, bool GLU>
__global__ __launch_bounds__(64 * WAVES, 2) void fp8_rows_kernel(
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

  // grouped: the workgroups of a column share out the segments
  Fp8Segments segments;
  for (int turn = blockIdx.y;; turn += gridDim.y) {
    int64_t m_begin, m_end;
    bool bad_expert = false;
    const uint8_t* wm = w;
    const float* wsm = ws;
    const int sb = GLU ? (nout + kFp8Block - 1) / kFp8Block : 0;   // scale rows of the gate half
    if constexpr (GROUPED) {
      const int s = segments.find(turn, grp, grp.n_seg);
      if (s < 0) return;
      m_begin = min(max(grp.seg_offsets[s], 0), grp.m_total);
      m_end = min(max(grp.seg_offsets[s + 1], int(m_begin)), grp.m_total);
      const int e = grp.seg_expert[s];
      bad_expert = e < 0 || e >= grp.n_experts;
      if (!bad_expert) {
        wm += int64_t(e) * n * d;
        wsm += int64_t(e) * (GLU ? 2 * sb : (n + kFp8Block - 1) / kFp8Block) * nb;
      }
    } else {
      m_begin = int64_t(turn) * kRows;
      if (m_begin >= t) return;
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
    const uint8_t* w0p = wm + int64_t(n0) * d;
    const uint8_t* w1p = GLU ? wm + int64_t(nout + n0) * d : w0p;
    const uint32_t w_bytes = uint32_t(live) * uint32_t(d);
    uint32_t woff[2 * RO];
#pragma unroll
    for (int i = 0; i < 2 * RO; ++i)
      woff[i] = 8 * i + crow < live ? uint32_t(8 * i + crow) * uint32_t(d) + uint32_t(cchunk) : kOOB8;

    // the wave's share of the reduction axis, and its ring
    const int b_begin = nb * wave / WAVES, b_end = nb * (wave + 1) / WAVES;
    const unsigned char* ring = lds + wave * T::kWave;
    const uint32_t ring_at = lds_addr(ring);
    const int o0 = 128 * col + 16 * (g ^ (col & 7));       // operand chunks g and g + 4 of row col

    for (int64_t m0 = m_begin; m0 < m_end; m0 += kRows) {
      // activation rows: dense rows are based at the pass's first row; grouped
      // rows can be anywhere in x (below 2 GiB, checked by the caller)
      const int64_t x_first = GROUPED ? 0 : m0;
      const uint32_t x_rows = GROUPED ? uint32_t(grp.t_x) : uint32_t(min(int64_t(kRows), m_end - m0));
      const uint8_t* xp = x + x_first * d;
      const float* sp = xs + x_first * nb;
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
        xoff[i] = src >= 0 ? uint32_t(src) * uint32_t(d) + uint32_t(cchunk) : kOOB8;
      }
#pragma unroll
      for (int i = 0; i < T::kSc; ++i) {
        const int src = 64 * i + lane < kRows ? source(64 * i + lane) : -1;
        soff[i] = src >= 0 ? uint32_t(src) * uint32_t(nb) * 4u : kOOB8;
      }
      // Copy `i` of block b into a stage.  A code's block is the scalar offset, so the
      // lanes' offsets stay as they are; past the wave's share the buffers are empty
      // (zeros, no reads, the same count of copies), and in a short last block the
      // chunks past d are out of range.
      struct Cursor {
        bool in;
        uint32_t at, k, past;
        uint32_t chunk;   // where the scales of its four blocks are
      };
      auto cursor = [&](int b, int stage) {
        return Cursor{b < b_end, ring_at + uint32_t(stage * T::kStage), fp8_block_at(b, b_end), fp8_past(cchunk, b, d),
                      uint32_t(D * T::kStage + ((b - b_begin) >> 2) % T::kChunks * T::kChunk)};
      };
      auto copy = [&](const Cursor& c, int i) {
        if (i < 2 * R)
          copy16_to_lds_from(make_rsrc(i < 2 * RO ? w0p : w1p, c.in ? w_bytes : 0u), woff[i % (2 * RO)] | c.past, c.k,
                             c.at + 1024u * i);
        else
          copy16_to_lds_from(make_rsrc(xp, c.in ? x_rows * uint32_t(d) : 0u), xoff[(i - 2 * R) % X8] | c.past, c.k,
                             c.at + T::kX + 1024u * (i - 2 * R));
      };
      // The scales of four blocks at once, before the first of them (rows lie far
      // apart: a copy costs a cache line for each row, whatever it takes of it).  The
      // last row may have fewer left: what is past the buffer reads zero.
      auto copy_scales = [&](const Cursor& c, int b) {
#pragma unroll
        for (int i = 0; i < T::kSc; ++i)
          copy16_to_lds(make_rsrc(sp, c.in ? x_rows * uint32_t(nb) * 4u : 0u), fp8_scales_at(soff[i], b),
                        ring_at + c.chunk + 1024u * i);
      };

      f32x4_t acc[R][C];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) acc[r][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll
      for (int i = 0; i < D; ++i) {
        const Cursor c = cursor(b_begin + i, i);
        if (i == 0) copy_scales(c, b_begin);
#pragma unroll
        for (int k = 0; k < T::kOps; ++k) copy(c, k);
      }
      float w0 = scalar_load(ws0, min(b_begin, nb - 1)), w1 = GLU ? scalar_load(ws1, min(b_begin, nb - 1)) : 0.f;
      int stage = 0;
      for (int b = b_begin; b < b_end; ++b) {
        const int next = min(b + 1, nb - 1);
        const float w0n = scalar_load(ws0, next), w1n = GLU ? scalar_load(ws1, next) : 0.f;
        // block b has landed: D - 1 blocks are in flight behind it, and scales if one
        // of them is the first of four
        if (((b - b_begin) & 3) + D - 1 >= 4)
          wait_copies<(D - 1) * T::kOps + T::kSc>();
        else
          wait_copies<(D - 1) * T::kOps>();
        const unsigned char* st = ring + stage * T::kStage;
        const float* sc = reinterpret_cast<const float*>(ring + cursor(b, 0).chunk) + ((b - b_begin) & 3);
        u32x4_t a[R][2], x2[C][2];
        float s[C];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            a[r][h] = *reinterpret_cast<const u32x4_t*>(st + 2048 * r + (o0 ^ (64 * h)));
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
          for (int h = 0; h < 2; ++h) x2[c][h] = *reinterpret_cast<const u32x4_t*>(st + T::kX + 2048 * c + (o0 ^ (64 * h)));
          s[c] = sc[4 * (16 * c + col)];
        }
        wait_reads();                       // ... and is in registers: its stage is free
        const Cursor nx = cursor(b + D, stage);
        stage = stage + 1 == D ? 0 : stage + 1;
        if (((b + D - b_begin) & 3) == 0) copy_scales(nx, b + D);
        if constexpr (T::kExact) {
#pragma unroll
          for (int k = 0; k < T::kOps; ++k) copy(nx, k);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const f32x4_t p = mfma_e4m3_exact(join(a[r][0], a[r][1]), join(x2[0][0], x2[0][1]));
            const float sv = s[0] * (r < RO ? w0 : w1);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][0][i] = __builtin_fmaf(p[i], sv, acc[r][0][i]);
          }
        } else {
          // block sums, their multiply-adds two matrix instructions later, and the
          // copies spread between them: a copy holds the wave while the memory
          // pipeline is busy, the matrix unit works on meanwhile
          constexpr int N = R * C, kAhead = 2;
          f32x4_t p[kAhead + 1];
#pragma unroll
          for (int m = 0; m < N + kAhead; ++m) {
            if (m < N) p[m % (kAhead + 1)] = mfma_e4m3(join(a[m % R][0], a[m % R][1]), join(x2[m / R][0], x2[m / R][1]));
#pragma unroll
            for (int k = 0; k < T::kOps; ++k)
              if (k * N / T::kOps == m) copy(nx, k);
            if (m >= kAhead) {
              const int u = m - kAhead, r = u % R, c = u / R;
              const float sv = s[c] * (r < RO ? w0 : w1);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[r][c][i] = __builtin_fmaf(p[u % (kAhead + 1)][i], sv, acc[r][c][i]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        w0 = w0n;
        w1 = w1n;
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
      const uint64_t no_source = __ballot(soff[0] == kOOB8);
      for (int q = threadIdx.x; q < kRows * 2 * RO; q += 64 * WAVES) {
        const int row = q / (2 * RO), chunk = q % (2 * RO), r = chunk >> 1, l = 32 * (chunk & 1) + (row & 15);
        if (m0 + row >= m_end) break;
        u32x4_t v16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4_t v = summed(r, row >> 4, l + 16 * h);
          if constexpr (GLU) {
            const f32x4_t up = summed(r + RO, row >> 4, l + 16 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = silu(v[i]) * up[i];
          }
          v16[2 * h] = pack_bf16x2(v[0], v[1]);
          v16[2 * h + 1] = pack_bf16x2(v[2], v[3]);
        }
        if (GROUPED && (no_source >> row & 1)) v16 = u32x4_t{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
        store8(y + (m0 + row) * ldy, n0 + 8 * chunk, nout, v16);
      }
      __syncthreads();   // the next pass fills the ring again
    }
  }
}

constexpr int kDepth = 2;   // a deeper ring measured no faster anywhere

template <int WAVES, int R, int X8, bool GROUPED, bool GLU>
int go(const Fp8GemmArgs& a, hipStream_t s) {
  using T = Fp8Rows<WAVES, R, X8, kDepth, GROUPED, GLU>;
  const int nout = GLU ? a.n / 2 : a.n, per = 16 * T::RO;
  const Fp8Grouped grp{a.row_index, a.seg_expert, a.seg_offsets, a.n_experts, a.m_total, int(a.t_x), a.n_seg};
  const int64_t tiles = (nout + per - 1) / per;
  int64_t gy = std::min<int64_t>((a.t + 8 * X8 - 1) / (8 * X8), 65535);   // the grid's limit: more take turns
  if (GROUPED) {
    // no more segments than rows have any; two rounds of the workgroups that the
    // LDS lets 256 CUs hold, each taking several segments (one workgroup for each
    // of 896 segments and 112 columns, 8 of them with a row: 36.6 us, 6.6 shared)
    const int64_t resident = 2 * 256 * (160 * 1024 / T::kLds);
    gy = std::max<int64_t>(1, std::min<int64_t>(std::min(a.n_seg, a.m_total), resident / tiles));
  }
  launch_kernel_lds(fp8_rows_kernel<WAVES, R, X8, kDepth, GROUPED, GLU>, dim3(unsigned(tiles), unsigned(gy)),
                    dim3(64 * WAVES), T::kLds, s, a.w, a.ws, a.n, a.d, fp8_blocks(a.d), a.x, a.xs, a.t, a.y, a.ldy, grp);
  return int(hipGetLastError());
}

int dense8(int x8, const Fp8GemmArgs& a, hipStream_t s) {
  if (x8 == 4) return go<8, 1, 4, false, false>(a, s);
  return x8 == 1 ? go<8, 1, 1, false, false>(a, s) : go<8, 1, 2, false, false>(a, s);
}

template <int R>
int dense(int x8, const Fp8GemmArgs& a, hipStream_t s) {
  if (x8 == 4) return go<4, R, 4, false, false>(a, s);
  if (x8 == 8) return go<4, R, 8, false, false>(a, s);
  if constexpr (R <= 2) return x8 == 1 ? go<4, R, 1, false, false>(a, s) : go<4, R, 2, false, false>(a, s);
  return int(hipErrorInvalidValue);
}

template <bool GLU>
int grouped(const Fp8RowsShape& p, const Fp8GemmArgs& a, hipStream_t s) {
  return p.waves == 4 ? go<4, 2, 1, true, GLU>(a, s) : go<2, 2, 1, true, GLU>(a, s);
}

}  // namespace

int launch_fp8_rows(const Fp8GemmArgs& a, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  const Fp8RowsShape p = fp8_rows_shape(a);
  if (a.n_seg == 0 && p.waves == 8) return dense8(p.x8, a, s);
  if (a.n_seg == 0) return p.r == 4 ? dense<4>(p.x8, a, s) : p.r == 2 ? dense<2>(p.x8, a, s) : dense<1>(p.x8, a, s);
  return a.glu ? grouped<true>(p, a, s) : grouped<false>(p, a, s);
}

}  // namespace qmm
