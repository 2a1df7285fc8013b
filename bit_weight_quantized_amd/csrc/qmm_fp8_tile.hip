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
// Both tiles go global -> LDS without passing registers, double-buffered.  A
// row's eight 16-byte chunks are stored at chunk ^ (row mod 8), done on the
// global side of the copy, so the operand reads of eight neighbouring rows fall
// into different banks.
//
// Two groups of waves work in opposite phases: while one reads the operands of half a
// step from LDS, the other multiplies, with a barrier between phases, so the matrix
// unit does not wait for LDS.  (The eight waves of a 256 x 256 tile are two on every
// SIMD; a 64 x 128 tile has four, and three such workgroups share a CU.)  A wave's
// step is
//   L1: read its weights and the first half of its activations   C1: multiply
//   L2: read the second half of its activations                  C2: multiply
// and the waves of the second group run one phase behind.  A part of the tiles
// that both groups have read is filled again at once: L1 of step b issues the
// second half of the activations of step b + 1, L2 the weights and the first half
// of step b + 2, so every copy has four phases to land, counted by vmcnt: after
// the copies that a phase needs, each wave has issued one set of each, kAfter
// copies, and never waits for the last ones.  (Two phases a step, with the second
// half read between the multiplications, were 4% slower: less time to land.)
//
// Bound by the matrix unit for long reductions, by a tile's start and end (4 and 3 us
// of 256 x 256) for short ones, and by the clock, which falls to 1.9 .. 2.0 GHz under
// this load, by what the codes are: 8192 x 8192 x 8192 423 us (2.60 PFLOP/s), 2048 x
// 13824 x 5120 126 to 141 us (2.30 to 2.06; 432 tiles in two rounds of 256 CUs), 64
// experts of 4096 x 3584 with 32768 rows 533 us (1.80).  256 x 256 is the largest tile whose fp32 sums leave registers
// for the operands (230 of 256); it reads half the bytes of 128 x 128 for a product.
#include <hip/hip_runtime.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"
#include "qmm_fp8_tile.h"
#include "qmm_launch.h"
#include "qmm_lds_copy.h"

#include <algorithm>
#include <type_traits>

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
  static constexpr int kStage = (kT + kN) * 128;       // both tiles of a step
  static constexpr int kScales = kT * 16;              // activation scales of four steps
  static constexpr int kBad = 2 * kStage + 2 * kScales;   // a bit for every row without a source
  static constexpr int kLds = kBad + kT / 8;
  static_assert(kT * kOut * 2 <= 2 * kStage, "the output tile takes the place of the operands'");
  static_assert(kT / 16 % kWaves == 0 && kN / 8 % kWaves == 0 && kT / 64 <= kWaves, "whole copies per wave");
  static constexpr int kXCopies = kT / 16 / kWaves, kWCopies = kN / 8 / kWaves;   // of half the activations
  static constexpr int kAfter = 2 * kXCopies + kWCopies;
};

template <int TS, int WS, int WT, int WN, bool GROUPED, bool GLU>
__global__ __launch_bounds__(64 * WT * WN) void fp8_tile_kernel(Fp8TileArgs A) {
  using T = Fp8Tile<TS, WS, WT, WN, GROUPED, GLU>;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int wt = wave % WT, wn = wave / WT;
  const int d = A.d, nb = A.nb, nout = GLU ? A.n / 2 : A.n;
  Fp8Place P;
  if (!fp8_place<T::kT, T::kOut, GROUPED, GLU>(A, P)) return;
  const int n0 = P.n0;

  // ---- copies: row 8·i + lane / 8 of a copy, LDS chunk lane % 8 holding the
  // global chunk (lane % 8) ^ (row % 8)
  const int crow = lane >> 3, cchunk = (lane & 7) ^ crow;
  uint32_t woff[T::kWCopies];
  // weight rows: a wave's WS blocks are consecutive LDS rows; with the
  // activation their upper half comes from the up rows (8·WS rows are whole
  // copies, so a copy reads one of the two halves)
  const int live = min(T::kOut, nout - n0);
  const __amdgpu_buffer_rsrc_t wr0 = make_rsrc(P.w + int64_t(n0) * d, uint32_t(live) * uint32_t(d));
  const __amdgpu_buffer_rsrc_t wr1 =
      GLU ? make_rsrc(P.w + int64_t(nout + n0) * d, uint32_t(live) * uint32_t(d)) : wr0;
#pragma unroll
  for (int i = 0; i < T::kWCopies; ++i) {
    int row = 8 * (wave * T::kWCopies + i) + crow;
    if constexpr (GLU) row = row / (16 * WS) * (8 * WS) + row % (8 * WS);   // output column
    woff[i] = row < live ? uint32_t(row) * uint32_t(d) : kOOB8;
  }
  const uint32_t base = lds_addr(lds);
  // a block past the last is all zeros and reads nothing: the counts stay the same
  auto at_block = [&](int b) {
    const uint32_t k = uint32_t(kFp8Block * b + 16 * cchunk);
    return k < uint32_t(d) ? k : kOOB8;
  };
  auto copy_w = [&](int b) {
    const uint32_t at = base + uint32_t(b & 1) * T::kStage + 128u * T::kT, ko = at_block(b);
#pragma unroll
    for (int i = 0; i < T::kWCopies; ++i)
      copy16_to_lds(GLU && ((wave * T::kWCopies + i) / WS & 1) ? wr1 : wr0, (woff[i] + ko) | ((woff[i] | ko) & kOOB8),
                    at + 1024u * uint32_t(wave * T::kWCopies + i));
  };
  copy_w(0);                                            // on its way while the rows are looked up

  uint32_t xoff[2][T::kXCopies], soff = kOOB8;
  const Fp8Source<GROUPED> src(A, P);
  // first row of a wave's i-th copy of half h of the activations
  auto x_row = [&](int h, int i) { return T::kT / 2 * h + 8 * (wave * T::kXCopies + i); };
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < T::kXCopies; ++i) {
      const int row = src(A, P, x_row(h, i) + crow);
      xoff[h][i] = row >= 0 ? uint32_t(row) * uint32_t(d) : kOOB8;
    }
  if (wave < T::kT / 64) {                              // scales of 64 rows a wave
    const int row = src(A, P, 64 * wave + lane);
    soff = row >= 0 ? uint32_t(row) * uint32_t(nb) * 4u : kOOB8;
    if constexpr (GROUPED)
      *reinterpret_cast<uint64_t*>(lds + T::kBad + 8 * wave) = __ballot(row < 0);
  }
  auto copy_x = [&](int b, int h) {
    const uint32_t at = base + uint32_t(b & 1) * T::kStage, ko = at_block(b);
#pragma unroll
    for (int i = 0; i < T::kXCopies; ++i)
      copy16_to_lds(src.x, (xoff[h][i] + ko) | ((xoff[h][i] | ko) & kOOB8), at + 128u * uint32_t(x_row(h, i)));
  };
  // scales of four steps at a time, 64 rows a wave (rows lie far apart: a copy
  // costs a cache line for each row, whatever it takes of it)
  auto copy_scales = [&](int b) {
    if ((b & 3) == 0 && wave < T::kT / 64)
      copy16_to_lds(src.s, fp8_scales_at(soff, b),
                    base + 2u * T::kStage + uint32_t(b >> 2 & 1) * T::kScales + 1024u * uint32_t(wave));
  };

  // ---- operands
  const float* ws0 = P.ws + int64_t(fp8_scale_row(n0 + (GLU ? 8 : 16) * WS * wn, nout)) * nb;
  const float* ws1 = P.ws + int64_t(P.sb + fp8_scale_row(n0 + 8 * WS * wn, nout)) * nb;
  const int o0 = 16 * (g ^ (col & 7));
  f32x4_t acc[TS][WS];
#pragma unroll
  for (int i = 0; i < TS; ++i)
#pragma unroll
    for (int j = 0; j < WS; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  constexpr int H = TS / 2;                             // activation blocks of a half step
  i32x8_t a[WS], bx[H];
  float sx[H];
  const unsigned char* st = lds;
  const float* sc = nullptr;
  auto operand = [&](const unsigned char* p) {
    return join(*reinterpret_cast<const u32x4_t*>(p + o0), *reinterpret_cast<const u32x4_t*>(p + (o0 ^ 64)));
  };
  auto read_w = [&]() {
#pragma unroll
    for (int j = 0; j < WS; ++j) a[j] = operand(st + 128 * (T::kT + 16 * WS * wn + col) + 2048 * j);
  };
  auto read_x = [&](auto half, auto blocks) {
    constexpr int h = decltype(half)::value;
#pragma unroll
    for (int i = 0; i < decltype(blocks)::value; ++i) {
      bx[i] = operand(st + 128 * (16 * wt + col) + 2048 * WT * (H * h + i));
      sx[i] = sc[64 * WT * (H * h + i)];
    }
  };
  // block sums and their multiply-adds, kAhead matrix instructions apart: the
  // order is fixed, since the scheduler would start all the block sums first and
  // keep them in registers that the accumulators need
  auto multiply = [&](auto half, auto blocks, auto exact, float w0, float w1) {
    constexpr int h = decltype(half)::value, kAhead = 4, N = decltype(blocks)::value * WS;
    constexpr bool kExact = decltype(exact)::value;
    f32x4_t p[kAhead + 1];
#pragma unroll
    for (int m = 0; m < (N ? N + kAhead : 0); ++m) {
      if (m < N)
        p[m % (kAhead + 1)] = kExact ? mfma_e4m3_exact(a[m % WS], bx[m / WS]) : mfma_e4m3(a[m % WS], bx[m / WS]);
      if (m >= kAhead) {
        const int u = m - kAhead, i = u / WS, j = u % WS;
        const float s = sx[i] * (GLU && j >= WS / 2 ? w1 : w0);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[H * h + i][j][e] = __builtin_fmaf(p[u % (kAhead + 1)][e], s, acc[H * h + i][j][e]);
        asm volatile("" : "+v"(acc[H * h + i][j]));      // and not later
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const bool behind = wave >= T::kWaves / 2;            // the second group: one phase later

  copy_scales(0);
  copy_x(0, 0);
  copy_x(0, 1);
  copy_w(1);
  copy_x(1, 0);
  wait_copies<T::kAfter>();
  phase_end();
  if (behind) phase_end();
  // The steps, with `first` and `second` live activation blocks of a half.
  auto steps = [&](auto first, auto second, auto exact) {
    float w0 = scalar_load(ws0, 0), w1 = GLU ? scalar_load(ws1, 0) : 0.f;
    for (int b = 0; b < nb; ++b) {
      st = lds + (b & 1) * T::kStage;
      sc = reinterpret_cast<const float*>(lds + 2 * T::kStage + (b >> 2 & 1) * T::kScales) + 4 * (16 * wt + col) + (b & 3);
      const int next = min(b + 1, nb - 1);
      const float w0n = scalar_load(ws0, next), w1n = GLU ? scalar_load(ws1, next) : 0.f;
      __builtin_amdgcn_s_setprio(1);                      // the reader's few instructions first
      read_w();
      read_x(std::integral_constant<int, 0>{}, first);
      copy_x(b + 1, 1);                                   // both groups have read that half of step b - 1
      __builtin_amdgcn_s_setprio(0);
      wait_reads();
      // second half of step b (a scale copy of this wave may be among the later ones)
      if (b % 4 == 3 && wave < T::kT / 64) wait_copies<T::kAfter + 1>();
      else wait_copies<T::kAfter>();
      phase_end();
      multiply(std::integral_constant<int, 0>{}, first, exact, w0, w1);
      phase_end();
      __builtin_amdgcn_s_setprio(1);
      read_x(std::integral_constant<int, 1>{}, second);
      copy_scales(b + 2);
      copy_w(b + 2);                                      // both groups have read these of step b
      copy_x(b + 2, 0);
      __builtin_amdgcn_s_setprio(0);
      wait_reads();
      // weights and first half of step b + 1
      if (b % 4 == 2 && wave < T::kT / 64) wait_copies<T::kAfter + 1>();
      else wait_copies<T::kAfter>();
      phase_end();
      multiply(std::integral_constant<int, 1>{}, second, exact, w0, w1);
      phase_end();
      w0 = w0n;
      w1 = w1n;
    }
  };
  // A tile with few live rows leaves out the block sums of dead ones, a quarter of
  // the tile at a time: the waves' blocks alternate, so all waves have less to do.
  // Segments of up to 16 rows have block sums in fp32, the last rows of a longer one
  // have them as its other rows do: a row's result depends on the rows that its
  // segment has, not on its place among them.
  const int rows = int(P.m_end - P.m0);
  using None = std::integral_constant<int, 0>;
  using Part = std::integral_constant<int, H / 2>;
  using Whole = std::integral_constant<int, H>;
  constexpr bool kShort = GROUPED && T::kT == 64;       // a quarter is 16 rows
  const std::false_type fast{};
  if (rows > T::kT / 4 * 3) steps(Whole{}, Whole{}, fast);
  else if (rows > T::kT / 2) steps(Whole{}, Part{}, fast);
  else if (rows > T::kT / 4) steps(Whole{}, None{}, fast);
  else if (kShort && P.starts) steps(Part{}, None{}, std::integral_constant<bool, kShort>{});
  else steps(Part{}, None{}, fast);
  if (!behind) phase_end();                             // the groups' barrier counts match
  wait_copies<0>();
  phase_end();

  // ---- epilogue: the output tile through LDS, so that a store has whole lines.
  // Lane (col, g) holds columns 4g .. 4g + 3 of activation row col; a row's 16-byte
  // chunks lie at chunk ^ (row mod 16 or 8).  (Straight from the registers, 32 bytes
  // of a row at a time, the stores of a 256 x 256 tile took 6.5 to 7.5 us.)
  constexpr int WO = GLU ? WS / 2 : WS, kChunks = T::kOut / 8, kMask = kChunks < 16 ? kChunks - 1 : 15;
#pragma unroll
  for (int i = 0; i < TS; ++i) {
    const int row = 16 * (WT * i + wt) + col;
    bool bad = false;
    if constexpr (GROUPED) bad = reinterpret_cast<const uint32_t*>(lds + T::kBad)[row >> 5] >> (row & 31) & 1;
#pragma unroll
    for (int j = 0; j < WO; ++j) {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = GLU ? quick_silu(acc[i][j][e]) * acc[i][WS - WO + j][e] : acc[i][j][e];
      const int chunk = (2 * (WO * wn + j) + (g >> 1)) ^ (col & kMask);
      *reinterpret_cast<u32x2_t*>(lds + 2 * T::kOut * row + 16 * chunk + 8 * (g & 1)) =
          bad ? u32x2_t{0x7FC07FC0u, 0x7FC07FC0u} : u32x2_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])};
    }
  }
  wait_reads();
  phase_end();
#pragma unroll 4
  for (int q = threadIdx.x; q < rows * kChunks; q += 64 * T::kWaves) {
    const int row = q / kChunks, chunk = q % kChunks;
    const u32x4_t v = *reinterpret_cast<const u32x4_t*>(lds + 2 * T::kOut * row + 16 * (chunk ^ (row & kMask)));
    store8(A.y + (P.m0 + row) * A.ldy, n0 + 8 * chunk, nout, v);
  }
}

template <int TS, int WS, int WT, int WN, bool GROUPED, bool GLU>
int go(const Fp8GemmArgs& a, hipStream_t s) {
  using T = Fp8Tile<TS, WS, WT, WN, GROUPED, GLU>;
  auto kernel = fp8_tile_kernel<TS, WS, WT, WN, GROUPED, GLU>;
  const size_t bytes = T::kLds;
  const int nout = GLU ? a.n / 2 : a.n;
  const int64_t tiles_n = (int64_t(nout) + T::kOut - 1) / T::kOut;
  // grouped: no more row tiles than whole tiles of rows and one part tile a segment
  const int64_t tiles_t = GROUPED ? int64_t(a.m_total) / T::kT + std::min(a.n_seg, a.m_total)
                                  : (a.t + T::kT - 1) / T::kT;
  if (tiles_t == 0) return 0;
  if (tiles_n * tiles_t * 64 * T::kWaves >= (int64_t(1) << 32)) return int(hipErrorInvalidValue);   // the grid's limit
  const Fp8TileArgs k{a.w, a.ws, a.n, a.d, fp8_blocks(a.d), a.x, a.xs, a.t, a.y, a.ldy, int(tiles_n), a.row_index,
                      a.seg_expert, a.seg_offsets, a.n_experts, a.n_seg, a.m_total, int(a.t_x)};
  launch_kernel_lds(kernel, dim3(unsigned(tiles_n * tiles_t)), dim3(64 * T::kWaves), bytes, s, k);
  return int(hipGetLastError());
}

template <bool GROUPED, bool GLU>
int go(bool large, const Fp8GemmArgs& a, hipStream_t s) {
  return large ? go<8, 4, 2, 4, GROUPED, GLU>(a, s) : go<4, 2, 1, 4, GROUPED, GLU>(a, s);
}

}  // namespace

int launch_fp8_tile(const Fp8GemmArgs& a, bool large, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.n_seg == 0) return go<false, false>(large, a, s);
  return a.glu ? go<true, true>(large, a, s) : go<true, false>(large, a, s);
}

int launch_fp8_product(const Fp8GemmArgs& a, void* stream) {
  const Fp8Kernel k = fp8_kernel(a);
  return k == Fp8Kernel::kRows ? launch_fp8_rows(a, stream) : launch_fp8_tile(a, k == Fp8Kernel::kTile256, stream);
}

}  // namespace qmm
