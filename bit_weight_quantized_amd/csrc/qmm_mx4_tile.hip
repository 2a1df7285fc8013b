// Microscaled 4-bit product for many activation rows: tiles of activations and weights in
// LDS, scaled fp4 matrix instructions.
//
//   y[t,n] = Σ_b 2^(Ex[t,b] + Ew[n,b] - 254) · Σ_{k in b} x[t,k]·w[n,k]
//
// A K step is 128 codes, 64 bytes of every row: one v_mfma_scale_f32_16x16x128_f8f6f4 for 16
// weight rows (A operand) and 16 activation rows (B operand), which applies the exponents of
// their blocks of 32 itself.  Lane (c, g) takes row c's 16-byte piece g, a whole block, and
// its exponent.
//
// Both tiles go global -> LDS without passing registers, into a ring of four stages.  A row's
// four pieces are stored at piece ^ (row / 2 mod 4), done on the global side of the copy: a
// 16-byte LDS read serves 16 lanes a cycle, lanes 0..3, 12..15 and 20..27 first, and these
// then lie in different banks (4.05 cycles a read measured, 8.05 with eight pieces at
// piece ^ (row mod 8)).  Exponents are copied a slab (four steps, 16 bytes a row) at a time and
// read once a slab, a word for a lane's four steps, put together from the row's four words:
// a read of one byte takes LDS as long as one of 16.
//
// Two waves on every SIMD, with 128 x 64 of the 256 x 256 tile each: one's products cover what
// the other waits for.  Nothing is read where it is needed: behind the products of an
// activation block go the reads of the block half a step further on, in the second half of a
// step those of the next step's weights, and the copies, spread over all blocks, since a copy
// holds its wave while the memory pipeline is busy.  One barrier a step, in its middle: after
// it the next step's stage has landed (counted by vmcnt; every wave issues the same number a
// step) and no wave reads the previous one's, whose place the copies then take: they have
// nearly two steps to land.
//
// Steps come in slabs; those past d are zeros.  Tiles of up to half of the rows leave out the
// products of the other half.  (A choice for each block costs 10%, one in quarters registers.)
//
// Bound by power for many tiles: 8192 x 8192 x 8192 260 us (4.23 PFLOP/s; the same without its
// copies 204, products alone run at 6 to 7), 2048 x 13824 x 5120 81 us (3.58; 432 tiles in two
// rounds of 256 CUs); by a tile's start and end (7 us) for short reductions, 4096 x 4096 x 4096
// 39 us; a step of a tile by itself takes 0.62 us, 0.43 of it products.
// Two groups of waves in opposite phases with a barrier between them (as the e4m3 tiles have
// it): 4 to 6% slower with all CUs at work, 25% with a quarter of them.
#include <hip/hip_runtime.h>

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"
#include "qmm_fp8_tile.h"
#include "qmm_launch.h"
#include "qmm_lds_copy.h"
#include "qmm_mx4.h"
#include "qmm_mx4_device.h"

#include <algorithm>
#include <type_traits>

namespace qmm {
namespace {

struct Mx4TileArgs {
  Fp8TileArgs place;       // sizes and tables, for the tile's place
  const uint8_t* codes;    // of the first matrix
  const uint8_t* meta;
  uint32_t codes_bytes, meta_bytes;
  int64_t expert_stride;
  const uint8_t* x;
  const uint8_t* xs;
  int t_x;
  uint16_t* y;
  int64_t ldy;
  bool fit;
  uint8_t* hq;
  uint8_t* hs;
};

// TS (WS) blocks of 16 activation (weight) rows a wave, WT × WN waves.
// GLU: the lower half of a wave's weight blocks are gate rows, the upper half
// the up rows of the same outputs.
template <int TS, int WS, int WT, int WN, bool GROUPED, bool GLU>
struct Mx4Tile {
  static constexpr int RING = 4;                       // stages
  static constexpr int kWaves = WT * WN;
  static constexpr int kT = 16 * TS * WT;              // activation rows
  static constexpr int kN = 16 * WS * WN;              // weight rows
  static constexpr int kOut = GLU ? kN / 2 : kN;       // output columns
  static constexpr int kStage = (kT + kN) * 64;        // both tiles of a step
  static constexpr int kXCopies = kT / 16 / kWaves, kWCopies = kN / 16 / kWaves, kOps = kXCopies + kWCopies;
  static constexpr int kSc = ((kT + kN) / 64 + kWaves - 1) / kWaves;   // copies of exponents of a wave and slab
  static constexpr int kScales = kSc * kWaves * 1024;  // exponents of a slab
  static constexpr int kBad = RING * kStage + 2 * kScales;   // a bit for every row without a source
  static constexpr int kLds = kBad + (kT + 31) / 32 * 4;
  static_assert(kT * kOut * 2 <= RING * kStage, "the output tile takes the place of the operands'");
  static_assert(kT / 16 % kWaves == 0 && kN / 16 % kWaves == 0 && kT % 64 == 0, "whole copies per wave");
  static_assert(TS % 4 == 0 && kOps <= TS, "reads and copies behind the products");
  static_assert(kLds <= 160 * 1024, "LDS");
};

template <int TS, int WS, int WT, int WN, bool GROUPED, bool GLU>
__global__ __launch_bounds__(64 * WT * WN) void mx4_tile_kernel(Mx4TileArgs A) {
  using T = Mx4Tile<TS, WS, WT, WN, GROUPED, GLU>;
  constexpr int RING = T::RING;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int wt = wave % WT, wn = wave / WT;
  const int n = A.place.n, d = A.place.d, nout = GLU ? n / 2 : n, steps = (d + 127) / 128;
  Fp8Place P;
  if (!fp8_place<T::kT, T::kOut, GROUPED, GLU>(A.place, P)) return;
  const int n0 = P.n0;
  const Slabs L{n, d, QMM_MXFP4_G32};
  const int64_t expert = GROUPED && !P.bad_expert ? int64_t(P.expert) * A.expert_stride : 0;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(A.codes + expert, A.codes_bytes);
  const __amdgpu_buffer_rsrc_t mr = make_rsrc(A.meta + expert, A.meta_bytes);

  // ---- copies: row lane / 4 of a copy's sixteen, LDS piece lane % 4 holding the global
  // piece (lane % 4) ^ (row / 2 % 4)
  const int crow = lane >> 2, cpiece = (lane & 3) ^ (crow >> 1 & 3);
  const int live = min(T::kOut, nout - n0);
  // packed row of a tile's weight row; -1 past the matrix
  auto w_row = [&](int row) {
    int up = 0;
    if constexpr (GLU) {
      up = (row / (8 * WS) & 1) ? nout : 0;
      row = row / (16 * WS) * (8 * WS) + row % (8 * WS);   // output column
    }
    return row < live ? up + n0 + row : -1;
  };
  // Offsets of a lane's pieces in slab 0; later slabs and steps are a scalar offset further.
  // The last slab's rows may be narrower: theirs are worked out when it is reached.
  const int last = L.count() - 1, width = L.width(0) / 2, width_last = L.width(last) / 2;
  const uint32_t slab_bytes = uint32_t(n) * (kSlabCodes / 2);   // of a slab that another follows
  auto w_offset = [&](int i, int bytes) {
    const int row = w_row(16 * (wave * T::kWCopies + i) + crow);
    return row >= 0 ? uint32_t(row) * uint32_t(bytes) + 16u * uint32_t(cpiece) : kOOB8;
  };
  uint32_t woff[T::kWCopies];
#pragma unroll
  for (int i = 0; i < T::kWCopies; ++i) woff[i] = w_offset(i, last == 0 ? width_last : width);
  const uint32_t base = lds_addr(lds);

  const uint32_t xstride = uint32_t(d) / 2, sstride = uint32_t(mx_scale_bytes(d));
  const uint32_t held = GROUPED ? uint32_t(A.t_x) : uint32_t(P.m_end - P.m0);
  const int64_t first = GROUPED ? 0 : P.m0;
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(A.x + first * xstride, held * xstride);
  const __amdgpu_buffer_rsrc_t sr = make_rsrc(A.xs + first * sstride, held * sstride);
  // row of the tile -> row of the buffers; -1 past the tile, or (grouped) for a bad row or expert
  auto source = [&](int row) {
    if (P.m0 + row >= P.m_end) return -1;
    if constexpr (!GROUPED) return row;
    const int src = A.place.row_index ? A.place.row_index[P.m0 + row] : int(P.m0 + row);
    return P.bad_expert || src < 0 || src >= A.t_x ? -1 : src;
  };
  uint32_t xoff[T::kXCopies];
#pragma unroll
  for (int i = 0; i < T::kXCopies; ++i) {
    const int row = source(16 * (wave * T::kXCopies + i) + crow);
    xoff[i] = row >= 0 ? uint32_t(row) * xstride + 16u * uint32_t(cpiece) : kOOB8;
  }
  // exponents of 64 rows a copy: the activations' first, then the weights'; the last may be of none
  auto m_offset = [&](int part, int row_bytes) {
    const int row = 64 * part < T::kT + T::kN ? w_row(64 * part - T::kT + lane) : -1;
    return row >= 0 ? uint32_t(row >> 2) * uint32_t(L.meta_quad()) + uint32_t(row & 3) * uint32_t(row_bytes) : kOOB8;
  };
  const int meta_last = L.meta_row(last), meta_row = L.meta_row(0);
  uint32_t soff[T::kSc];
#pragma unroll
  for (int i = 0; i < T::kSc; ++i) {
    const int part = wave + T::kWaves * i;
    if (part < T::kT / 64) {
      const int row = source(64 * part + lane);
      soff[i] = row >= 0 ? uint32_t(row) * sstride : kOOB8;
      if constexpr (GROUPED) *reinterpret_cast<uint64_t*>(lds + T::kBad + 8 * part) = __ballot(row < 0);
    } else {
      soff[i] = m_offset(part, last == 0 ? meta_last : meta_row);
    }
  }
  // copy `i` of step h: the weights', then the activations'
  auto past = [&](int h) { return 128 * h + kMxBlock * cpiece < d ? 0u : kOOB8; };
  auto copy = [&](int i, int h, uint32_t none) {
    const uint32_t at = base + uint32_t(h & (RING - 1)) * T::kStage;
    const bool in = h < steps;
    if (i < T::kWCopies)
      copy16_to_lds_from(wr, woff[i < T::kWCopies ? i : 0] | none,
                         in ? uint32_t(h >> 2) * slab_bytes + 64u * uint32_t(h & 3) : 0u,
                         at + 64u * T::kT + 1024u * uint32_t(wave * T::kWCopies + i));
    else
      copy16_to_lds_from(xr, xoff[i < T::kWCopies ? 0 : i - T::kWCopies] | none, in ? 64u * uint32_t(h) : 0u,
                         at + 1024u * uint32_t(wave * T::kXCopies + i - T::kWCopies));
  };
  // before the first copy of a narrow last slab
  auto enter = [&](int s) {
    if (s != last || last == 0 || width_last == width) return;
#pragma unroll
    for (int i = 0; i < T::kWCopies; ++i) woff[i] = w_offset(i, width_last);
  };
  auto copy_scales = [&](int s) {
    const bool in = s <= last;
    const uint32_t at = base + uint32_t(RING * T::kStage) + uint32_t(s & 1) * T::kScales, none = in ? 0u : kOOB8;
#pragma unroll
    for (int i = 0; i < T::kSc; ++i) {
      const int part = wave + T::kWaves * i;
      const bool x = part < T::kT / 64;
      if (in && s == last && last > 0 && meta_last != meta_row && !x) soff[i] = m_offset(part, meta_last);
      copy16_to_lds_from(x ? sr : mr, soff[i] | none, in ? uint32_t(s) * (x ? 16u : 64u) : 0u, at + 1024u * uint32_t(part));
    }
  };

  // ---- operands and sums: the weights' of two steps, the activations' of the next H blocks,
  // the exponents of a slab (byte q of a word for its step q) and of the next
  constexpr int H = TS / 2;
  const unsigned char* const lane_at = lds + 64 * col + 16 * (g ^ (col >> 1 & 3));
  const unsigned char* const x_at = lane_at + 1024 * wt;
  const unsigned char* const w_at = lane_at + 64 * T::kT + 1024 * WS * wn;
  const unsigned char* const scale_at = lds + RING * T::kStage + 16 * col;
  // bytes g of two words, of the later one in the upper half
  const uint32_t pick = 0x0C0C0400u + 0x0101u * uint32_t(g);
  u32x4_t a[2][WS], bx[H];
  uint32_t sa[WS], na[WS], sx[TS];
  f32x4_t acc[TS][WS];
#pragma unroll
  for (int i = 0; i < TS; ++i)
#pragma unroll
    for (int j = 0; j < WS; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  auto read_w = [&](auto to, int j, int q) {
    a[decltype(to)::value][j] = *reinterpret_cast<const u32x4_t*>(w_at + (q & 3) * T::kStage + 1024 * j);
  };
  auto read_x = [&](int i, int q) {
    bx[i % H] = *reinterpret_cast<const u32x4_t*>(x_at + (q & 3) * T::kStage + 1024 * WT * i);
  };
  // exponents of block r of slab s, the weights', then the activations', as LDS has them and
  // as the lane needs them: those of its pieces of the four steps
  auto read_scale = [&](int r, int s) {
    const int row = r < WS ? T::kT + 16 * (WS * wn + r) : 16 * (WT * (r - WS) + wt);
    return *reinterpret_cast<const u32x4_t*>(scale_at + (s & 1) * T::kScales + 16 * row);
  };
  auto mine = [&](const u32x4_t v) {
    return __builtin_amdgcn_perm(v[1], v[0], pick) | __builtin_amdgcn_perm(v[3], v[2], pick) << 16;
  };
  // the copy behind block `slot` of the TS that follow a barrier
  auto copies_at = [&](int slot, int h) {
    const uint32_t none = past(h);
#pragma unroll
    for (int k = 0; k < T::kOps; ++k)
      if (k * TS / T::kOps == slot) copy(k, h, none);
  };

  copy_scales(0);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < T::kOps; ++i) copy(i, h, past(h));
  wait_copies<T::kOps>();
#pragma unroll
  for (int i = 0; i < H; ++i) copies_at(i, 2);
  phase_end();
#pragma unroll
  for (int j = 0; j < WS; ++j) sa[j] = mine(read_scale(j, 0));
#pragma unroll
  for (int i = 0; i < TS; ++i) sx[i] = mine(read_scale(WS + i, 0));
#pragma unroll
  for (int j = 0; j < WS; ++j) read_w(std::integral_constant<int, 0>{}, j, 0);
#pragma unroll
  for (int i = 0; i < H; ++i) read_x(i, 0);

  const int rows = int(P.m_end - P.m0);
  const int live_blocks = min(TS, (rows + 16 * WT - 1) / (16 * WT));   // activation blocks of a wave that have rows
  // Step q of slab s.  ALL: every activation block has rows; else those without are left out.
  auto step = [&](auto of, auto count, int s) {
    constexpr int q = decltype(of)::value, cur = q & 1;
    std::integral_constant<int, 1 - cur> next;
    const int h = 4 * s + q;
    u32x4_t raw;
#pragma unroll
    for (int i = 0; i < TS; ++i) {
      if (i == H) {
        // step h + 1 has landed; no wave reads step h - 1 any more
        wait_copies<T::kOps + (q == 1 ? T::kSc : 0)>();
        phase_end();
        __builtin_amdgcn_sched_barrier(0);
        if (q == 0) copy_scales(s + 1);
        if (q == 1) enter(s + 1);
      }
      if (i < decltype(count)::value) {
#pragma unroll
        for (int j = 0; j < WS; ++j) acc[i][j] = mfma_fp4<q, q>(a[cur][j], bx[i % H], acc[i][j], sa[j], sx[i]);
      }
      __builtin_amdgcn_sched_barrier(0);
      if (i < H) read_x(i + H, q);
      else read_x(i - H, q + 1);
#pragma unroll
      for (int j = 0; j < WS; ++j)
        if (i >= H && j * (H - 1) / WS == i - H) read_w(next, j, q + 1);
      // The exponents of slab s + 1 have landed before the second half of step 2: the weights' are
      // read then, the activations' behind the last products with their predecessors.
      if (q == 2 && i > H && i - H <= WS) na[i - H > 0 ? i - H - 1 : 0] = mine(raw);
      if (q == 2 && i >= H && i - H < WS) raw = read_scale(i - H, s + 1);
      if (q == 3 && i > 0) sx[i > 0 ? i - 1 : 0] = mine(raw);
      if (q == 3) raw = read_scale(WS + i, s + 1);
      copies_at(i < H ? i + H : i - H, i < H ? h + 2 : h + 3);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (q == 2 && WS == TS - H) na[WS - 1] = mine(raw);
    if (q == 3) {
      sx[TS - 1] = mine(raw);
#pragma unroll
      for (int j = 0; j < WS; ++j) sa[j] = na[j];
    }
#pragma unroll
    for (int i = 0; i < TS; ++i)
#pragma unroll
      for (int j = 0; j < WS; ++j) asm volatile("" : "+v"(acc[i][j]));
  };
  auto run = [&](auto count) {
    for (int s = 0; s <= last; ++s) {
      step(std::integral_constant<int, 0>{}, count, s);
      step(std::integral_constant<int, 1>{}, count, s);
      step(std::integral_constant<int, 2>{}, count, s);
      step(std::integral_constant<int, 3>{}, count, s);
    }
  };
  if (live_blocks > TS / 2) run(std::integral_constant<int, TS>{});
  else run(std::integral_constant<int, TS / 2>{});
  wait_copies<0>();
  phase_end();

  // ---- epilogue: the output tile through LDS, so that a store has whole lines.
  // Lane (col, g) holds columns 4g .. 4g + 3 of activation row col.
  constexpr int WO = GLU ? WS / 2 : WS;
  auto is_bad = [&](int row) {
    if constexpr (!GROUPED) return false;
    return bool(reinterpret_cast<const uint32_t*>(lds + T::kBad)[row >> 5] >> (row & 31) & 1);
  };
  if constexpr (GLU) {
#pragma unroll
    for (int i = 0; i < TS; ++i)
#pragma unroll
      for (int j = 0; j < WO; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = quick_silu(acc[i][j][e]) * acc[i][WS - WO + j][e];
    if (A.hq) {
      // A block's 32 columns are two neighbouring 16s: their largest values meet in LDS, behind
      // the tile of codes, in which 16-byte pieces are blocks.
      constexpr int kPieces = T::kOut / 32, kRowBytes = T::kOut / 2;
      uint32_t* most = reinterpret_cast<uint32_t*>(lds + T::kT * kRowBytes);   // [row][column / 16]
#pragma unroll
      for (int i = 0; i < TS; ++i) {
        const int row = 16 * (WT * i + wt) + col;
        const bool bad = is_bad(row);
#pragma unroll
        for (int j = 0; j < WO; ++j) {
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) m = umax(m, __float_as_uint(acc[i][j][e]) & 0x7FFFFFFFu);
          m = umax(m, uint32_t(__shfl_xor(int(m), 16)));
          m = umax(m, uint32_t(__shfl_xor(int(m), 32)));
          if (g == 0) most[2 * kPieces * row + WO * wn + j] = bad ? 0x7FC00000u : m;
        }
      }
      wait_reads();
      phase_end();
#pragma unroll
      for (int i = 0; i < TS; ++i) {
        const int row = 16 * (WT * i + wt) + col;
#pragma unroll
        for (int j = 0; j < WO; ++j) {
          const int at = WO * wn + j;
          const u32x2_t pair = *reinterpret_cast<const u32x2_t*>(most + 2 * kPieces * row + (at & ~1));
          const uint32_t ex = mx_exponent(umax(pair[0], pair[1]), A.fit);
          uint32_t q = 0;
          q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, acc[i][j][0], acc[i][j][1], mx_scale(ex), 0);
          q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, acc[i][j][2], acc[i][j][3], mx_scale(ex), 1);
          *reinterpret_cast<uint16_t*>(lds + kRowBytes * row + 8 * at + 2 * g) = ex != 255u ? uint16_t(q) : uint16_t(0);
        }
      }
      wait_reads();
      phase_end();
      const int64_t scale_bytes = mx_scale_bytes(nout);
      for (int q = threadIdx.x; q < rows * kPieces; q += 64 * T::kWaves) {
        const int row = q / kPieces, piece = q % kPieces, c = n0 + 32 * piece;
        if (c >= nout) continue;
        const u32x2_t pair = *reinterpret_cast<const u32x2_t*>(most + 2 * kPieces * row + 2 * piece);
        uint8_t* hs = A.hs + (P.m0 + row) * scale_bytes;
        *reinterpret_cast<u32x4_t*>(A.hq + (P.m0 + row) * (nout / 2) + c / 2) =
            *reinterpret_cast<const u32x4_t*>(lds + kRowBytes * row + 16 * piece);
        hs[c / 32] = uint8_t(mx_exponent(umax(pair[0], pair[1]), A.fit));
        if (c + 32 == nout)                             // zeros past the row's blocks
          for (int b = nout / 32; b < scale_bytes; ++b) hs[b] = 0;
      }
      return;
    }
  }
  // a row's 16-byte pieces lie at piece ^ (row mod 16 or 8)
  constexpr int kChunks = T::kOut / 8, kMask = kChunks < 16 ? kChunks - 1 : 15;
#pragma unroll
  for (int i = 0; i < TS; ++i) {
    const int row = 16 * (WT * i + wt) + col;
    const bool bad = is_bad(row);
#pragma unroll
    for (int j = 0; j < WO; ++j) {
      const f32x4_t f = acc[i][j];
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
int go(const Mx4GemmArgs& a, hipStream_t s) {
  using T = Mx4Tile<TS, WS, WT, WN, GROUPED, GLU>;
  Layout l;
  if (!layout_of(QMM_MXFP4_G32, a.n, a.d, &l)) return int(hipErrorInvalidValue);
  static_assert(T::kWaves * 64 == (T::kT == 256 ? 512 : 256) && T::kOut == (T::kT == 256 ? 256 : 128) / (GLU ? 2 : 1), "mx4_tiles");
  const Mx4Tiles tiles = mx4_tiles(a, T::kT == 256);
  if (tiles.t == 0) return 0;
  if (!tiles.fit) return int(hipErrorInvalidValue);
  Mx4TileArgs k{};
  k.place.n = a.n;
  k.place.d = a.d;
  k.place.t = a.t;
  k.place.tiles_n = int(tiles.n);
  k.place.row_index = a.row_index;
  k.place.seg_expert = a.seg_expert;
  k.place.seg_offsets = a.seg_offsets;
  k.place.n_experts = a.n_experts;
  k.place.n_seg = a.n_seg;
  k.place.m_total = a.m_total;
  k.codes = a.packed + l.codes_offset;
  k.meta = a.packed + l.meta_offset;
  k.codes_bytes = uint32_t(int64_t(a.n) * (a.d / 2));
  k.meta_bytes = uint32_t(l.meta_bytes);
  k.expert_stride = a.expert_stride;
  k.x = a.x;
  k.xs = a.xs;
  k.t_x = int(a.t_x);
  k.y = a.y;
  k.ldy = a.ldy;
  k.fit = a.fit;
  k.hq = a.hq;
  k.hs = a.hs;
  launch_kernel_lds((mx4_tile_kernel<TS, WS, WT, WN, GROUPED, GLU>), dim3(unsigned(tiles.n * tiles.t)),
                    dim3(64 * T::kWaves), size_t(T::kLds), s, k);
  return int(hipGetLastError());
}

template <bool GROUPED, bool GLU>
int go(bool large, const Mx4GemmArgs& a, hipStream_t s) {
  return large ? go<8, 4, 2, 4, GROUPED, GLU>(a, s) : go<4, 2, 1, 4, GROUPED, GLU>(a, s);
}

}  // namespace

int launch_mx4_tile(const Mx4GemmArgs& a, bool large, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (a.n_seg == 0) return go<false, false>(large, a, s);
  return a.glu ? go<true, true>(large, a, s) : go<true, false>(large, a, s);
}

int launch_mx4_product(const Mx4GemmArgs& a, void* stream) {
  const MxKernel k = mx4_kernel(a);
  return k == MxKernel::kRows ? launch_mx4_rows(a, stream) : launch_mx4_tile(a, k == MxKernel::kTile256, stream);
}

}  // namespace qmm
