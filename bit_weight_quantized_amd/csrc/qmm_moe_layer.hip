// A mixture-of-experts layer for up to 16 tokens in two launches, MXFP4 weights and bf16
// activations:
//
//   1  logits -> k experts a token and their weights;  h[t,j] = silu(G_e x_t)·(U_e x_t)
//   2  out[t] = Σ_j weight[t,j]·D_e h[t,j] (+ shared[t])
//
// Bound by the chosen experts' bytes, read once each whatever the tokens.  Every workgroup
// (one a CU) makes the choice itself, a wave a token: a launch of its own would take as long
// as the layer's start.  The second kernel reads the choice that the first one's workgroup 0
// has written.  From the choice follow, by a bit for each token of an expert and one scan, the
// groups of rows that the waves work on.
//
// A wave goes through its pieces of work (first kernel: up to 8 gate rows and the 8 up rows of
// the same outputs, whose sums meet in registers; second: a share of the steps of a block of
// up to 16 columns over all experts) as one sequence of steps of 256 codes: weights, exponents
// and the group's activation rows of a step come through a private LDS ring (global -> LDS, no
// registers, no barriers), the copies a whole ring ahead, across the borders of pieces.  A
// copy takes a CU 25 to 30 clocks whatever its size, which counts where a wave has few steps,
// so a step has as few as possible: with groups of two rows four for 256 codes (steps of 128
// codes had six: 38.3 and 32.8 us at one token, 174 and 147 at 16, as below), and none past
// the work.  A lane's 16-byte piece of weights is a block of 32 codes, converted to bf16
// (exactly up to E8M0 252; values of 2^128 and more are infinite) for four
// v_mfma_f32_16x16x32_bf16 with 16 weight rows (A operand) and the group's rows (B operand).  The
// second kernel's waves' weighted sums meet in LDS in the waves' order: nothing depends on timing.
//
// h is kept in two bf16 parts: rounded to one, the output's error against 64 bits was up to 1.55
// times that of its own rounding, now 1.0 (second kernel 48 -> 54 us at 16 tokens, 11.7 -> 11.4
// at one).  In a workspace of half the size, which the call took first, two neighbours share an
// exponent and have 12 bits each; a wave takes a step's rows apart into the same two parts before it
// reads operands (one token, 8 of 256 experts: 31.6 us, 16 of 8 of 64: 153).  One bf16 part takes 29.8
// and 129 there, at 1.35 to 1.55 times the error.
//
// Measured, back to back, logits that favour no expert, the whole workspace (the two kernels by
// themselves), half of it, and the four calls that the layer joins: one token, 8 of 256 experts of
// 3584 x 2048: 30.2 us (18.8 and 11.2; 93.6 MB, 3.1 TB/s: 3 us choice and 1 tables, then 62 MB at 5
// TB/s; 3 us before the second one's first copy), 31.5, 61.2; 2 tokens, 2 of 8, 1024 x 512: 14.0, 14.3,
// 19.2; 4 tokens, 8 of 128, 2048 x 768: 30.2, 32.4, 37.9; 7 tokens, 4 of 60, 2080 x 1056: 32.2, 35.4,
// 36.7; 16 tokens, 8 of 64 (57 have a row), 3584 x 2048: 146 (93 and 54; 666 MB, 4.6 TB/s), 154, 143; 8
// of 256 (102 have one): 227 (5.2 TB/s), 240, 237.
#include <hip/hip_runtime.h>

#include "qmm_device.h"
#include "qmm_fp8_device.h"
#include "qmm_fp8_tile.h"
#include "qmm_launch.h"
#include "qmm_lds_copy.h"
#include "qmm_moe_layer.h"
#include "qmm_topk_wave.h"

#include <algorithm>

namespace qmm {
namespace {

constexpr int kLayerWaves = 8;
constexpr int kLayerRing = 3 * 6400;      // a wave's ring
constexpr int kLayerTokens = 8 * 1024;    // in the first wave's ring, before it is one: masks of the experts' tokens
static_assert(kLayerTokens + 4 * kRouteMaxExperts <= kLayerRing, "LDS");
constexpr int kRowKinds = 4;              // groups of up to 2, 4, 8 or 16 rows

struct LayerChoice {
  int32_t ids[kLayerMaxPairs];            // experts of the pairs (token, choice), -1: none
  float weights[kLayerMaxPairs];          // of the pairs
};
struct LayerTables {
  // "rows" are the pairs with an expert, by expert, then token
  float row_weight[kLayerMaxPairs];
  uint8_t token[kLayerMaxPairs];          // of the rows
  uint16_t tokens[kLayerMaxPairs];        // of a group, a bit each
  uint16_t expert[kLayerMaxPairs];        // of the groups
  uint16_t first[kLayerMaxPairs + 2];     // a group's first row
  uint32_t sums[2][kLayerWaves];
  int32_t groups, kind;                   // groups, of up to 2 << kind rows
};
constexpr int kLayerRed = kLayerWaves * kLayerRing;                    // sums of waves but the first
constexpr int kLayerTables = kLayerRed + (kLayerWaves - 1) * 1024;
constexpr int kLayerLds = kLayerTables + int(sizeof(LayerTables));
static_assert(kLayerRed + sizeof(LayerChoice) <= kLayerTables, "the choice lies where the sums will");
static_assert(kLayerLds <= 160 * 1024, "LDS");

// Inclusive sums of a wave's lanes.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15, 31
  return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
}

__device__ __forceinline__ void clear_tokens(uint32_t* tokens, int ne) {
  for (int e = threadIdx.x; e < ne; e += 64 * kLayerWaves) tokens[e] = 0u;
  __syncthreads();
}

// The tables from ids; every thread of the workgroup calls it.  An expert's rows are taken in
// groups of up to 2 << kind, each of which reads the expert's weights: the fewer rows a step
// of the ring holds, the fewer copies it takes and the more steps fit.  The smallest kind with
// at most 1.25 groups an expert: 16 tokens, 8 of 64 experts of 3584 x 2048, 155 us so (groups
// of 4) and 181 with up to 1.5 (groups of 2).  `tokens`, n_experts words, has
// which tokens an expert has, a bit each, and gets its first row in the upper half.  Thread i
// counts for experts 2i and 2i + 1; the counts of all kinds go through one scan, 10 bits each.
__device__ __forceinline__ void make_tables(LayerTables& T, const LayerChoice& C, uint32_t* tokens, int pairs, int k, int ne) {
  static_assert(kRouteMaxExperts <= 2 * 64 * kLayerWaves, "a thread has two experts");
  const int tid = threadIdx.x, wave = tid >> 6;
  const int id = tid < pairs ? C.ids[tid] : -1, tok = tid / k;
  uint32_t mask[2], a = 0, b = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    mask[i] = 2 * tid + i < ne ? tokens[2 * tid + i] : 0u;
    const uint32_t r = __builtin_popcount(mask[i]);
    a += r | (r + 1) / 2 << 10 | (r + 3) / 4 << 20;
    b += (r + 7) / 8 | (r + 15) / 16 << 10;
  }
  const uint32_t as = wave_scan(a), bs = wave_scan(b);
  if ((tid & 63) == 63) {
    T.sums[0][wave] = as;
    T.sums[1][wave] = bs;
  }
  __syncthreads();
  uint32_t at_a = as - a, at_b = bs - b, all_a = 0, all_b = 0;
#pragma unroll
  for (int w = 0; w < kLayerWaves; ++w) {
    const uint32_t sa = T.sums[0][w], sb = T.sums[1][w];
    at_a += w < wave ? sa : 0u;
    at_b += w < wave ? sb : 0u;
    all_a += sa;
    all_b += sb;
  }
  auto of = [](int kind, uint32_t u, uint32_t v) {
    return int((kind == 0 ? u >> 10 : kind == 1 ? u >> 20 : kind == 2 ? v : v >> 10) & 1023u);
  };
  const int most = of(kRowKinds - 1, all_a, all_b);   // chosen experts
  int kind = 0;
  while (kind < kRowKinds - 1 && 4 * of(kind, all_a, all_b) > 5 * most) ++kind;
  int at = of(kind, at_a, at_b), row = int(at_a & 1023u);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = __builtin_popcount(mask[i]);
    if (r) tokens[2 * tid + i] = mask[i] | uint32_t(row) << 16;
    uint32_t left = mask[i];
    for (int q = 0; q < r; q += 2 << kind) {
      uint32_t rest = left;
      for (int n = 0; n < 2 << kind; ++n) rest &= rest - 1u;
      T.tokens[at] = uint16_t(left ^ rest);
      T.expert[at] = uint16_t(2 * tid + i);
      T.first[at++] = uint16_t(row + q);
      left = rest;
    }
    row += r;
  }
  if (tid == 0) {
    T.groups = of(kind, all_a, all_b);
    T.kind = kind;
    T.first[T.groups] = uint16_t(all_a & 1023u);
  }
  __syncthreads();
  if (id >= 0) {
    const uint32_t m = tokens[id];
    const int r = int(m >> 16) + __builtin_popcount(m & 0xffffu & ((1u << tok) - 1u));
    T.token[r] = uint8_t(tok);
    T.row_weight[r] = C.weights[tid];
  }
  __syncthreads();
}

// One wave's choice for token tok, or for it and the wave's second one.
template <int J, bool SIGMOID, int N>
__device__ __forceinline__ void choose(const MoeLayerArgs& a, int tok, float* mine, LayerChoice& C, uint32_t* tokens) {
  const int lane = threadIdx.x & 63;
  const TopkRule rule = topk_rule<J, SIGMOID>(a.n_experts, a.k, a.bias != nullptr, a.groups, a.keep, a.top2, a.renorm);
  float l[N][J], b[J];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = J * lane + j;
      const int64_t at = int64_t(tok + kLayerWaves * n) * a.ld + min(e, a.n_experts - 1);
      const float v = a.bf16 ? logit<true>(a.logits, at) : logit<false>(a.logits, at);
      l[n][j] = e < a.n_experts ? v : -INFINITY;
    }
#pragma unroll
  for (int j = 0; j < J; ++j) b[j] = a.bias ? a.bias[min(J * lane + j, a.n_experts - 1)] : 0.f;
  TopkChoice c[N];
  topk_wave<J, SIGMOID, J <= 4>(
      l, rule, [&](int j) { return b[j]; },
      [&](int j) { return min(J * lane + j, a.n_experts - 1) / rule.gs * rule.per; }, mine, c);
#pragma unroll
  for (int n = 0; n < N; ++n)
    if (lane < a.k) {
      const int p = (tok + kLayerWaves * n) * a.k + lane;
      C.ids[p] = c[n].expert;
      C.weights[p] = c[n].weight * a.scale;
      if (c[n].expert >= 0) atomicOr(&tokens[c[n].expert], 1u << (tok + kLayerWaves * n));
    }
}

template <int J, bool SIGMOID>
__device__ __forceinline__ void choose_all(const MoeLayerArgs& a, int wave, float* mine, LayerChoice& C, uint32_t* tokens) {
  static_assert(kLayerMaxTokens <= 2 * kLayerWaves, "a wave has up to two tokens");
  static_assert(2 * 64 * J * 4 <= kLayerTokens, "LDS");
  if (wave + kLayerWaves < a.t) choose<J, SIGMOID, 2>(a, wave, mine, C, tokens);
  else if (wave < a.t) choose<J, SIGMOID, 1>(a, wave, mine, C, tokens);
}

// 16-byte pieces of a row of 128 activations lie in LDS at piece ^ spread(row): 16 lanes that
// an LDS read serves at once (rows 0..3, 12..15 of one piece, 4..11 of the fourth after it)
// are then in different banks.
__device__ __forceinline__ int spread(int row) { return (row & 7) | ((row >> 3 ^ row >> 2) & 1) << 3; }

// Two neighbours of h in 32 bits: whole numbers of 12 bits, the even one's lowest, and the exponent
// byte, as fp32 has it, of their unit, 2^-10 of the larger one's binade.  0 stands for zeros.
constexpr uint32_t kPairEnds = 0xF5000000u;       // from here on: pairs with an infinity (what rounds to 2^128 too), NaN
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  const uint32_t most = umax(__float_as_uint(a) & 0x7FFFFFFFu, __float_as_uint(b) & 0x7FFFFFFFu);
  if (most > 0x7F800000u) return 0xFF000000u;     // 0·inf, NaN
  if (most == 0x7F800000u) {
    // 2^11 - 1 times 2^127 is infinite; a number beside an infinity does not matter
    auto end = [](float v) { return __builtin_isinf(v) ? v > 0.f ? 0x7FFu : 0x801u : 0u; };
    return 0xFE000000u | end(b) << 12 | end(a);
  }
  // the larger one to the next binade where it rounds there; no unit below fp32's smallest normal
  const uint32_t unit = umax((most + 0x1000u) >> 23, 11u) - 10u;
  const float per = __uint_as_float((254u - unit) << 23);
  const uint32_t qa = uint32_t(int(__builtin_rintf(a * per))), qb = uint32_t(int(__builtin_rintf(b * per)));
  return unit << 24 | (qb & 0xFFFu) << 12 | (qa & 0xFFFu);
}
// The pair as two bf16 parts each, exact: cut to 8 bits, and the rest (0 beside an infinity).
__device__ __forceinline__ void pair_parts(uint32_t v, uint32_t& high, uint32_t& low) {
  const float unit = __uint_as_float(v >> 1 & 0x7F800000u);
  const uint32_t a = __float_as_uint(float(int(v << 20) >> 20) * unit), b = __float_as_uint(float(int(v << 8) >> 20) * unit);
  auto rest = [](uint32_t p) { return __float_as_uint(__uint_as_float(p) - __uint_as_float(p & 0xFFFF0000u)); };
  high = __builtin_amdgcn_perm(b, a, 0x07060302u);
  low = __builtin_amdgcn_perm(rest(b), rest(a), 0x07060302u);
}

// The steps of a wave, CODES codes each, groups of up to ROWS tokens.  PAIRS: how the second kernel finds h.
template <bool DOWN, bool PAIRS, int ROWS, int CODES>
__device__ __forceinline__ void stream(const MoeLayerArgs& a, unsigned char* lds, LayerTables& T) {
  constexpr int kParts = CODES / 128;             // 1 KB of weights each
  constexpr int kRowBytes = 2 * CODES, kPieces = kRowBytes / 16, kPerCopy = 1024 / kRowBytes;   // rows of activations
  constexpr int kPlanes = DOWN && !PAIRS ? 2 : 1, kOfPlane = ROWS / kPerCopy;   // as copied
  constexpr int kCopies = kPlanes * kOfPlane, kOps = kParts + kCopies + 1;
  constexpr int kRowsAt = 1024 * kParts, kMetaAt = kRowsAt + 1024 * kCopies, kStage = kMetaAt + 256;
  constexpr int kRests = DOWN && PAIRS ? 1024 * kOfPlane : 0;         // behind the ring: pairs' lower parts of a step
  constexpr int D = (kLayerRing - kRests) / kStage;
  constexpr bool kBoth = DOWN && ROWS <= 8;
  constexpr int kReads = DOWN && !kBoth ? 2 : 1;  // of a column
  static_assert((D - 1) * kOps <= 63, "the waits count the copies in flight");
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int axis = DOWN ? a.inter : a.d, n = DOWN ? a.d : 2 * a.inter;
  const int steps = (axis + CODES - 1) / CODES, groups = __builtin_amdgcn_readfirstlane(T.groups);
  const Slabs L{n, axis, QMM_MXFP4_G32};
  const int last = L.count() - 1;
  const uint32_t width = uint32_t(L.width(0) / 2), width_last = uint32_t(L.width(last) / 2);
  const uint32_t mrow = uint32_t(L.meta_row(0)), mrow_last = uint32_t(L.meta_row(last)), mquad = uint32_t(L.meta_quad());
  const uint32_t slab_bytes = uint32_t(n) * (kSlabCodes / 2);   // of a slab that another follows
  const uint32_t codes_bytes = uint32_t(n) * (uint32_t(axis) / 2), meta_bytes = (uint32_t(n) + 3) / 4 * mquad;
  const int64_t meta_offset = (kHeaderBytes + int64_t(codes_bytes) + 255) / 256 * 256;
  const uint8_t* stack = DOWN ? a.down : a.gate_up;
  const int64_t stride = DOWN ? a.down_stride : a.gate_up_stride;
  const uint32_t row_bytes = uint32_t(axis) * 2u;
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(DOWN ? a.h : a.x, uint32_t(DOWN ? kPlanes * a.t * a.k : a.t) * row_bytes);
  const uint32_t plane = DOWN ? uint32_t(a.t * a.k) * row_bytes : 0u;
  unsigned char* ring = lds + wave * kLayerRing;
  const uint32_t ring_at = lds_addr(ring);

  // Pieces of work.  First kernel: up to 8 outputs of a group, as many as give all waves of the
  // grid as many pieces, dealt out in turn.  Second: a wave has an even share, in a row, of the
  // (group, step) of a block of columns; a piece is its steps of a group.
  const int waves = kLayerWaves * int(gridDim.x), me = wave * int(gridDim.x) + int(blockIdx.x);
  int outputs = 8;
  if (!DOWN) {
    const int turns = (groups * (a.inter / 8) + waves - 1) / waves;
    outputs = max(1, (groups * a.inter + turns * waves - 1) / max(turns * waves, 1));
    while (outputs < 8 && groups * ((a.inter + outputs - 1) / outputs) > turns * waves) ++outputs;
    if (a.pairs) outputs += outputs & 1;
  }
  const int of_group = DOWN ? steps : (a.inter + outputs - 1) / outputs;
  const int work = groups * of_group;
  const int begin = DOWN ? work * wave / kLayerWaves : me, end = DOWN ? work * (wave + 1) / kLayerWaves : work;
  const int blocks = DOWN ? (a.d + a.cols - 1) / a.cols : 0;
  const int rounds = DOWN ? (blocks - int(blockIdx.x) + int(gridDim.x) - 1) / int(gridDim.x) : 1;
  struct Piece {
    int pos, j, at;     // in the work; its group, and its place in it
    // its first output or step, and how many it has
    __device__ int from(int outputs) const { return DOWN ? at : at * outputs; }
  };
  auto size = [&](const Piece& p) { return DOWN ? min(end - p.pos, steps - p.at) : min(outputs, a.inter - p.at * outputs); };
  const Piece start{begin, begin / of_group, begin % of_group};
  const int hop_j = waves / of_group, hop_at = waves % of_group;
  auto advance = [&](Piece& p) {
    if (DOWN) {
      p.pos += size(p);
      p.at = 0;
      ++p.j;
      return;
    }
    p.pos += waves;
    p.at += hop_at;
    p.j += hop_j;
    if (p.at >= of_group) {
      p.at -= of_group;
      ++p.j;
    }
  };

  // ---- the copies' place in the sequence
  // A copy of weights: 16 >> (kParts - 1) rows of 64 * kParts bytes.  Reads of 16-byte pieces by
  // 16 rows are free of conflicts with the pieces at piece ^ (row >> 1).
  constexpr int kRowPieces = 4 * kParts, kRowsOf = 64 / kRowPieces;
  auto wrow = [&](int i) { return kRowsOf * i + lane / kRowPieces; };
  auto wpiece = [&](int i) { return (lane % kRowPieces) ^ (wrow(i) >> 1 & (kRowPieces - 1)); };
  const int part = lane % kParts;                 // of a step's exponents
  int c_round = 0, c_h = 0, c_to = 0;
  Piece next = start;
  __amdgpu_buffer_rsrc_t cr = make_rsrc(stack, 0), mr = cr;
  uint32_t w_full[kParts], w_last[kParts], m_full = 0, m_last = 0, aoff[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) aoff[i] = kOOB8;
#pragma unroll
  for (int i = 0; i < kParts; ++i) w_full[i] = w_last[i] = kOOB8;
  auto copied_row = [&](int i) { return kPerCopy * (i % kOfPlane) + lane / kPieces; };
  auto column = [&](int i) { return copied_row(i) + (kBoth && i >= kOfPlane ? 8 : 0); };
  auto copied_at = [&](int i) { return 8 * ((lane % kPieces) ^ spread(column(i))); };       // code
  auto open = [&]() {
    int e = __builtin_amdgcn_readfirstlane(T.expert[next.j]), at = __builtin_amdgcn_readfirstlane(T.first[next.j]);
    int stop = __builtin_amdgcn_readfirstlane(T.first[next.j + 1]);
    const int from = next.from(outputs), many = size(next);
    // wait states between these, which vector instructions write, and the copies that read what follows from them
    asm volatile("s_nop 4" : "+s"(e), "+s"(at), "+s"(stop));
    const uint8_t* blob = stack + int64_t(e) * stride;
    cr = make_rsrc(blob + kHeaderBytes, codes_bytes);
    mr = make_rsrc(blob + meta_offset, meta_bytes);
    // row r of the 16: columns of the block, or 8 outputs' gate rows and their up rows
    const int n0 = (int(blockIdx.x) + c_round * int(gridDim.x)) * a.cols;
    const int rows = DOWN ? min(a.cols, a.d - n0) : many;
    auto row = [&](int r) { return uint32_t(DOWN ? n0 + r : from + (r & 7) + (r >= 8 ? a.inter : 0)); };
    auto any = [&](int r) { return (DOWN ? r : r & 7) < rows; };
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      w_full[i] = any(wrow(i)) ? row(wrow(i)) * width + 16u * uint32_t(wpiece(i)) : kOOB8;
      w_last[i] = any(wrow(i)) ? row(wrow(i)) * width_last + 16u * uint32_t(wpiece(i)) : kOOB8;
    }
    const int mr16 = lane / kParts & 15;
    const bool meta = lane < 16 * kParts && any(mr16);
    m_full = meta ? (row(mr16) >> 2) * mquad + (row(mr16) & 3u) * mrow + 4u * uint32_t(part) : kOOB8;
    m_last = meta ? (row(mr16) >> 2) * mquad + (row(mr16) & 3u) * mrow_last + 4u * uint32_t(part) : kOOB8;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int r = at + copied_row(i), q = min(r, kLayerMaxPairs - 1);
      aoff[i] = r < stop ? uint32_t(DOWN ? q : T.token[q]) * row_bytes + 2u * uint32_t(copied_at(i)) + (i < kOfPlane ? 0u : plane) : kOOB8;
    }
    c_h = DOWN ? from : 0;
    c_to = DOWN ? from + many : steps;
    advance(next);
  };
  bool more = rounds > 0 && begin < end;          // copies left
  auto copies = [&](int stage) {
    const int h = c_h, s = h * CODES / kSlabCodes, in_slab = h & (kSlabCodes / CODES - 1);
    const uint32_t at = ring_at + uint32_t(stage * kStage);
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      copy16_to_lds_from(cr, (s == last ? w_last[i] : w_full[i]) | (CODES * h + 32 * wpiece(i) < axis ? 0u : kOOB8),
                         uint32_t(s) * slab_bytes + uint32_t(CODES / 2 * in_slab), at + 1024u * uint32_t(i));
#pragma unroll
    for (int i = 0; i < kCopies; ++i)
      copy16_to_lds_from(ar, aoff[i] | (CODES * h + copied_at(i) < axis ? 0u : kOOB8), uint32_t(kRowBytes * h),
                         at + kRowsAt + 1024u * uint32_t(i));
    copy4_to_lds(mr, ((s == last ? m_last : m_full) + uint32_t(64 * s + CODES / 32 * in_slab)) |
                         (CODES * h + 128 * part < axis ? 0u : kOOB8), at + kMetaAt);
    if (++c_h == c_to) {
      if (next.pos >= end) {
        next = start;
        more = ++c_round < rounds;
      }
      if (more) open();
    }
  };
  if (more) open();
#pragma unroll 1
  for (int i = 0; i < D && more; ++i) copies(i);

  // Of the two waves on a SIMD the one with the lower index issues its copies first and is done
  // earlier, and the tail has half the copies in flight.  The other half of the workgroup is
  // therefore raised; over many steps the first is too, every other step.  One token, 8 of 256
  // experts of 3584x2048 (before later steps): 32.8 us without, 32.0 as it is, 32.6 in turns; 16
  // tokens, 8 of 256: 232.7, 232.5, 224.8.
  const int mine = DOWN ? end - begin : (work - begin + waves - 1) / waves * steps;
  const bool in_turns = mine > 40;
  if (wave >= kLayerWaves / 2) __builtin_amdgcn_s_setprio(1);

  // A column of the products is a row of the group (zeros past it); with up to 8 rows both
  // parts of h have columns in one product, h's rests those from 8 on.
  const int row = min(kBoth ? c & 7 : c, ROWS - 1);
  const bool low = kBoth && c >= 8;
  const int x0 = spread(row + (low ? 8 : 0));
  unsigned char* const rests = ring + D * kStage;

  // Pairs of a step into their parts, a row of the group at once, the upper parts in place, the
  // lower ones behind the ring.
  auto part_pairs = [&](unsigned char* st, int rows) {
    constexpr int kWords = kRowBytes / 256;       // of a lane
    typedef uint32_t words_t __attribute__((ext_vector_type(kWords)));
    words_t v[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) v[r] = reinterpret_cast<const words_t*>(st + kRowsAt + kRowBytes * r)[lane];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (r > 0 && r >= rows) break;
      words_t high, rest;
      uint32_t most = 0;
#pragma unroll
      for (int q = 0; q < kWords; ++q) {
        uint32_t h, l;
        pair_parts(v[r][q], h, l);
        high[q] = h;
        rest[q] = l;
        most = umax(most, v[r][q]);
      }
      if (__ballot(most >= kPairEnds)) {
#pragma unroll
        for (int q = 0; q < kWords; ++q) rest[q] = v[r][q] >= kPairEnds ? 0u : rest[q];
      }
      reinterpret_cast<words_t*>(st + kRowsAt + kRowBytes * r)[lane] = high;
      // row r's rests as row r + 8 of the columns: spread(r) ^ spread(r + 8) is piece 8
      *reinterpret_cast<words_t*>(rests + kRowBytes * r + ((4 * kWords * lane) ^ (kBoth ? 128 : 0))) = rest;
    }
    asm volatile("" : : : "memory");              // before the operands' reads, in the wave's own order
  };

  int stage = 0;
  f32x4_t* red = reinterpret_cast<f32x4_t*>(lds + kLayerRed);
  for (int round = 0; round < rounds; ++round) {
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};           // token c, columns 4g .. 4g + 3
    for (Piece t = start; t.pos < end; advance(t)) {
      const int from = t.from(outputs), many = size(t);
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
      const int n_steps = DOWN ? many : steps;
      const int rows_of_group = DOWN && PAIRS ? __builtin_amdgcn_readfirstlane(T.first[t.j + 1] - T.first[t.j]) : 0;
      for (int h = 0; h < n_steps; ++h) {
        if (in_turns && wave < kLayerWaves / 2) {
          if (h & 1) __builtin_amdgcn_s_setprio(1);
          else __builtin_amdgcn_s_setprio(0);
        }
        if (more) wait_copies<(D - 1) * kOps>();
        else wait_copies<0>();
        unsigned char* st = ring + stage * kStage;
        u32x4_t w[kParts], b[kParts][4][kReads];
        uint32_t e8[kParts];
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          w[i] = *reinterpret_cast<const u32x4_t*>(st + 64 * kParts * c + 16 * ((4 * i + g) ^ (c >> 1 & (kRowPieces - 1))));
          e8[i] = st[kMetaAt + 4 * kParts * c + 4 * i + g];
        }
        if constexpr (kRests > 0) part_pairs(st, rows_of_group);
        // the parts' rows of column c
        const unsigned char* const upper = st + kRowsAt + kRowBytes * row;
        const unsigned char* const lower = (kRests ? rests : st + kRowsAt + 1024 * kOfPlane) + kRowBytes * row;
#pragma unroll
        for (int i = 0; i < kParts; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int p = 0; p < kReads; ++p)
              b[i][j][p] = *reinterpret_cast<const u32x4_t*>((p || low ? lower : upper) + 16 * ((16 * i + 4 * g + j) ^ x0));
        wait_reads();                             // ... and is in registers: its stage is free
        if (more) copies(stage);
        stage = stage + 1 == D ? 0 : stage + 1;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          const float scale = e8m0_scale(e8[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bf16x8_t v = __builtin_bit_cast(bf16x8_t, mxfp4_word_to_bf16x8(w[i][j], scale));
#pragma unroll
            for (int p = 0; p < kReads; ++p)
              acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8_t, b[i][j][p]), acc, 0, 0, 0);
          }
        }
      }
      if (DOWN) {
        // to the lanes of the rows' tokens: column c is token c
        const uint32_t m = T.tokens[t.j];
        const int of_token = __builtin_popcount(m & ((1u << c) - 1u));
        const bool has = m >> c & 1u;
        const float weight = has ? T.row_weight[T.first[t.j] + of_token] : 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v = __shfl(acc[e], 16 * g + of_token);
          if (kBoth) v += __shfl(acc[e], 16 * g + of_token + 8);
          sum[e] = has ? __builtin_fmaf(weight, v, sum[e]) : sum[e];
        }
      } else {
        // gate rows in the lanes with g < 2, the same outputs' up rows 32 lanes on
        const int at = T.first[t.j], rows = T.first[t.j + 1] - at;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = silu(acc[e]) * __shfl_xor(acc[e], 32);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          if (c >= rows || g >= 2 || 4 * g + e >= many) continue;
          uint16_t* const h = a.h + int64_t(at + c) * a.inter + from + 4 * g + e;
          if (a.pairs) {                          // `from` and `many` are even
            *reinterpret_cast<uint32_t*>(h) = pack_pair(v[e], v[e + 1]);
            continue;
          }
          // the nearest bf16 and what it leaves: 16 bits of v, so that out has its own rounding alone
          const uint32_t hi = pack_bf16x2(v[e], v[e + 1]);
          const float r0 = __builtin_isfinite(bf16_lo(hi)) ? v[e] - bf16_lo(hi) : 0.f;
          const float r1 = __builtin_isfinite(bf16_hi(hi)) ? v[e + 1] - bf16_hi(hi) : 0.f;
          const uint32_t rest = pack_bf16x2(r0, r1);
          uint16_t* const low = h + int64_t(a.t) * a.k * a.inter;
          h[0] = uint16_t(hi);
          low[0] = uint16_t(rest);
          if (4 * g + e + 1 < many) {
            h[1] = uint16_t(hi >> 16);
            low[1] = uint16_t(rest >> 16);
          }
        }
      }
    }
    if (DOWN) {
      if (wave) red[64 * (wave - 1) + lane] = sum;
      wait_reads();
      phase_end();
      if (wave == 0 && c < a.t) {
#pragma unroll
        for (int w = 0; w < kLayerWaves - 1; ++w) sum += red[64 * w + lane];
        const int column = (int(blockIdx.x) + round * int(gridDim.x)) * a.cols, cols = min(a.cols, a.d - column);
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          if (4 * g + e >= cols) continue;
          const int64_t o = int64_t(c) * a.d + column + 4 * g + e;
          uint32_t v = 0;
          if (a.shared) v = *reinterpret_cast<const uint32_t*>(a.shared + o);
          *reinterpret_cast<uint32_t*>(a.out + o) = pack_bf16x2(sum[e] + bf16_lo(v), sum[e + 1] + bf16_hi(v));
        }
      }
      wait_reads();
      phase_end();                                // the next columns' sums take the place
    }
  }
  wait_copies<0>();
}

template <bool DOWN, bool PAIRS>
__device__ __forceinline__ void stream_any(const MoeLayerArgs& a, unsigned char* lds, LayerTables& T) {
  // with 8 and 16 rows steps of 128 codes: of 256 the ring would hold one or two
  const int kind = __builtin_amdgcn_readfirstlane(T.kind);
  if (kind == 0) stream<DOWN, PAIRS, 2, 256>(a, lds, T);
  else if (kind == 1) stream<DOWN, PAIRS, 4, 256>(a, lds, T);
  else if (kind == 2) stream<DOWN, PAIRS, 8, 128>(a, lds, T);
  else stream<DOWN, PAIRS, 16, 128>(a, lds, T);
}

__global__ __launch_bounds__(64 * kLayerWaves) void layer_gate_up_kernel(MoeLayerArgs a) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  LayerTables& T = *reinterpret_cast<LayerTables*>(lds + kLayerTables);
  LayerChoice& C = *reinterpret_cast<LayerChoice*>(lds + kLayerRed);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float* mine = reinterpret_cast<float*>(lds + wave * kLayerRing);
  uint32_t* tokens = reinterpret_cast<uint32_t*>(lds + kLayerTokens);
  clear_tokens(tokens, a.n_experts);
  // experts a lane: as few as hold them (16 tokens, 6 of 300 experts of 512 x 256: 34.1 us with 8,
  // 40.1 with 16)
  if (a.n_experts <= 64) {
    if (a.sigmoid) choose_all<1, true>(a, wave, mine, C, tokens);
    else choose_all<1, false>(a, wave, mine, C, tokens);
  } else if (a.n_experts <= 128) {
    if (a.sigmoid) choose_all<2, true>(a, wave, mine, C, tokens);
    else choose_all<2, false>(a, wave, mine, C, tokens);
  } else if (a.n_experts <= 256) {
    if (a.sigmoid) choose_all<4, true>(a, wave, mine, C, tokens);
    else choose_all<4, false>(a, wave, mine, C, tokens);
  } else if (a.n_experts <= 512) {
    if (a.sigmoid) choose_all<8, true>(a, wave, mine, C, tokens);
    else choose_all<8, false>(a, wave, mine, C, tokens);
  } else {
    if (a.sigmoid) choose_all<16, true>(a, wave, mine, C, tokens);
    else choose_all<16, false>(a, wave, mine, C, tokens);
  }
  __syncthreads();
  const int pairs = a.t * a.k, tid = threadIdx.x;
  if (blockIdx.x == 0 && tid < pairs) {
    a.topk[tid] = C.ids[tid];
    a.weights[tid] = C.weights[tid];
  }
  make_tables(T, C, tokens, pairs, a.k, a.n_experts);
  stream_any<false, false>(a, lds, T);
}

template <bool PAIRS>
__global__ __launch_bounds__(64 * kLayerWaves) void layer_down_kernel(MoeLayerArgs a) {
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  LayerTables& T = *reinterpret_cast<LayerTables*>(lds + kLayerTables);
  LayerChoice& C = *reinterpret_cast<LayerChoice*>(lds + kLayerRed);
  const int pairs = a.t * a.k, tid = threadIdx.x;
  uint32_t* tokens = reinterpret_cast<uint32_t*>(lds + kLayerTokens);
  int e = -1;
  if (tid < pairs) {
    e = a.topk[tid];
    e = e < a.n_experts ? e : -1;
    C.ids[tid] = e;
    C.weights[tid] = a.weights[tid];
  }
  clear_tokens(tokens, a.n_experts);
  if (e >= 0) atomicOr(&tokens[e], 1u << tid / a.k);
  __syncthreads();
  make_tables(T, C, tokens, pairs, a.k, a.n_experts);
  stream_any<true, PAIRS>(a, lds, T);
}

}  // namespace

int launch_moe_layer(const MoeLayerArgs& args, void* stream) {
  hipStream_t s = static_cast<hipStream_t>(stream);
  DevInfo di{};
  const int cus = device_info(&di) == 0 && di.cus > 0 ? di.cus : 256;
  MoeLayerArgs a = args;
  // columns of a workgroup: as many as give every CU the same number of blocks
  const int rounds = (a.d + 16 * cus - 1) / (16 * cus);
  a.cols = std::max(8, (a.d + 2 * cus * rounds - 1) / (2 * cus * rounds) * 2);
  const int64_t outputs = int64_t(a.t) * a.k * a.inter;
  const int blocks = (a.d + a.cols - 1) / a.cols;
  const dim3 block(64 * kLayerWaves), up_grid(unsigned(std::min<int64_t>(cus, (outputs + 31) / 32)));
  const ProfileEvents pe = take_profile_events();
  hipExtLaunchKernelGGL(layer_gate_up_kernel, up_grid, block, kLayerLds, s, static_cast<hipEvent_t>(pe.start), nullptr,
                        0, a);
  const int err = int(hipGetLastError());
  if (err) return err;
  hipExtLaunchKernelGGL(a.pairs ? layer_down_kernel<true> : layer_down_kernel<false>, dim3(unsigned(std::min(cus, blocks))),
                        block, kLayerLds, s, nullptr, static_cast<hipEvent_t>(pe.stop), 0, a);
  return int(hipGetLastError());
}

}  // namespace qmm
