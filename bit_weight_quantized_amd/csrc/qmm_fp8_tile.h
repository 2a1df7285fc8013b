// What the LDS tile kernels of the block-scaled e4m3 product share: waits, the
// place of a workgroup's tile, and the rows that it reads.
#pragma once

#include "qmm_fp8.h"
#include "qmm_fp8_device.h"

namespace qmm {

// Waits and barriers as fences of their own (the copies are asm): at most N
// copies of the wave in flight; every LDS read of the wave done; end of a phase.
template <int N>
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory"); }
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }
__device__ __forceinline__ void phase_end() {
  asm volatile("" : : : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
}

// Arguments of the kernels, as they come from the entry points.
struct Fp8TileArgs {
  const uint8_t* w;
  const float* ws;
  int n, d, nb;
  const uint8_t* x;
  const float* xs;
  int64_t t;
  uint16_t* y;
  int64_t ldy;
  int tiles_n;
  // grouped
  const int32_t* row_index;
  const int32_t* seg_expert;
  const int32_t* seg_offsets;
  int n_experts, n_seg, m_total, t_x;
};

// A workgroup's tile: rows [m0, m_end) of the grouped or dense rows, output
// columns from n0, the matrix of its expert.
struct Fp8Place {
  int64_t m0, m_end;
  int n0;
  bool bad_expert;
  bool starts;            // the first rows of its segment
  const uint8_t* w;
  const float* ws;
  int sb;                 // scale rows of the gate half
};

// Row tiles of 256 segments from s0 on, four neighbouring ones a lane.
template <int kT>
struct Fp8Tiles {
  int at[5], tiles[4], sum, first, all;   // offsets, tiles; of the lane, before it, of the wave

  __device__ __forceinline__ void scan(const Fp8TileArgs& a, int s0) {
    const int lane = threadIdx.x & 63;
    sum = 0;
#pragma unroll
    for (int u = 0; u < 5; ++u) at[u] = min(max(a.seg_offsets[min(s0 + 4 * lane + u, a.n_seg)], 0), a.m_total);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int rows = at[u + 1] - at[u];
      tiles[u] = rows > 0 ? (rows + kT - 1) / kT : 0;
      sum += tiles[u];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int up = __shfl_up(incl, o);
      if (lane >= o) incl += up;
    }
    first = incl - sum;
    all = __builtin_amdgcn_readlane(incl, 63);
  }

  // The tt-th tile, if it is one of these: its segment's number from s0, rows [lo, hi),
  // and whether they are the segment's first.
  __device__ __forceinline__ int find(int tt, int& lo, int& hi, bool& starts) const {
    const uint64_t who = __ballot(tt >= first && tt < first + sum);
    if (!who) return -1;
    int s = -1, b = 0, e = 0, f = first, nth = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (s < 0 && tt >= f && tt < f + tiles[u]) {
        s = 4 * int(threadIdx.x & 63) + u;
        nth = tt - f;
        b = at[u] + nth * kT;
        e = min(b + kT, at[u + 1]);
      }
      f += tiles[u];
    }
    const int src = __builtin_ctzll(who);
    lo = __builtin_amdgcn_readlane(b, src);
    hi = __builtin_amdgcn_readlane(e, src);
    starts = __builtin_amdgcn_readlane(nth, src) == 0;
    return __builtin_amdgcn_readlane(s, src);
  }
};

// The tile of this workgroup, kT rows by kOut columns; false where the grid's
// bound has more row tiles than there are.  XCD id mod 8 takes a contiguous run
// of tiles, in blocks of 8 weight tiles by all activation tiles, activation
// tiles slowest: the 32 workgroups at work on an XCD share 8 weight and 4
// activation tiles in its L2.  The runs are equal parts of the tiles that there
// are, not of the grid: with the grid's, whose bound is 192 row tiles where 64
// segments of 512 rows have 159, two XCDs had a third of the others' work.
template <int kT, int kOut, bool GROUPED, bool GLU>
__device__ __forceinline__ bool fp8_place(const Fp8TileArgs& a, Fp8Place& p) {
  const int nout = GLU ? a.n / 2 : a.n;
  int tiles_t = gridDim.x / a.tiles_n;
  Fp8Tiles<kT> some;
  if constexpr (GROUPED) {
    // every wave looks for itself
    int all = 0;
    for (int s0 = 0; s0 < a.n_seg; s0 += 256) {
      some.scan(a, s0);
      all += some.all;
    }
    tiles_t = min(tiles_t, all);
  }
  const int total = tiles_t * a.tiles_n;
  const int xcd = blockIdx.x & 7, share = total >> 3, extra = total & 7;
  if (int(blockIdx.x >> 3) >= share + (xcd < extra ? 1 : 0)) return false;
  const int id = xcd * share + min(xcd, extra) + (blockIdx.x >> 3);
  const int strip = id / (8 * tiles_t), in_strip = id - strip * 8 * tiles_t;
  const int width = min(8, a.tiles_n - 8 * strip);
  int tt = in_strip / width;
  const int tn = 8 * strip + in_strip - tt * width;
  p.n0 = tn * kOut;
  p.bad_expert = false;
  p.starts = false;
  p.w = a.w;
  p.ws = a.ws;
  p.sb = GLU ? (nout + kFp8Block - 1) / kFp8Block : 0;
  if constexpr (!GROUPED) {
    p.m0 = int64_t(tt) * kT;
    p.m_end = min(a.t, p.m0 + kT);
    return true;
  }
  for (int s0 = 0; s0 < a.n_seg; s0 += 256) {
    if (a.n_seg > 256) some.scan(a, s0);
    int lo, hi;
    const int s = some.find(tt, lo, hi, p.starts);
    if (s >= 0) {
      p.m0 = lo;
      p.m_end = hi;
      const int e = a.seg_expert[s0 + s];
      p.bad_expert = e < 0 || e >= a.n_experts;
      if (!p.bad_expert) {
        p.w += int64_t(e) * a.n * a.d;
        p.ws += int64_t(e) * (GLU ? 2 * p.sb : (a.n + kFp8Block - 1) / kFp8Block) * a.nb;
      }
      return true;
    }
    tt -= some.all;
  }
  return false;
}

// Activation rows as the copies address them: dense rows from the tile's first
// row, grouped rows anywhere in x (below 2 GiB, checked by the caller).
template <bool GROUPED>
struct Fp8Source {
  __amdgpu_buffer_rsrc_t x, s;
  __device__ __forceinline__ Fp8Source(const Fp8TileArgs& a, const Fp8Place& p) {
    const uint32_t rows = GROUPED ? uint32_t(a.t_x) : uint32_t(p.m_end - p.m0);
    const int64_t first = GROUPED ? 0 : p.m0;
    x = make_rsrc(a.x + first * a.d, rows * uint32_t(a.d));
    s = make_rsrc(a.xs + first * a.nb, rows * uint32_t(a.nb) * 4u);
  }
  // row of the tile -> row of the buffers; -1 past the tile, or (grouped) for a
  // bad row or expert
  __device__ __forceinline__ int operator()(const Fp8TileArgs& a, const Fp8Place& p, int row) const {
    if (p.m0 + row >= p.m_end) return -1;
    if constexpr (!GROUPED) return row;
    const int src = a.row_index ? a.row_index[p.m0 + row] : int(p.m0 + row);
    return p.bad_expert || src < 0 || src >= a.t_x ? -1 : src;
  }
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

// formats 0: e4m3; block exponents 0 select the unscaled instruction
__device__ __forceinline__ f32x4_t mfma_e4m3(const i32x8_t a, const i32x8_t b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
// the same from exact bf16, with fp32 sums
__device__ __forceinline__ f32x4_t mfma_e4m3_exact(const i32x8_t a, const i32x8_t b) {
  f32x4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < 4; ++q)
    p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(e4m3x8_to_bf16(uint32_t(a[2 * q]), uint32_t(a[2 * q + 1])),
                                                e4m3x8_to_bf16(uint32_t(b[2 * q]), uint32_t(b[2 * q + 1])), p, 0, 0, 0);
  return p;
}

// Eight neighbouring output columns c .. c + 7 of a row, at any alignment: the
// memory takes 16 unaligned bytes in one store (rows of an odd length, 1449 x 10945,
// d = 336: 54 us with single columns).
typedef uint32_t u32x4_at2_t __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ void store8(uint16_t* row, int c, int nout, u32x4_t v) {
  if (c + 8 <= nout) {
    *reinterpret_cast<u32x4_at2_t*>(row + c) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < nout) row[c + e] = uint16_t(v[e >> 1] >> (16 * (e & 1)));
  }
}

}  // namespace qmm
