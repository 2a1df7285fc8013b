// Routing tables of a grouped call, and the search for the segments that have rows, shared
// by the few-row kernels whose workgroups share out the segments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {

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

}  // namespace qmm
