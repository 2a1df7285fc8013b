// Kernel launch helper shared by the .hip files: a plain launch, or, when the
// caller armed profiling events with qmm_profile_next(), a launch whose start
// and stop events are stamped by the dispatch itself (hipExtLaunchKernelGGL),
// so their interval is the kernel's own execution time.
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>

#include "qmm_internal.h"

namespace qmm {

// Rows of one launch of launch_rows.
constexpr int64_t max_launch_rows(unsigned threads) { return (int64_t(1) << 31) / threads; }

template <typename K, typename... Args>
inline void launch_kernel(K kernel, dim3 grid, dim3 block, hipStream_t s, Args... args) {
  ProfileEvents pe = take_profile_events();
  if (pe.start || pe.stop)
    hipExtLaunchKernelGGL(kernel, grid, block, 0, s, static_cast<hipEvent_t>(pe.start),
                          static_cast<hipEvent_t>(pe.stop), 0, args...);
  else
    hipLaunchKernelGGL(kernel, grid, block, 0, s, args...);
}

template <typename K, typename... Args>
inline void launch_kernel_lds(K kernel, dim3 grid, dim3 block, size_t lds, hipStream_t s,
                              Args... args) {
  ProfileEvents pe = take_profile_events();
  if (pe.start || pe.stop)
    hipExtLaunchKernelGGL(kernel, grid, block, uint32_t(lds), s, static_cast<hipEvent_t>(pe.start),
                          static_cast<hipEvent_t>(pe.stop), 0, args...);
  else
    hipLaunchKernelGGL(kernel, grid, block, lds, s, args...);
}

// One workgroup of `threads` for each row and column block (grid y), kernel(args, first
// row).  A grid may have fewer than 2^32 threads along x, so 2^31 threads of rows are
// one launch and the rest take further ones; the events bracket them all.
template <typename A>
inline int launch_rows(void (*kernel)(A, int64_t), const A& args, int64_t rows, unsigned blocks_y, unsigned threads,
                       hipStream_t s) {
  const ProfileEvents pe = take_profile_events();
  const int64_t most = max_launch_rows(threads);
  for (int64_t first = 0; first < rows; first += most) {
    const bool last = rows - first <= most;
    const dim3 grid(unsigned(last ? rows - first : most), blocks_y);
    if (pe.start || pe.stop)
      hipExtLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, static_cast<hipEvent_t>(first ? nullptr : pe.start),
                            static_cast<hipEvent_t>(last ? pe.stop : nullptr), 0, args, first);
    else
      hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, args, first);
    const int err = int(hipGetLastError());
    if (err) return err;
  }
  return 0;
}

}  // namespace qmm
