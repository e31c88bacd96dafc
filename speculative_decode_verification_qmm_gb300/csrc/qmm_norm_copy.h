// qmm_norm_copy.h -- how the threads of a CTA share the copy of a row whose ends lie
// anywhere (internal; qmm_norm.cu).  Host and device, so that its bounds are tested
// without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define QMM_HD __host__ __device__ __forceinline__
#else
#define QMM_HD inline
#endif

namespace qmm {

// Row m of a tensor whose row 0 has nothing readable before it and whose last row has nothing
// behind it: `bytes` (more than 16, even) from `skew` (even) behind a boundary of 16 bytes.
// Thread t of `threads` calls group(at, n) for n bytes from the boundary plus `at` on, a
// multiple of 16, and pair(at) for two bytes.  Groups of 16 bytes, the last one ends with the row;
// the first one begins before the row, in or between the tensor's other rows, and is taken in
// pairs where there is none.
template <typename Group, typename Pair>
QMM_HD void copy_row(int t, int threads, int64_t m, int skew, int bytes, Group group, Pair pair) {
  const int end = skew + bytes, head = m == 0 && skew > 0 ? 16 : 0;
  for (int at = head + t * 16; at < end; at += threads * 16) group(at, end - at < 16 ? end - at : 16);
  for (int at = skew + t * 2; at < head; at += threads * 2) pair(at);
}

}  // namespace qmm
