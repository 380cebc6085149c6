// The segment that a tile of padded columns lies in, found by a whole workgroup.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nv4 {

struct SegmentOf {
  int32_t index, start, first_row, end_row;  // the segment, its padded start, its rows
};

// The last of nseg segments whose padded start is <= p0, every thread a candidate: one round trip for
// up to NT segments where a binary search takes eight.  All threads call it; *out is in LDS.
template <int NT>
__device__ __forceinline__ void find_segment(const int32_t *offsets, const int32_t *padded, int nseg, int64_t p0,
                                             SegmentOf *out) {
  const int tid = threadIdx.x;
  if (tid == 0) *out = SegmentOf{0, 0, 0, 0};  // (starts that do not begin at 0 leave an empty segment)
  __syncthreads();
  for (int lo = 0, n = nseg;;) {
    const int step = (n + NT - 1) / NT, at = lo + tid * step;
    if (tid * step < n) {
      const int32_t start = padded[at], r0 = offsets[at], r1 = offsets[at + 1];
      const bool last = (tid + 1) * step >= n || padded[at + step] > p0;
      if (start <= p0 && last) *out = SegmentOf{at, start, r0, r1};
    }
    __syncthreads();
    if (step == 1) break;
    n = min(step, n - (out->index - lo));
    lo = out->index;
    __syncthreads();
  }
}

}  // namespace nv4
