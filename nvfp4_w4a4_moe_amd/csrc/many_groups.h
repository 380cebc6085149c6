// Launches of more workgroups than one dimension of a grid can hold.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace nv4 {

// A dimension of a launch counts its work-items in 32 bits, and a launch of more returns success with the grid cut to
// what is left of them modulo 2^32.  The workgroups behind the first 2^21 (of 1024 threads at most) go into the grid's
// second dimension.  2^21 is a multiple of the XCDs: workgroup i still runs on XCD i % 8.
constexpr int64_t kGroupsX = 1 << 21;
inline dim3 many_groups(int64_t groups) {
  return dim3((unsigned)std::min(groups, kGroupsX), (unsigned)((groups + kGroupsX - 1) / kGroupsX));
}

// This workgroup's number; the grid may hold more than were asked for.
__device__ __forceinline__ uint32_t group_index() { return blockIdx.y * gridDim.x + blockIdx.x; }

}  // namespace nv4
