// FP8 grouped GEMM: the tile for the problem.  The kernel is in f8_gemm_kernel.h.
#include "f8_gemm_kernel.h"

namespace nv4 {

hipError_t launch_f8_gemm(const F8GemmArgs &g, hipStream_t stream) {
  if (g.group_mode == NV4_GROUP_K) return f8_launch<F8Tile<2, 2, 2, 2>, NV4_GROUP_K, NV4_EPI_NONE>(g, stream);
  if (g.epilogue == NV4_EPI_SWIGLU) return f8_launch<F8Tile<1, 4, 2, 2>, NV4_GROUP_M, NV4_EPI_SWIGLU>(g, stream);
  return f8_launch<F8Tile<2, 2, 2, 2>, NV4_GROUP_M, NV4_EPI_NONE>(g, stream);
}

}  // namespace nv4
