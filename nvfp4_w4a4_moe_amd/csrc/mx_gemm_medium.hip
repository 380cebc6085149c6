// MXFP4 grouped GEMM, 128 x 128 tiles: four waves of 64 x 64, stages of K = 256, two workgroups per CU.
#include "mx_gemm_kernel.h"

namespace nv4 {

hipError_t launch_mx_gemm_medium(const MxGemmArgs &g, hipStream_t stream) {
  typedef MxTile<2, 2, 2, 2, 4, 2, 2> Tile;
  if (g.group_mode == NV4_GROUP_K) return mx_launch<Tile, NV4_GROUP_K, NV4_EPI_NONE>(g, stream);
  if (g.epilogue == NV4_EPI_SWIGLU) return mx_launch<Tile, NV4_GROUP_M, NV4_EPI_SWIGLU>(g, stream);
  return mx_launch<Tile, NV4_GROUP_M, NV4_EPI_NONE>(g, stream);
}

}  // namespace nv4
