// MXFP4 grouped GEMM: dispatch to the tile for the problem's size.
#include "mx_gemm_kernel.h"

namespace nv4 {

typedef MxTile<4, 2, 2, 4, 3, 2> MxLarge;  // 256 x 256, eight waves of 64 x 128

hipError_t launch_mx_gemm(const MxGemmArgs &g, hipStream_t stream) {
  if (g.group_mode == NV4_GROUP_K) return mx_launch<MxLarge, NV4_GROUP_K, NV4_EPI_NONE>(g, stream);
  if (g.epilogue == NV4_EPI_SWIGLU) return mx_launch<MxLarge, NV4_GROUP_M, NV4_EPI_SWIGLU>(g, stream);
  return mx_launch<MxLarge, NV4_GROUP_M, NV4_EPI_NONE>(g, stream);
}

}  // namespace nv4
