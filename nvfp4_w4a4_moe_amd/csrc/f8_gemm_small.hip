// FP8 grouped GEMM, 64-row tiles: 64 x 128, or 64 x 256 where the result is re-quantised.
#include "f8_gemm_kernel.h"

namespace nv4 {

hipError_t launch_f8_gemm_small(const F8GemmArgs &g, hipStream_t stream) {
  typedef F8Tile<2, 2, 1, 2, 2, 2> Tile;
  typedef F8Tile<2, 4, 1, 2, 3, 2> Broad;
  if (g.epilogue != NV4_EPI_SWIGLU)
    return g.c_is_f32 ? f8_launch<Tile, NV4_GROUP_M, NV4_EPI_NONE, true>(g, stream)
                      : f8_launch<Tile, NV4_GROUP_M, NV4_EPI_NONE, false>(g, stream);
  if (g.q_codes)
    return g.c_is_f32 ? f8_launch<Broad, NV4_GROUP_M, NV4_EPI_SWIGLU, true, true>(g, stream)
                      : f8_launch<Broad, NV4_GROUP_M, NV4_EPI_SWIGLU, false, true>(g, stream);
  return g.c_is_f32 ? f8_launch<Tile, NV4_GROUP_M, NV4_EPI_SWIGLU, true>(g, stream)
                    : f8_launch<Tile, NV4_GROUP_M, NV4_EPI_SWIGLU, false>(g, stream);
}

}  // namespace nv4
