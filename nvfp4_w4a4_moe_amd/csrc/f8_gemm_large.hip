// FP8 grouped GEMM, 256-row tiles: 256 x 256 on the FP8 instruction, 256 x 128 on converted codes (whose registers
// do not last for more).
#include "f8_gemm_kernel.h"

namespace nv4 {

hipError_t launch_f8_gemm_large(const F8GemmArgs &g, hipStream_t stream) {
  typedef F8Tile<4, 2, 2, 4, 2, 2> Square;
  typedef F8Tile<4, 2, 2, 2, 2, 2> Half;
  // BF16 rows that start between lines have a kernel of their own: 8192 rows of 8191 columns, K = 2048: 150 against 219 us,
  // while its registers cost rows at lines up to 5 % (64 experts, K = 768, 2048 columns: 65 against 61)
  typedef F8Tile<4, 2, 2, 4, 2, 2, true> AnyRows;
  if (g.epilogue != NV4_EPI_SWIGLU) {
    if (g.c_is_f32) return f8_launch<Half, NV4_GROUP_M, NV4_EPI_NONE, true>(g, stream);
    const bool lines = (reinterpret_cast<uintptr_t>(g.C) | (uintptr_t)g.ldc * 2) % 64 == 0;
    return lines ? f8_launch<Square, NV4_GROUP_M, NV4_EPI_NONE, false>(g, stream)
                 : f8_launch<AnyRows, NV4_GROUP_M, NV4_EPI_NONE, false>(g, stream);
  }
  if (g.q_codes) return f8_launch<Square, NV4_GROUP_M, NV4_EPI_SWIGLU, false, true>(g, stream);
  return g.c_is_f32 ? f8_launch<Half, NV4_GROUP_M, NV4_EPI_SWIGLU, true>(g, stream)
                    : f8_launch<Square, NV4_GROUP_M, NV4_EPI_SWIGLU, false>(g, stream);
}

}  // namespace nv4
