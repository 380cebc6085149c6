// MXFP4 grouped GEMM: the tile for the problem's size.  The kernel is in mx_gemm_kernel.h; its
// tiles are compiled in mx_gemm_large.hip, mx_gemm_medium.hip and mx_gemm_small.hip.
#include <algorithm>

#include "mx_internal.h"
#include "nv4_internal.h"
#include "../../include/nv4moe.h"

namespace nv4 {

hipError_t launch_mx_gemm_large(const MxGemmArgs &g, hipStream_t stream);
hipError_t launch_mx_gemm_medium(const MxGemmArgs &g, hipStream_t stream);
hipError_t launch_mx_gemm_small(const MxGemmArgs &g, hipStream_t stream);

namespace {

// 256-, 128- or 64-row tiles (wider ones do more products per byte, narrower ones waste fewer
// rows behind an expert's last; the narrowest streams its weights).  The row counts stay on the
// device: the choice goes by their mean.  Measured in us with several layers' weights in turn,
// 64 x 128 / 128 x 128 / 256 x 256 tiles:
//   gate and up, K = 2048, N = 768, 128 experts of  16 rows  47.4 / 55.6 / 69.6
//                                                   32       53.3 / 56.5 / 68.1
//                                                   64       67.3 / 67.8 / 71.2
//                                                   96       98.2 / 79.4 / 86.2
//                                                  128        111 / 83.1 / 88.2
//                                                  144        116 / 95.0 / 93.2
//                                                  192        154 /  114 /  105
//                                                  384        266 /  172 /  152
//   K = 768, N = 2048, 64 experts of                32       21.4 / 22.3 / 26.1
//                                                   64       26.4 / 27.3 / 27.6
//                                                  128       39.2 / 35.6 / 37.8
//                                                  160       45.4 / 41.8 / 42.5
//                                                  256       64.0 / 51.3 / 44.1
//   one expert, K = N = 2048, rows                 1024      17.6 / 15.7 / 22.9   (32 large tiles)
//                                                  4096      35.2 / 19.6 / 24.6   (128)
//                                                  8192      62.7 / 32.9 / 31.0   (256)
hipError_t launch_rows(const MxGemmArgs &g, hipStream_t stream) {
  const int64_t n = g.epilogue == NV4_EPI_SWIGLU ? 2 * g.N : g.N;
  const int64_t large = (g.M_cap / 256 + g.E / 2) * ((n + 255) / 256);
  if (g.M_cap >= 144 * (int64_t)g.E && large >= device_cu_count()) return launch_mx_gemm_large(g, stream);
  if (g.M_cap >= 64 * (int64_t)g.E) return launch_mx_gemm_medium(g, stream);
  return launch_mx_gemm_small(g, stream);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs &g, hipStream_t stream) {
  if (g.group_mode != NV4_GROUP_K) return launch_rows(g, stream);
  // weight gradients: no row is wasted, so the large tile as soon as it fills the chip (64
  // experts of 768 x 2048, FP32 results of 32768 rows: 105 us against 106; 128 of 1536 x 2048 and
  // 131072 rows: 572 against 630)
  const int64_t large = (int64_t)g.E * ((g.a_rows + 255) / 256) * ((g.b_rows + 255) / 256);
  return large >= device_cu_count() ? launch_mx_gemm_large(g, stream) : launch_mx_gemm_medium(g, stream);
}

}  // namespace nv4
