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
// rows behind an expert's last and give more workgroups).  The row counts stay on the device:
// the choice goes by their mean.  Measured in us, 64 x 128 / 128 x 128 / 256 x 256 tiles:
//   gate and up, K = 2048, N = 768, 128 experts of  32 rows  38.6 / 43.5 / 64.2
//                                                   48       43.3 / 44.2 / 65.6
//                                                   64       53.4 / 44.9 / 65.2
//                                                  128       81.8 / 69.8 / 70.7
//                                                  160       91.4 / 83.0 / 73.5
//                                                  384        202 /  154 /  136
//   one expert, K = N = 2048, rows 2048             14.2 / 17.4 / 21.9   (512, 256, 64 tiles)
//                                  4096             23.3 / 20.3 / 24.4
//                                  8192             40.9 / 33.0 / 28.1
hipError_t launch_rows(const MxGemmArgs &g, hipStream_t stream) {
  const int64_t n = g.epilogue == NV4_EPI_SWIGLU ? 2 * g.N : g.N, cus = device_cu_count();
  const auto tiles = [&](int64_t bm, int64_t bn) { return (g.M_cap / bm + g.E / 2) * ((n + bn - 1) / bn); };
  if (g.M_cap >= 144 * (int64_t)g.E && tiles(256, 256) >= cus) return launch_mx_gemm_large(g, stream);
  if (g.M_cap >= 50 * (int64_t)g.E && tiles(128, 128) > cus) return launch_mx_gemm_medium(g, stream);
  return launch_mx_gemm_small(g, stream);
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs &g, hipStream_t stream) {
  if (g.group_mode != NV4_GROUP_K) return launch_rows(g, stream);
  // weight gradients: no row is wasted, so the large tile as soon as it fills the chip (64
  // experts of 768 x 2048: 138 us against 160)
  const int64_t large = (int64_t)g.E * ((g.a_rows + 255) / 256) * ((g.b_rows + 255) / 256);
  return large >= device_cu_count() ? launch_mx_gemm_large(g, stream) : launch_mx_gemm_medium(g, stream);
}

}  // namespace nv4
