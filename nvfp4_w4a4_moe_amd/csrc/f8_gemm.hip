// FP8 grouped GEMM: the tile for the problem's size.  The kernel is in f8_gemm_kernel.h; its tiles are
// compiled in f8_gemm_large.hip, f8_gemm_medium.hip and f8_gemm_small.hip.
#include <algorithm>

#include "f8_internal.h"
#include "nv4_internal.h"
#include "../../include/nv4moe.h"

namespace nv4 {

hipError_t launch_f8_gemm_large(const F8GemmArgs &g, hipStream_t stream);
hipError_t launch_f8_gemm_medium(const F8GemmArgs &g, hipStream_t stream);
hipError_t launch_f8_gemm_small(const F8GemmArgs &g, hipStream_t stream);

hipError_t launch_f8_gemm(const F8GemmArgs &g, hipStream_t stream) {
  if (g.group_mode == NV4_GROUP_K) {
    const int64_t large = (int64_t)g.E * ((g.a_rows + 255) / 256) * ((g.b_rows + 127) / 128);
    return large >= device_cu_count() ? launch_f8_gemm_large(g, stream) : launch_f8_gemm_medium(g, stream);
  }
  const bool wide_quant = g.q_codes && g.c_is_f32;
  const int64_t n = g.epilogue == NV4_EPI_SWIGLU ? 2 * g.N : g.N;
  const int64_t large = (g.M_cap / 256 + g.E / 2) * ((n + 255) / 256);
  if (!wide_quant && g.M_cap >= 144 * (int64_t)g.E && large >= device_cu_count()) return launch_f8_gemm_large(g, stream);
  if (g.M_cap >= 64 * (int64_t)g.E) return launch_f8_gemm_medium(g, stream);
  return launch_f8_gemm_small(g, stream);
}

}  // namespace nv4
