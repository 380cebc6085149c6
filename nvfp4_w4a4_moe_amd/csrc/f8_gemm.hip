// FP8 grouped GEMM: the kernel for the problem's size.  f8_gemm_kernel.h has the pipelined kernel, whose tiles are
// compiled in f8_gemm_large.hip, f8_gemm_medium.hip and f8_gemm_small.hip; f8_gemm_few.hip is for a few rows.
// Times in us, K = 2048 or, with FP32 results, 768.
#include <algorithm>

#include "f8_internal.h"
#include "nv4_internal.h"
#include "../../include/nv4moe.h"

namespace nv4 {

hipError_t launch_f8_gemm_large(const F8GemmArgs &g, hipStream_t stream);
hipError_t launch_f8_gemm_medium(const F8GemmArgs &g, hipStream_t stream);
hipError_t launch_f8_gemm_small(const F8GemmArgs &g, hipStream_t stream);
hipError_t launch_f8_gemm_few(const F8GemmArgs &g, hipStream_t stream);
int64_t f8_few_tiles(const F8GemmArgs &g);

hipError_t launch_f8_gemm(const F8GemmArgs &g, hipStream_t stream) {
  // weight gradients: 128 x 128 (256 x 128 has too few registers for a scale of every weight row: 64 experts, 768 x
  // 2048, 512 rows each, BF16: 98 against 102; 128 experts, 1536 x 2048, 1024 rows: 782 against 834)
  if (g.group_mode == NV4_GROUP_K) return launch_f8_gemm_medium(g, stream);
  const bool swiglu = g.epilogue == NV4_EPI_SWIGLU;
  const int64_t n = swiglu ? 2 * g.N : g.N, cus = device_cu_count();
  // Few rows: up to four of that kernel's workgroups for each CU (they are resident at once).  SwiGLU to 768 columns, a row
  // for each of 8, 16, 24, 32 experts: 11.0, 14.5, 20.6, 24.7, with 64 x 128 tiles 18, 20, 24, 24; 96 and 128 rows against
  // 2048 x 2048: 11.6 and 14.1 against 17.7 and 18.1 with 128 x 128, FP32 16 experts to 2048: 16.3 against 11.4.
  if (!g.q_codes && f8_few_tiles(g) * ((g.N + 15) / 16) <= 4 * cus) return launch_f8_gemm_few(g, stream);
  // 64 x 128 up to 64 rows per expert (128 experts, SwiGLU to 768: 48, 64, 80, 128 rows each: 72, 75, 135, 139, with 128 x
  // 128 tiles 90, 91, 90, 98)
  if (g.M_cap <= 64 * (int64_t)g.E) return launch_f8_gemm_small(g, stream);
  // 256-row tiles from about 144 rows per expert (192 rows each: 131 against 141, 128: 109 against 97) where the rounds
  // of tiles on the CUs, an expert's last tile half full in the mean, come out cheaper: a 256 x 256 tile takes 3.4 times
  // a 128 x 128 tile's share of a CU, a 256 x 128 tile with FP32 results 1.8 times (8192^3: 527 against 699, FP32 930
  // against 1049; 8192 x 2048 x 768, 96 large tiles: 34 against 24; 4096^3, 256 of them: 71 against 91).
  const auto rounds = [&](int64_t bm, int64_t bn) {
    return (((g.M_cap + bm - 1) / bm + (g.E - 1) / 2) * ((n + bn - 1) / bn) + cus - 1) / cus;
  };
  const bool wide = g.c_is_f32, broad = g.q_codes;
  if (g.M_cap >= 144 * (int64_t)g.E && !(wide && broad) &&
      rounds(256, wide ? 128 : 256) * (wide ? 18 : 34) <= rounds(128, broad ? 256 : 128) * (broad ? 20 : 10))
    return launch_f8_gemm_large(g, stream);
  return launch_f8_gemm_medium(g, stream);
}

}  // namespace nv4
