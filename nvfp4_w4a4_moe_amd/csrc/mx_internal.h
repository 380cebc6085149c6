// Internal launch interface of the MXFP4 kernels (mx_api.cpp to the kernel files).
// Every launcher only enqueues work on `stream`; arguments are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nv4 {

inline int64_t mx_scale_stride(int64_t K) { return (K / 32 + 3) / 4 * 4; }

struct MxQuantArgs {
  const void *x;
  int x_is_f32;
  int64_t x_rows, rows, K, ldx;
  const int32_t *row_index;  // may be null
  int layout;                // NV4_ROWS / NV4_COLS / NV4_COLS_BATCHED / NV4_ROWS_AND_COLS
  int nseg;
  const int32_t *seg_offsets, *seg_padded_offsets;
  int ceil_rule;
  uint8_t *codes, *scales;    // the layout's output ([rows][K], or the transpose)
  uint8_t *codes2, *scales2;  // NV4_ROWS_AND_COLS: the row-direction output
  int64_t out_K;              // columns of the transpose
  int32_t *dev_status;
};
hipError_t launch_mx_quantize(const MxQuantArgs &a, hipStream_t stream);

struct MxDequantArgs {
  const uint8_t *codes, *scales;
  int64_t rows, K;
  void *out;
  int out_is_f32;
  int64_t ldo;
};
hipError_t launch_mx_dequantize(const MxDequantArgs &a, hipStream_t stream);
hipError_t launch_mx_padded_offsets(const int32_t *offsets, int nseg, int32_t *padded, hipStream_t stream);

struct MxGemmArgs {
  const uint8_t *a_codes, *a_scales;
  int64_t a_rows, K;
  const int32_t *a_rows_index;  // may be null
  const uint8_t *b_codes, *b_scales;
  int64_t b_rows;
  const int32_t *offsets;
  int E;
  int64_t M_cap, N;  // N = output columns
  int group_mode, epilogue;
  void *C;           // may be null with q_codes
  int c_is_f32;
  int64_t ldc;
  uint8_t *q_codes, *q_scales;  // SwiGLU: the quantised result [M_cap][N], or null
  int ceil_rule;
};
hipError_t launch_mx_gemm(const MxGemmArgs &a, hipStream_t stream);

struct MxFewArgs {
  const void *x;
  int x_is_f32;
  int64_t ldx;
  const float *logits;  // null: topk_ids and topk_w are inputs
  int T, E, k, flags;
  int32_t *topk_ids;
  float *topk_w;
  const uint8_t *w13_codes, *w13_scales, *w2_codes, *w2_scales;
  int H, I;
  int ceil_rule;
  void *out;
  int out_is_f32;
  int64_t ldo;
  void *ws;
  int32_t *dev_status;
};
size_t mx_few_workspace_bytes(int64_t T, int E, int k, int64_t H, int64_t I);
hipError_t launch_mx_few(const MxFewArgs &a, hipStream_t stream);

}  // namespace nv4
