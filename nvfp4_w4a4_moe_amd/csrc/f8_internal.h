// Internal launch interface of the FP8 kernels (f8_api.cpp to the kernel files).
// Every launcher only enqueues work on `stream`; arguments are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nv4 {

constexpr int64_t kF8Block = 128;  // NV4_F8_BLOCK
inline int64_t f8_blocks(int64_t n) { return (n + kF8Block - 1) / kF8Block; }

struct F8QuantArgs {
  const void *x;
  int x_is_f32;
  int64_t x_rows, rows, K, ldx;
  const int32_t *row_index;  // may be null
  int layout;                // NV4_ROWS / NV4_COLS / NV4_ROWS_AND_COLS / NV4_F8_TILES
  int nseg;
  const int32_t *seg_offsets, *seg_padded_offsets;
  int pow2;
  uint8_t *codes;    // the layout's output ([rows][K], or the transpose)
  float *scales;
  uint8_t *codes2;   // NV4_ROWS_AND_COLS: the row-direction output
  float *scales2;
  int64_t out_K;     // columns of the transpose
  int32_t *dev_status;
};
hipError_t launch_f8_quantize(const F8QuantArgs &a, hipStream_t stream);

struct F8DequantArgs {
  const uint8_t *codes;
  const float *scales;
  int64_t rows, K;
  int nseg;
  void *out;
  int out_is_f32;
  int64_t ldo;
};
hipError_t launch_f8_dequantize(const F8DequantArgs &a, hipStream_t stream);

struct F8TransposeArgs {
  const uint8_t *codes;
  const float *scales;
  int64_t nseg, m, K;
  uint8_t *out_codes;
  float *out_scales;
};
hipError_t launch_f8_transpose(const F8TransposeArgs &a, hipStream_t stream);

struct F8GemmArgs {
  const uint8_t *a_codes;
  const float *a_scales;
  int64_t a_rows, K;
  const int32_t *a_rows_index;  // may be null
  const uint8_t *b_codes;
  const float *b_scales;
  int64_t b_rows;
  const int32_t *offsets;
  int E;
  int64_t M_cap, N;  // N = output columns
  int group_mode, epilogue;
  int pow2;          // every scale of both operands is a power of two
  void *C;           // may be null with q_codes
  int c_is_f32;
  int64_t ldc;
  uint8_t *q_codes;  // SwiGLU: the quantised result [M_cap][N], or null
  float *q_scales;
  int q_pow2;
};
hipError_t launch_f8_gemm(const F8GemmArgs &a, hipStream_t stream);

}  // namespace nv4
