// Internal launch interface of the router's training kernels (router_api.cpp to the kernel files).
// Every launcher only enqueues work on `stream`; arguments are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nv4 {

struct BalanceArgs {
  const float *logits;
  int64_t T;
  int E, k;
  const int32_t *topk_ids;
  const uint8_t *mask;         // may be null
  int nseg;
  const int32_t *seg_offsets;  // null: one segment of all tokens
  int32_t *counts;
  float *prob_sums;
  int32_t *tokens;
  float *loss;
  void *ws;
  int32_t *dev_status;
};
size_t balance_workspace_bytes(int64_t T, int E, int nseg);
hipError_t launch_balance_loss(const BalanceArgs &a, hipStream_t stream);

struct BalanceBackwardArgs {
  const float *logits;
  int64_t T;
  int E, k;
  const int32_t *topk_ids;
  const uint8_t *mask;
  int nseg;
  const int32_t *seg_offsets;
  const int32_t *counts, *tokens;
  const float *dloss;    // may be null
  const float *dtopk_w;  // may be null
  int renorm;
  float *dlogits;
  int32_t *dev_status;
};
hipError_t launch_balance_backward(const BalanceBackwardArgs &a, hipStream_t stream);

struct CombineBackwardArgs {
  const void *dout;
  int dout_is_f32;
  const void *Y;
  int y_is_f32;
  int64_t ldy, rows;
  const int32_t *token_row;
  const float *topk_w;
  int64_t T;
  int k;
  int64_t H;
  void *dY;        // may be null
  int64_t lddy;
  float *dtopk_w;  // may be null
};
hipError_t launch_combine_backward(const CombineBackwardArgs &a, hipStream_t stream);

}  // namespace nv4
