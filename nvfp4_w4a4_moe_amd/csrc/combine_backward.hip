// The gradients of the top-k weighted combine for gfx950:
//   dY[token_row[t][j]] = w[t][j] dout[t],   dw[t][j] = sum_h dout[t][h] Y[token_row[t][j]][h].
//
// Memory bound: a token's row of dout is read, k rows of Y read and k rows of dY written.  One workgroup a
// token; every thread owns 4 consecutive columns and keeps a partial dot product for each of up to eight
// choices at a time.
#include "nv4_device.h"
#include "nv4_internal.h"
#include "router_internal.h"
#include "topk_device.h"

namespace nv4 {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 8;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <bool F32>
__device__ __forceinline__ f32x4 load4(const void *p, int64_t at) {
  if constexpr (F32) {
    return __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + at));
  } else {
    const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(p) + at));
    return f32x4{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u), __uint_as_float(v[1] << 16),
                 __uint_as_float(v[1] & 0xFFFF0000u)};
  }
}
template <bool F32>
__device__ __forceinline__ void store4(void *p, int64_t at, f32x4 v) {
  if constexpr (F32) {
    __builtin_nontemporal_store(v, reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at));
  } else {
    __builtin_nontemporal_store(u32x2{f32_to_bf16_rne(v[0]) | (f32_to_bf16_rne(v[1]) << 16),
                                      f32_to_bf16_rne(v[2]) | (f32_to_bf16_rne(v[3]) << 16)},
                                reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p) + at));
  }
}

template <bool DOUT_F32, bool Y_F32>
__global__ __launch_bounds__(kThreads) void k_combine_backward(CombineBackwardArgs a) {
  __shared__ float sums[kThreads / 64][kAtOnce];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
    const int nj = min(a.k - j0, kAtOnce);
    int64_t row[kAtOnce];
    float w[kAtOnce], dot[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      row[j] = j < nj ? a.token_row[t * a.k + j0 + j] : -1;
      if (row[j] >= a.rows) row[j] = -1;
      w[j] = j < nj ? a.topk_w[t * a.k + j0 + j] : 0.0f;
      dot[j] = 0.0f;
    }
    for (int64_t c = (int64_t)tid * 4; c < a.H; c += kThreads * 4) {
      const f32x4 d = load4<DOUT_F32>(a.dout, t * a.H + c);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        if (row[j] < 0) continue;  // uniform
        if (a.dtopk_w) {
          const f32x4 y = load4<Y_F32>(a.Y, row[j] * a.ldy + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) dot[j] = __builtin_fmaf(d[i], y[i], dot[j]);
        }
        if (a.dY) store4<Y_F32>(a.dY, row[j] * a.lddy + c, d * w[j]);
      }
    }
    if (a.dtopk_w) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const float x = wave_sum_dpp(dot[j]);
        if ((tid & 63) == 0) sums[tid >> 6][j] = x;
      }
      __syncthreads();
      if (tid < nj) {
        float x = sums[0][tid];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) x += sums[i][tid];
        a.dtopk_w[t * a.k + j0 + tid] = x;
      }
    }
  }
}

}  // namespace

hipError_t launch_combine_backward(const CombineBackwardArgs &a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const unsigned grid = (unsigned)a.T;
  if (a.dout_is_f32) {
    if (a.y_is_f32) k_combine_backward<true, true><<<grid, kThreads, 0, stream>>>(a);
    else k_combine_backward<true, false><<<grid, kThreads, 0, stream>>>(a);
  } else {
    if (a.y_is_f32) k_combine_backward<false, true><<<grid, kThreads, 0, stream>>>(a);
    else k_combine_backward<false, false><<<grid, kThreads, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace nv4
