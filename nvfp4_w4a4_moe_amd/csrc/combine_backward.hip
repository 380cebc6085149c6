// The gradients of the top-k weighted combine for gfx950:
//   dY[token_row[t][j]] = w[t][j] dout[t],   dw[t][j] = sum_h dout[t][h] Y[token_row[t][j]][h].
//
// Memory bound: a token's row of dout is read, k rows of Y read and k rows of dY written.  One workgroup a
// token; every thread owns V consecutive columns (16 bytes of a row of Y, or 8 of BF16 where rows start between
// 16-byte steps) and keeps a partial dot product for each of up to eight choices at a time, whose loads are all
// under way together.  16384 tokens of eight BF16 rows of 2048: 227 us, 5.0 TB/s (with 8-byte accesses 284).
#include "many_groups.h"
#include "nv4_device.h"
#include "nv4_internal.h"
#include "router_internal.h"
#include "topk_device.h"

namespace nv4 {
namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 8;

// V values of a row as they are in memory, and as FP32
template <bool F32, int V>
struct Cols {
  typedef uint32_t Words __attribute__((ext_vector_type(F32 ? 4 : V / 2)));
  static constexpr int N = F32 ? V / 4 : 1;
  Words w[N];
  __device__ __forceinline__ void load(const void *p, int64_t at) {
    const Words *q = reinterpret_cast<const Words *>(static_cast<const char *>(p) + at * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = __builtin_nontemporal_load(q + i);
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (F32) return __uint_as_float(w[i / 4][i % 4]);
    else return __uint_as_float(i % 2 ? w[0][i / 2] & 0xFFFF0000u : w[0][i / 2] << 16);
  }
  // d times s, each product rounded to the type
  template <class D>
  __device__ __forceinline__ void store(void *p, int64_t at, const D &d, float s) {
    Words *q = reinterpret_cast<Words *>(static_cast<char *>(p) + at * (F32 ? 4 : 2));
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i / 4][i % 4] = __float_as_uint(d.get(i) * s);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2)
        w[0][i / 2] = f32_to_bf16_rne(d.get(i) * s) | (f32_to_bf16_rne(d.get(i + 1) * s) << 16);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) __builtin_nontemporal_store(w[i], q + i);
  }
};

template <bool DOUT_F32, bool Y_F32, int V>
__global__ __launch_bounds__(kThreads) void k_combine_backward(CombineBackwardArgs a) {
  __shared__ float sums[kThreads / 64][kAtOnce];
  const int64_t t = group_index();
  if (t >= a.T) return;
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
    for (int64_t c = (int64_t)tid * V; c < a.H; c += kThreads * V) {
      Cols<DOUT_F32, V> d;
      Cols<Y_F32, V> y[kAtOnce];
      d.load(a.dout, t * a.H + c);
      if (a.dtopk_w) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
          if (row[j] >= 0) y[j].load(a.Y, row[j] * a.ldy + c);  // (the same for the workgroup)
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          if (row[j] < 0) continue;
#pragma unroll
          for (int i = 0; i < V; ++i) dot[j] = __builtin_fmaf(d.get(i), y[j].get(i), dot[j]);
        }
      }
      if (a.dY) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
          if (row[j] >= 0) y[j].store(a.dY, row[j] * a.lddy + c, d, w[j]);
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

template <bool DOUT_F32, bool Y_F32, int V>
hipError_t launch(const CombineBackwardArgs &a, hipStream_t stream) {
  k_combine_backward<DOUT_F32, Y_F32, V><<<many_groups(a.T), kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_backward(const CombineBackwardArgs &a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  if (a.y_is_f32) return a.dout_is_f32 ? launch<true, true, 4>(a, stream) : launch<false, true, 4>(a, stream);
  // 16-byte accesses where every row that is touched allows them
  const auto steps = [](const void *p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0; };
  const bool wide = a.H % 8 == 0 && (a.dout_is_f32 || steps(a.dout, a.H)) && (!a.dtopk_w || steps(a.Y, a.ldy)) &&
                    (!a.dY || steps(a.dY, a.lddy));
  if (wide) return a.dout_is_f32 ? launch<true, false, 8>(a, stream) : launch<false, false, 8>(a, stream);
  return a.dout_is_f32 ? launch<true, false, 4>(a, stream) : launch<false, false, 4>(a, stream);
}

}  // namespace nv4
