// FP8 grouped GEMM for a few rows: a single token's experts, small batches.
//
// The same sums as in f8_gemm_kernel.h.  With a few rows there are fewer large tiles than CUs, and a tile's K / 128 stages
// follow one another: 16 us for one row against 2048 x 2048, of which each stage's latency is 0.5.  Here a
// workgroup has 16 columns (SwiGLU: of gate and up) of 16 rows, and its four waves take the blocks of K in
// turn, so that all of K is in flight at once.  Operands go from memory to registers as the matrix instruction wants
// them (16 x 16 x 128: four lanes read 64 consecutive bytes of a row); the waves' sums meet in LDS and are added in
// the waves' order.  (A quantised result is not for this kernel: a block's 128 columns in one workgroup leave a token's
// eight experts to 48 CUs, which took 27 us against the 64 x 256 tiles' 17.)
#include <algorithm>

#include "f8_device.h"
#include "f8_internal.h"
#include "grouped_tiles.h"
#include "nv4_internal.h"
#include "../../include/nv4moe.h"

namespace nv4 {
namespace {

constexpr int kWaves = 4;  // wave w takes blocks w, w + 4, ..
constexpr int kRows = 16, kCols = 16;
constexpr uint32_t kAbsent = 0xFFFFFF00u;  // behind every buffer: reads as zero

struct FewBlock {  // a lane's 32 codes of one row and block
  i32x4 lo, hi;
};
__device__ __forceinline__ f32x4 few_product(const FewBlock &w, const FewBlock &t, bool wide) {
  f32x4 p = {};
  if (wide) {
    p = __builtin_amdgcn_mfma_f32_16x16x32_f16(f8_to_f16(w.lo.x, w.lo.y), f8_to_f16(t.lo.x, t.lo.y), p, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_f16(f8_to_f16(w.lo.z, w.lo.w), f8_to_f16(t.lo.z, t.lo.w), p, 0, 0, 0);
    p = __builtin_amdgcn_mfma_f32_16x16x32_f16(f8_to_f16(w.hi.x, w.hi.y), f8_to_f16(t.hi.x, t.hi.y), p, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(f8_to_f16(w.hi.z, w.hi.w), f8_to_f16(t.hi.z, t.hi.w), p, 0, 0, 0);
  }
  const i32x8 a{w.lo.x, w.lo.y, w.lo.z, w.lo.w, w.hi.x, w.hi.y, w.hi.z, w.hi.w};
  const i32x8 b{t.lo.x, t.lo.y, t.lo.z, t.lo.w, t.hi.x, t.hi.y, t.hi.z, t.hi.w};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, p, 0, 0, 0, 0, 0, 0);
}

// The expert and first row of row tile `slot` (tiles of 16 rows, in the experts' order), by every wave for
// itself; false if there are fewer.  Offsets below zero or decreasing are taken as empty, those behind M_cap as M_cap.
__device__ __forceinline__ bool few_tile(const F8GemmArgs &g, int slot, int &e, int &m0, int &m_end) {
  const int lane = threadIdx.x & 63, per = (g.E + 63) / 64;
  const auto off = [&](int i) { return min(max(g.offsets[min(i, g.E)], 0), (int)g.M_cap); };
  const auto tiles = [&](int lo, int hi) { return (max(hi - lo, 0) + kRows - 1) / kRows; };
  int own = 0;
  for (int i = 0; i < per; ++i) {
    const int x = lane * per + i;
    own += tiles(off(x), off(x + 1));
  }
  int run = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(run, o, 64);
    if (lane >= o) run += x;
  }
  const uint64_t behind = __ballot(run > slot);
  if (behind == 0) return false;
  const int l = __ffsll((unsigned long long)behind) - 1;  // the lane whose experts have it
  int left = slot - __builtin_amdgcn_readlane(run - own, l);
  for (e = l * per; e < g.E; ++e) {
    m0 = off(e);
    m_end = off(e + 1);
    const int n = tiles(m0, m_end);
    if (left < n) {
      m0 += left * kRows;
      return true;
    }
    left -= n;
  }
  return false;
}

// four consecutive columns of a row
template <bool OUT_F32>
__device__ __forceinline__ void few_store(const F8GemmArgs &g, int row, int col, f32x4 v) {
  const int n = (int)g.N - col;
  const int64_t at = (int64_t)row * g.ldc + col;
  if constexpr (OUT_F32) {
    float *c = static_cast<float *>(g.C) + at;
    if (n >= 4 && reinterpret_cast<uintptr_t>(c) % 16 == 0) {
      *reinterpret_cast<f32x4 *>(c) = v;
      return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < n) c[r] = v[r];
  } else {
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
    const bf16x4 b{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
    __bf16 *c = static_cast<__bf16 *>(g.C) + at;
    if (n >= 4 && reinterpret_cast<uintptr_t>(c) % 8 == 0) {
      *reinterpret_cast<bf16x4 *>(c) = b;
      return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < n) c[r] = b[r];
  }
}

template <int EPI, bool OUT_F32>
__global__ __launch_bounds__(kWaves * 64) __attribute__((amdgpu_waves_per_eu(4)))
void k_f8_gemm_few(F8GemmArgs g) {
  constexpr bool SWIGLU = EPI == NV4_EPI_SWIGLU;
  constexpr int F = SWIGLU ? 2 : 1;  // the gate rows' fragment and the up rows'
  constexpr int kAhead = 4 / F;      // blocks of K that a wave has in flight, as the registers last
  __shared__ f32x4 sums[kWaves - 1][F][64];
  int e, m0, m_end;
  if (!few_tile(g, blockIdx.y, e, m0, m_end)) return;
  e = __builtin_amdgcn_readfirstlane(e);
  m0 = __builtin_amdgcn_readfirstlane(m0);
  m_end = __builtin_amdgcn_readfirstlane(m_end);
  const int lane = threadIdx.x & 63, i16 = lane & 15, part = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) ;
  const int n0 = blockIdx.x * kCols, N = (int)g.N;
  const int blocks = (int)((g.K + 127) / 128);
  const uint32_t ld = (uint32_t)g.K, sld = (uint32_t)blocks * 4;
  const int64_t b_rows = (SWIGLU ? 2 : 1) * g.N, b_srows = (b_rows + 127) / 128;
  const auto codes_a = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(g.a_codes), (short)0,
                                                         (int)(uint32_t)(g.a_rows * g.K), 0x00020000);
  const auto scales_a = __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(g.a_scales), (short)0,
                                                          (int)(uint32_t)(g.a_rows * sld), 0x00020000);
  const auto codes_b = __builtin_amdgcn_make_buffer_rsrc(
      mx_uniform_ptr(g.b_codes + (int64_t)e * b_rows * g.K), (short)0, (int)(uint32_t)(b_rows * g.K), 0x00020000);
  const float *scales_b[F];
  // this lane's token and weight rows; four lanes share a row, 16 bytes each of its next 64
  const int row = m0 + i16;
  uint32_t at_a = kAbsent, at_sa = kAbsent, at_b[F];
  if (row < m_end) {
    const uint32_t r = g.a_rows_index ? (uint32_t)min(max(g.a_rows_index[row], 0), (int)g.a_rows - 1) : (uint32_t)row;
    at_a = r * ld;
    at_sa = r * sld;
  }
#pragma unroll
  for (int f = 0; f < F; ++f) {
    const uint32_t n = (uint32_t)(n0 + f * N);
    at_b[f] = n0 + i16 < N ? (n + i16) * ld : kAbsent;
    scales_b[f] = g.b_scales + ((int64_t)e * b_srows + n / 128) * blocks;  // the same for the wave
  }
  struct Stage {
    FewBlock t, w[F];
    float ts, ws[F];
  } st[kAhead];
  const auto load = [&](Stage &s, int b) MX_INLINE {
    const uint32_t k = (uint32_t)b * 128 + part * 16;
    const bool lo = k < (uint32_t)g.K, hi = k + 64 < (uint32_t)g.K;
    // (saturating: without a row the sum stays behind the buffer)
    const auto at = [&](uint32_t base, bool in, uint32_t kk) MX_INLINE {
      return in ? __builtin_elementwise_add_sat(base, kk) : kAbsent;
    };
#pragma unroll
    for (int f = 0; f < F; ++f) {
      s.w[f].lo = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(codes_b, at(at_b[f], lo, k), 0, kStream));
      s.w[f].hi = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(codes_b, at(at_b[f], hi, k + 64), 0, kStream));
    }
    s.t.lo = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(codes_a, at(at_a, lo, k), 0, 0));
    s.t.hi = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(codes_a, at(at_a, hi, k + 64), 0, 0));
    s.ts = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(scales_a, at(at_sa, b < blocks, (uint32_t)b * 4), 0, 0));
#pragma unroll
    for (int f = 0; f < F; ++f) s.ws[f] = b < blocks ? scales_b[f][b] : 0.0f;
  };
  f32x4 acc[F] = {};
#pragma unroll
  for (int d = 0; d < kAhead; ++d) load(st[d], wave + d * kWaves);
  for (int b = wave; b < blocks; b += kAhead * kWaves) {
#pragma unroll
    for (int d = 0; d < kAhead; ++d) {
      // (blocks behind the last one are zeros under scales of zero)
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const f32x4 p = few_product(st[d].w[f], st[d].t, OUT_F32);
        const float s = st[d].ts * st[d].ws[f];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[f][r] = __builtin_fmaf(p[r], s, acc[f][r]);
      }
      load(st[d], b + (d + kAhead) * kWaves);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int f = 0; f < F; ++f) sums[wave - 1][f][lane] = acc[f];
  }
  __syncthreads();
  if (wave > 0 || row >= m_end) return;
#pragma unroll
  for (int w = 0; w < kWaves - 1; ++w)
#pragma unroll
    for (int f = 0; f < F; ++f) acc[f] += sums[w][f][lane];
  if constexpr (SWIGLU) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[0][r] = mx_swiglu(acc[0][r], acc[1][r]);
  }
  few_store<OUT_F32>(g, row, n0 + part * 4, acc[0]);
}

}  // namespace

int64_t f8_few_tiles(const F8GemmArgs &g) {
  return g.M_cap / kRows + std::min<int64_t>(g.E, g.M_cap);
}

hipError_t launch_f8_gemm_few(const F8GemmArgs &g, hipStream_t stream) {
  if (g.M_cap == 0) return hipSuccess;
  const dim3 grid((unsigned)((g.N + kCols - 1) / kCols), (unsigned)f8_few_tiles(g));
  if (g.epilogue == NV4_EPI_SWIGLU) {
    if (g.c_is_f32) k_f8_gemm_few<NV4_EPI_SWIGLU, true><<<grid, kWaves * 64, 0, stream>>>(g);
    else k_f8_gemm_few<NV4_EPI_SWIGLU, false><<<grid, kWaves * 64, 0, stream>>>(g);
  } else {
    if (g.c_is_f32) k_f8_gemm_few<NV4_EPI_NONE, true><<<grid, kWaves * 64, 0, stream>>>(g);
    else k_f8_gemm_few<NV4_EPI_NONE, false><<<grid, kWaves * 64, 0, stream>>>(g);
  }
  return hipGetLastError();
}

}  // namespace nv4
