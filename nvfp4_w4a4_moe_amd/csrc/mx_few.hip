// A whole MXFP4 expert layer for a few tokens (T <= 64, a decode step) in three kernels.
//
// At this size the layer is bound by reading the chosen experts' weights once (0.53 bytes per
// element; 2.5 MB per expert at hidden size 2048 and expert size 768) and, below that, by
// launches and dependent latencies.  So: few launches, every weight byte requested by a
// 16-byte load whose address depends on one table look-up, and no intermediate but the
// quantised rows.
//
//   1. k_few_route    one workgroup routes all tokens (topk_device.h) and lists the experts in
//                     use: a 64-bit token mask per expert gives its rows in token order without
//                     sorting (row = expert's start + number of lower tokens in the mask).  The
//                     other workgroups quantise x meanwhile.
//   2. k_few_gate_up  one workgroup per (expert in use, 32 columns of I): gate and up products
//                     for all the expert's tokens, SwiGLU and re-quantisation: 32 columns are
//                     one MX block.  The K dimension is split over the four waves.
//   3. k_few_down     one workgroup per 16 columns of H: its waves walk over the experts, add
//                     weight * product into a token table in LDS (one per wave), and the tables
//                     are summed in wave order.  No atomics: the result is deterministic.
//
// Products: v_mfma_scale_f32_16x16x128_f8f6f4 with weight rows as the first operand and up to
// 16 of the expert's tokens as the second, straight from global memory: lane (row, g) holds
// the 16-byte block g of the row's 128-element step, so one load of a wave covers 16 rows x 64
// bytes.
#include <algorithm>

#include "mx_device.h"
#include "mx_internal.h"
#include "mx_rows.h"
#include "topk_device.h"
#include "../../include/nv4moe.h"

namespace nv4 {
namespace {

constexpr int kMaxT = 64;      // tokens (one bit each in an expert's mask)
constexpr int kMaxE = 1024;
constexpr int kGroups = kMaxT / 16;  // 16-token groups of one expert
constexpr int kNone = 0x7FFFFFFF;

// Workspace: [0] the number of experts in use; their ids and first rows; token and weight of
// every row; the quantised x and SwiGLU rows.
struct FewWs {
  int32_t *n_active, *act_e, *act_row, *row_token;
  float *row_w;
  uint8_t *x_codes, *x_scales, *h_codes, *h_scales;
};
__host__ __device__ inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
__host__ __device__ inline size_t few_ws(void *base, int64_t T, int E, int k, int64_t H, int64_t I, FewWs &w) {
  const int64_t R = T * k, A = E < R ? E : R;
  char *p = static_cast<char *>(base);
  size_t at = 0;
  const auto take = [&](size_t b) {
    char *q = p + at;
    at += up256(b);
    return q;
  };
  w.n_active = reinterpret_cast<int32_t *>(take(4));
  w.act_e = reinterpret_cast<int32_t *>(take(A * 4));
  w.act_row = reinterpret_cast<int32_t *>(take((A + 1) * 4));
  w.row_token = reinterpret_cast<int32_t *>(take(R * 4));
  w.row_w = reinterpret_cast<float *>(take(R * 4));
  w.x_codes = reinterpret_cast<uint8_t *>(take(T * (H / 2)));
  w.x_scales = reinterpret_cast<uint8_t *>(take(T * ((H / 32 + 3) / 4 * 4)));
  w.h_codes = reinterpret_cast<uint8_t *>(take(R * (I / 2)));
  w.h_scales = reinterpret_cast<uint8_t *>(take(R * ((I / 32 + 3) / 4 * 4)));
  return at;
}

// NPL, LPT: topk_token's.  Block 0 routes; blocks 1.. quantise 64 units of x each.
template <int NPL, int LPT, bool F32>
__global__ __launch_bounds__(1024) void k_few_route(MxFewArgs a) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x > 0) {
    const int l16 = lane & 15, spr = (a.H + 127) / 128;
    const int unit = (blockIdx.x - 1) * 64 + (tid >> 4);
    const int row = unit / spr, seg = unit - row * spr, col = seg * 128 + l16 * 8;
    uint4 v[F32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (row < a.T && col < a.H) {
        const int64_t at = row * a.ldx + col;
        v[i] = F32 ? reinterpret_cast<const uint4 *>(static_cast<const float *>(a.x) + at)[i]
                   : reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + at)[i];
      }
    }
    uint32_t c, d;
    const bool bad = mx_unit<F32>(v, l16, a.ceil_rule, c, d);
    if (row < a.T) {
      if (col < a.H) *reinterpret_cast<uint32_t *>(ws.x_codes + row * (a.H / 2) + col / 2) = c;
      if (l16 == 0) *reinterpret_cast<uint32_t *>(ws.x_scales + row * ((a.H / 32 + 3) / 4 * 4) + seg * 4) = d;
    }
    if (bad && a.dev_status) atomicOr(a.dev_status, kDsNonFinite);
    return;
  }
  __shared__ unsigned long long mask[kMaxE];
  __shared__ int row0[kMaxE];
  __shared__ int ids[kMaxT * 32];
  __shared__ float wts[kMaxT * 32];
  __shared__ int wsum[16];
  mask[tid] = 0ull;
  __syncthreads();
  const int R = a.T * a.k;
  if (a.logits) {
    constexpr int TPW = kWave / LPT;
    const int sub = lane / LPT, ll = lane % LPT;
    for (int t0 = wave * TPW; t0 < a.T; t0 += 16 * TPW) {
      const int t = t0 + sub;
      const bool valid = t < a.T;
      int id;
      float w;
      const bool nan = topk_token<NPL, LPT>(a.logits + (int64_t)t * a.E, valid, a.E, a.k, a.flags, lane, sub, ll, id, w);
      if (valid && ll < a.k) {
        ids[t * a.k + ll] = id < a.E ? id : kNone;  // every remaining logit was NaN: no expert
        wts[t * a.k + ll] = w;
        if (id < a.E) atomicOr(&mask[id], 1ull << t);
        if (a.topk_ids) a.topk_ids[t * a.k + ll] = id;
        if (a.topk_w) a.topk_w[t * a.k + ll] = w;
      }
      if (nan && lane == 0 && a.dev_status) atomicOr(a.dev_status, kDsNanLogit);
    }
  } else {
    for (int f = tid; f < R; f += 1024) {
      const int id = a.topk_ids[f];
      const bool good = id >= 0 && id < a.E;
      ids[f] = good ? id : kNone;
      wts[f] = a.topk_w[f];
      if (good) atomicOr(&mask[id], 1ull << (f / a.k));
      else if (a.dev_status) atomicOr(a.dev_status, kDsBadExpert);
    }
  }
  __syncthreads();
  // exclusive prefix over the experts of (in use, rows), packed: both stay below 2^16
  const int n = __popcll(mask[tid]);
  const int own = n | (n ? 1 << 16 : 0);
  int s = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(s, o, 64);
    if (lane >= o) s += x;
  }
  if (lane == 63) wsum[wave] = s;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < 16; ++w) before += w < wave ? wsum[w] : 0;
  s += before;
  const int ex = s - own;
  row0[tid] = ex & 0xFFFF;
  if (n) {
    ws.act_e[ex >> 16] = tid;
    ws.act_row[ex >> 16] = ex & 0xFFFF;
  }
  if (tid == 1023) {
    *ws.n_active = s >> 16;
    ws.act_row[s >> 16] = s & 0xFFFF;
  }
  __syncthreads();
  for (int f = tid; f < R; f += 1024) {
    const int id = ids[f];
    if (id == kNone) continue;
    const int t = f / a.k, f0 = t * a.k;
    float w = 0.0f;
    bool first = true;
    if (a.logits) {
      w = wts[f];
    } else {  // the caller's ids may repeat: their weights add up, in order
      for (int j = 0; j < a.k; ++j) {
        if (ids[f0 + j] != id) continue;
        if (f0 + j < f) first = false;
        w += wts[f0 + j];
      }
    }
    if (first) {
      const int r = row0[id] + __popcll(mask[id] & ((1ull << t) - 1ull));
      ws.row_token[r] = t;
      ws.row_w[r] = w;
    }
  }
}

struct Frag {
  int4 c;
  uint32_t s;
};
// Step's block g of a row: 16 bytes of codes and, in byte 0, the block's scale; zeros behind K
// (nb blocks) or without a row.
__device__ __forceinline__ Frag load_frag(const uint8_t *codes, const uint8_t *scales, int64_t row, bool live, int step,
                                          int g, int nb, int sld) {
  Frag f{make_int4(0, 0, 0, 0), 0u};
  const int b = step * 4 + g;
  if (live && b < nb) {
    f.c = *reinterpret_cast<const int4 *>(codes + row * ((int64_t)nb * 16) + b * 16);
    f.s = scales[row * sld + b];
  }
  return f;
}
__device__ __forceinline__ f32x4 mfma16(const Frag &a, const Frag &b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(i32x8{a.c.x, a.c.y, a.c.z, a.c.w, 0, 0, 0, 0},
                                                          i32x8{b.c.x, b.c.y, b.c.z, b.c.w, 0, 0, 0, 0}, c, 4, 4, 0,
                                                          (int)a.s, 0, (int)b.s);
}

constexpr int kGuWaves = 4, kGuSteps = 4;  // steps a wave holds at a time

__global__ __launch_bounds__(kGuWaves * 64) void k_few_gate_up(MxFewArgs a) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  __shared__ float part[kGuWaves][16][64];
  if ((int)blockIdx.y >= *ws.n_active) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int e = ws.act_e[blockIdx.y], r0 = ws.act_row[blockIdx.y], n = ws.act_row[blockIdx.y + 1] - r0;
  const int c0 = blockIdx.x * 32;
  const int nb = a.H / 32, sld = (nb + 3) / 4 * 4, steps = (a.H + 127) / 128;
  const int ng = (n + 15) / 16;
  int tok[kGroups];
#pragma unroll
  for (int q = 0; q < kGroups; ++q) tok[q] = q * 16 + l < n ? ws.row_token[r0 + q * 16 + l] : -1;
  f32x4 acc[kGroups][4];
#pragma unroll
  for (int q = 0; q < kGroups; ++q)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[q][t] = f32x4{0, 0, 0, 0};
  // tiles: gate columns c0.., c0 + 16.., then the up rows
  const int64_t base = (int64_t)e * 2 * a.I + c0 + l;
  for (int s0 = wave; s0 < steps; s0 += kGuWaves * kGuSteps) {
    Frag w[kGuSteps][4];
#pragma unroll
    for (int i = 0; i < kGuSteps; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        w[i][t] = load_frag(a.w13_codes, a.w13_scales, base + (t & 1) * 16 + (t >> 1) * (int64_t)a.I, true,
                            s0 + i * kGuWaves, g, nb, sld);
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      if (q < ng) {
        Frag x[kGuSteps];
#pragma unroll
        for (int i = 0; i < kGuSteps; ++i)
          x[i] = load_frag(ws.x_codes, ws.x_scales, tok[q], tok[q] >= 0, s0 + i * kGuWaves, g, nb, sld);
#pragma unroll
        for (int i = 0; i < kGuSteps; ++i)
#pragma unroll
          for (int t = 0; t < 4; ++t) acc[q][t] = mfma16(w[i][t], x[i], acc[q][t]);
      }
    }
  }
  // sum over the waves, SwiGLU, re-quantise: thread = token slot of 16, two columns
  const int slot = tid >> 4, cc = (tid & 15) * 2;
  const int hnb = a.I / 32, hsld = (hnb + 3) / 4 * 4;
  bool bad = false;
#pragma unroll
  for (int q = 0; q < kGroups; ++q) {
    if (q >= ng) break;
    if (q) __syncthreads();
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[wave][t * 4 + r][lane] = acc[q][t][r];
    __syncthreads();
    // column c sits in tile c / 16, lane (c % 16) / 4 * 16 + slot, register c % 4
    float h[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = cc + u, reg = (c >> 4) * 4 + (c & 3), at = ((c & 15) >> 2) * 16 + slot;
      float gate = 0, up = 0;
#pragma unroll
      for (int w = 0; w < kGuWaves; ++w) {
        gate += part[w][reg][at];
        up += part[w][reg + 8][at];
      }
      h[u] = gate * __builtin_amdgcn_rcpf(1.0f + __expf(-gate)) * up;
    }
    uint32_t m = max(__float_as_uint(h[0]) & 0x7FFFFFFFu, __float_as_uint(h[1]) & 0x7FFFFFFFu);
    m = oct_umax(m);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, false));  // row_mirror
    const uint32_t byte = mx_scale_byte(m, a.ceil_rule);
    uint32_t c = mx_pack_f32<0>(0u, h[0], h[1], mx_scale_value(byte));
    if (byte == kMxNan) c = 0u;
    if (q * 16 + slot < n) {
      bad |= byte == kMxNan;
      const int64_t r = r0 + q * 16 + slot;
      ws.h_codes[r * (a.I / 2) + (c0 + cc) / 2] = (uint8_t)c;
      if ((tid & 15) == 0) ws.h_scales[r * hsld + c0 / 32] = (uint8_t)byte;
    }
  }
  if (bad && a.dev_status) atomicOr(a.dev_status, kDsNonFinite);
}

constexpr int kDnWaves = 16, kDnSteps = 6;

// A wave's share: experts in use wave / parts, + 16 / parts, ..; of each the steps part,
// part + parts, ..  (parts > 1 when fewer than 16 experts are in use).
template <bool OUT_F32>
__global__ __launch_bounds__(kDnWaves * 64) void k_few_down(MxFewArgs a) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  extern __shared__ float table[];  // [wave][token][16 columns]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l = lane & 15, g = lane >> 4;
  const int na = *ws.n_active;
  const int parts = na > 8 ? 1 : na > 4 ? 2 : 4;
  const int part = wave % parts;
  const int nb = a.I / 32, sld = (nb + 3) / 4 * 4, steps = (a.I + 127) / 128;
  const int c0 = blockIdx.x * 16;
  const bool row_live = c0 + l < a.H;
  float *mine = table + wave * a.T * 16;
  for (int i = lane; i < a.T * 4; i += 64) reinterpret_cast<f32x4 *>(mine)[i] = f32x4{0, 0, 0, 0};
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  for (int i = wave / parts; i < na; i += kDnWaves / parts) {
    const int e = ws.act_e[i], r0 = ws.act_row[i], n = ws.act_row[i + 1] - r0;
    const int ng = (n + 15) / 16;
    f32x4 acc[kGroups];
#pragma unroll
    for (int q = 0; q < kGroups; ++q) acc[q] = f32x4{0, 0, 0, 0};
    for (int s0 = part; s0 < steps; s0 += parts * kDnSteps) {
      Frag w[kDnSteps];
#pragma unroll
      for (int s = 0; s < kDnSteps; ++s)
        w[s] = load_frag(a.w2_codes, a.w2_scales, (int64_t)e * a.H + c0 + l, row_live, s0 + s * parts, g, nb, sld);
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        if (q < ng) {
          Frag x[kDnSteps];
#pragma unroll
          for (int s = 0; s < kDnSteps; ++s)
            x[s] = load_frag(ws.h_codes, ws.h_scales, r0 + q * 16 + l, q * 16 + l < n, s0 + s * parts, g, nb, sld);
#pragma unroll
          for (int s = 0; s < kDnSteps; ++s) acc[q] = mfma16(w[s], x[s], acc[q]);
        }
      }
    }
    // lane = row slot l, columns 4 g ..: an expert's rows are different tokens, so no two
    // lanes meet in the table
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      if (q * 16 + l < n) {
        const int r = r0 + q * 16 + l;
        const float w = ws.row_w[r];
        f32x4 *p = reinterpret_cast<f32x4 *>(mine + ws.row_token[r] * 16 + g * 4);
        f32x4 v = *p;
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] += w * acc[q][u];
        *p = v;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");  // the next expert's lanes read what these wrote
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  for (int i = tid; i < a.T * 16; i += kDnWaves * 64) {
    float s = 0;
#pragma unroll
    for (int w = 0; w < kDnWaves; ++w) s += table[w * a.T * 16 + i];
    const int t = i >> 4, c = c0 + (i & 15);
    if (c < a.H) {
      if constexpr (OUT_F32) static_cast<float *>(a.out)[t * a.ldo + c] = s;
      else reinterpret_cast<__bf16 *>(a.out)[t * a.ldo + c] = (__bf16)s;
    }
  }
}

template <bool F32>
void launch_route(const MxFewArgs &a, hipStream_t stream) {
  const int64_t units = (int64_t)a.T * ((a.H + 127) / 128);
  const unsigned grid = 1 + (unsigned)((units + 63) / 64);
  if (a.E <= 64) k_few_route<2, 32, F32><<<grid, 1024, 0, stream>>>(a);
  else if (a.E <= 128) k_few_route<4, 32, F32><<<grid, 1024, 0, stream>>>(a);
  else if (a.E <= 256) k_few_route<4, 64, F32><<<grid, 1024, 0, stream>>>(a);
  else if (a.E <= 512) k_few_route<8, 64, F32><<<grid, 1024, 0, stream>>>(a);
  else k_few_route<16, 64, F32><<<grid, 1024, 0, stream>>>(a);
}

}  // namespace

size_t mx_few_workspace_bytes(int64_t T, int E, int k, int64_t H, int64_t I) {
  FewWs w;
  return few_ws(nullptr, T, E, k, H, I, w);
}

hipError_t launch_mx_few(const MxFewArgs &a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  if (a.x_is_f32) launch_route<true>(a, stream); else launch_route<false>(a, stream);
  const int most = std::min(a.E, a.T * a.k);  // experts in use
  k_few_gate_up<<<dim3((unsigned)(a.I / 32), (unsigned)most), kGuWaves * 64, 0, stream>>>(a);
  const unsigned lds = (unsigned)(kDnWaves * a.T * 16 * sizeof(float));
  const unsigned grid = (unsigned)((a.H + 15) / 16);
  if (a.out_is_f32) k_few_down<true><<<grid, kDnWaves * 64, lds, stream>>>(a);
  else k_few_down<false><<<grid, kDnWaves * 64, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nv4
