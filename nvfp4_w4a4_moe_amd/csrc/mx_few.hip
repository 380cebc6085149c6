// A whole MXFP4 expert layer for a few tokens (T <= 64, a decode step) in three kernels.
//
// At this size the layer is bound by reading the chosen experts' weights once (0.53 bytes per
// element; 2.5 MB per expert at hidden size 2048 and expert size 768) and, below that, by
// launches and dependent latencies.  So: few launches, weight loads that wait for one table
// look-up only and are all under way at once, and no intermediate but the quantised rows.
//
//   1. k_few_route    routes the tokens (topk_device.h), a few per workgroup, and quantises x.
//   2. k_few_gate_up  one workgroup per (expert in use, 32 columns of I): gate and up products
//                     for all the expert's tokens, SwiGLU and re-quantisation: 32 columns are
//                     one MX block.  The K dimension is split over the four waves.  Each
//                     workgroup finds its expert's rows itself from the T * k ids (a 64-bit
//                     token mask gives their order without sorting); one more workgroup lists
//                     all experts' rows for the next kernel meanwhile.
//   3. k_few_down     one workgroup per 16 columns of H: its waves walk over the experts, add
//                     weight * product into a token table in LDS (one per wave), and the tables
//                     are summed in wave order.  No atomics on sums: the result is
//                     deterministic.
// With at most 16 assignments (T * k) and no fewer experts nothing is grouped: every assignment
// is taken as an expert with one row.
//
// Products: v_mfma_scale_f32_16x16x128_f8f6f4 with weight rows as the first operand and up to
// 16 of the expert's tokens as the second, straight from global memory: lane (row, g) holds
// the 16-byte block g of the row's 128-element step, so one load of a wave covers 16 rows x 64
// bytes.  Loads are buffer loads, whose offsets behind the row's end or without a row give
// zeros without a branch.
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
constexpr int kMaxR = kMaxT * 32;
constexpr int kDirect = 16;    // up to this many assignments are taken one by one
constexpr uint32_t kOut = 0xFFFFFF00u;  // a byte offset behind every buffer

// Workspace: per assignment f = t * k + j the expert (or -1) and its weight; the experts in use
// with the start of their rows, and the rows' assignments; the quantised x and SwiGLU rows.
struct FewWs {
  int32_t *id;
  float *w;
  int32_t *n_active, *act_e, *act_row, *row_f;
  uint8_t *x_codes, *x_scales, *h_codes, *h_scales;
};
__host__ __device__ inline size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
__host__ __device__ inline int sc_stride(int64_t K) { return (int)((K / 32 + 3) / 4 * 4); }
__host__ __device__ inline size_t few_ws(void *base, int64_t T, int E, int k, int64_t H, int64_t I, FewWs &w) {
  const int64_t R = T * k, A = E < R ? E : R;
  char *p = static_cast<char *>(base);
  size_t at = 0;
  const auto take = [&](size_t b) {
    char *q = p + at;
    at += up256(b);
    return q;
  };
  w.id = reinterpret_cast<int32_t *>(take(R * 4));
  w.w = reinterpret_cast<float *>(take(R * 4));
  w.n_active = reinterpret_cast<int32_t *>(take(4));
  w.act_e = reinterpret_cast<int32_t *>(take(A * 4));
  w.act_row = reinterpret_cast<int32_t *>(take((A + 1) * 4));
  w.row_f = reinterpret_cast<int32_t *>(take(R * 4));
  w.x_codes = reinterpret_cast<uint8_t *>(take(T * (H / 2)));
  w.x_scales = reinterpret_cast<uint8_t *>(take(T * sc_stride(H)));
  w.h_codes = reinterpret_cast<uint8_t *>(take(R * (I / 2)));
  w.h_scales = reinterpret_cast<uint8_t *>(take(R * sc_stride(I)));
  return at;
}

__host__ __device__ inline bool few_direct(const MxFewArgs &a) {
  return a.T * a.k <= kDirect && a.T * a.k <= a.E;
}

// ---------------------------------------------------------------- 1. routing, x

// NPL, LPT: topk_token's.  The first `nroute` workgroups route, the others quantise 16 units of
// x each.
template <int NPL, int LPT, bool F32>
__global__ __launch_bounds__(256) void k_few_route(MxFewArgs a, int nroute) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if ((int)blockIdx.x >= nroute) {
    const int l16 = lane & 15, spr = (a.H + 127) / 128;
    const int unit = (blockIdx.x - nroute) * 16 + (tid >> 4);
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
      if (l16 == 0) *reinterpret_cast<uint32_t *>(ws.x_scales + row * sc_stride(a.H) + seg * 4) = d;
    }
    if (bad && a.dev_status) atomicOr(a.dev_status, kDsNonFinite);
    return;
  }
  if (a.logits) {
    constexpr int TPW = kWave / LPT;
    const int sub = lane / LPT, ll = lane % LPT;
    const int t0 = (blockIdx.x * 4 + wave) * TPW;
    if (t0 >= a.T) return;  // uniform over the wave
    const int t = t0 + sub;
    const bool valid = t < a.T;
    int id;
    float w;
    const bool nan = topk_token<NPL, LPT>(a.logits + (int64_t)t * a.E, valid, a.E, a.k, a.flags, lane, sub, ll, id, w);
    if (valid && ll < a.k) {
      const int f = t * a.k + ll;
      ws.id[f] = id < a.E ? id : -1;  // every remaining logit was NaN: no expert
      ws.w[f] = w;
      if (a.topk_ids) a.topk_ids[f] = id;
      if (a.topk_w) a.topk_w[f] = w;
    }
    if (nan && lane == 0 && a.dev_status) atomicOr(a.dev_status, kDsNanLogit);
    return;
  }
  // the caller's ids may repeat within a token: the first takes the sum of the weights, in order
  const int R = a.T * a.k;
  for (int f = blockIdx.x * 256 + tid; f < R; f += nroute * 256) {
    const int f0 = f / a.k * a.k, id = a.topk_ids[f];
    const bool good = id >= 0 && id < a.E;
    bool first = true;
    float w = 0.0f;
    for (int j = f0; j < f0 + a.k; ++j) {
      if (a.topk_ids[j] != id) continue;
      if (j < f) first = false;
      w += a.topk_w[j];
    }
    ws.id[f] = good && first ? id : -1;
    ws.w[f] = w;
    if (!good && a.dev_status) atomicOr(a.dev_status, kDsBadExpert);
  }
}

// ---------------------------------------------------------------- products

// (device-only helpers: the buffer-resource type exists only on the GPU target)
__device__ __forceinline__ int4 load16(const void *base, uint32_t bytes, uint32_t off) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000), off, 0, 0);
  return make_int4((int)v[0], (int)v[1], (int)v[2], (int)v[3]);
}
__device__ __forceinline__ uint32_t load1(const void *base, uint32_t bytes, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b8(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000), off, 0, 0);
}
__device__ __forceinline__ const uint8_t *uniform_ptr(const uint8_t *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t *>(((uint64_t)hi << 32) | lo);
}

struct Frag {
  int4 c;      // 32 codes
  uint32_t s;  // their scale byte
};
// One matrix (or one expert's part of it): K = 32 nb
struct Mat {
  const uint8_t *codes, *scales;
  uint32_t cbytes, sbytes;
  int nb, sld;
};
__device__ __forceinline__ Mat matrix(const uint8_t *codes, const uint8_t *scales, int64_t row0, uint32_t rows, int K) {
  const int nb = K / 32, sld = sc_stride(K);
  return Mat{uniform_ptr(codes + row0 * (nb * 16)), uniform_ptr(scales + row0 * sld), rows * (uint32_t)(nb * 16),
             rows * (uint32_t)sld, nb, sld};
}
// block b of a row (row < 0: none); zeros behind K
__device__ __forceinline__ Frag load_frag(const Mat &m, int row, int b) {
  const bool live = row >= 0 && b < m.nb;
  return Frag{load16(m.codes, m.cbytes, live ? (uint32_t)(row * m.nb + b) * 16u : kOut),
              load1(m.scales, m.sbytes, live ? (uint32_t)(row * m.sld + b) : kOut)};
}
__device__ __forceinline__ f32x4 mfma16(const Frag &a, const Frag &b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(i32x8{a.c.x, a.c.y, a.c.z, a.c.w, 0, 0, 0, 0},
                                                          i32x8{b.c.x, b.c.y, b.c.z, b.c.w, 0, 0, 0, 0}, c, 4, 4, 0,
                                                          (int)a.s, 0, (int)b.s);
}

// ---------------------------------------------------------------- 2. gate and up

constexpr int kGuWaves = 4, kGuSteps = 4;  // steps of K = 128 a wave holds at a time

// The experts in use, the starts of their rows and the rows' assignments, for k_few_down.
__device__ void list_experts(const MxFewArgs &a, const FewWs &ws, unsigned long long *mask, int *start, int *wsum) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, R = a.T * a.k;
  for (int e = tid; e < kMaxE; e += 256) mask[e] = 0ull;
  __syncthreads();
  for (int f = tid; f < R; f += 256)
    if (ws.id[f] >= 0) atomicOr(&mask[ws.id[f]], 1ull << (f / a.k));
  __syncthreads();
  // exclusive prefix over the experts of (in use, rows), packed: both stay below 2^16
  int own[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = __popcll(mask[tid * 4 + i]);
    own[i] = n | (n ? 1 << 16 : 0);
    sum += own[i];
  }
  int s = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(s, o, 64);
    if (lane >= o) s += x;
  }
  if (lane == 63) wsum[wave] = s;
  __syncthreads();
  for (int w = 0; w < wave; ++w) s += wsum[w];
  int ex = s - sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    start[tid * 4 + i] = ex & 0xFFFF;
    if (own[i]) {
      ws.act_e[ex >> 16] = tid * 4 + i;
      ws.act_row[ex >> 16] = ex & 0xFFFF;
    }
    ex += own[i];
  }
  if (tid == 255) {
    *ws.n_active = ex >> 16;
    ws.act_row[ex >> 16] = ex & 0xFFFF;
  }
  __syncthreads();
  for (int f = tid; f < R; f += 256) {
    const int id = ws.id[f];
    if (id >= 0) ws.row_f[start[id] + __popcll(mask[id] & ((1ull << (f / a.k)) - 1ull))] = f;
  }
}

__global__ __launch_bounds__(kGuWaves * 64) void k_few_gate_up(MxFewArgs a) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  __shared__ union {
    float part[kGuWaves][16][64];
    struct {
      unsigned long long mask[kMaxE];
      int start[kMaxE];
    } list;
  } sh;
  __shared__ unsigned long long smask;
  __shared__ int rows[kMaxT];
  __shared__ int wsum[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int R = a.T * a.k;
  const bool direct = few_direct(a);
  if (blockIdx.x == 0) {
    if (!direct) list_experts(a, ws, sh.list.mask, sh.list.start, wsum);
    return;
  }
  const int tiles = a.I / 32;
  const int y = (int)(blockIdx.x - 1) / tiles, c0 = ((int)(blockIdx.x - 1) - y * tiles) * 32;
  // y counts assignments or, when there are fewer of them, experts
  const bool by_f = R <= a.E;
  const int e = by_f ? __builtin_amdgcn_readfirstlane(ws.id[y]) : y;
  if (e < 0) return;
  int n = 1;
  if (direct) {
    if (tid == 0) rows[0] = y;
  } else {
    if (tid == 0) smask = 0ull;
    int mine[kMaxR / 256];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxR / 256; ++i) {
      const int f = tid + i * 256;
      mine[i] = f < R && ws.id[f] == e ? f / a.k : -1;
    }
#pragma unroll
    for (int i = 0; i < kMaxR / 256; ++i)
      if (mine[i] >= 0) atomicOr(&smask, 1ull << mine[i]);
    __syncthreads();
    const unsigned long long m = smask;
    // nobody's expert, or an earlier assignment's workgroup has it
    if (m == 0ull || (by_f && y / a.k != __builtin_ctzll(m))) return;
#pragma unroll
    for (int i = 0; i < kMaxR / 256; ++i)
      if (mine[i] >= 0) rows[__popcll(m & ((1ull << mine[i]) - 1ull))] = tid + i * 256;
    n = __builtin_amdgcn_readfirstlane(__popcll(m));
  }
  const int l = lane & 15, g = lane >> 4;
  const Mat w13 = matrix(a.w13_codes, a.w13_scales, (int64_t)e * 2 * a.I, 2 * a.I, a.H);
  const Mat x = matrix(ws.x_codes, ws.x_scales, 0, a.T, a.H);
  const int steps = (a.H + 127) / 128;
  const int per = min(kGuSteps, (steps + kGuWaves - 1) / kGuWaves);  // consecutive steps of a wave
  const int chunk = per * kGuWaves;
  // tiles: gate columns c0.., c0 + 16.., then the up rows
  Frag w[kGuSteps][4];
  const auto load_w = [&](int s0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kGuSteps; ++i)
#pragma unroll
      for (int t = 0; t < 4; ++t)
        w[i][t] = load_frag(w13, i < per ? c0 + (t & 1) * 16 + (t >> 1) * a.I + l : -1, (s0 + i) * 4 + g);
  };
  load_w(wave * per);
  __syncthreads();  // the row list
  const int slot = tid >> 4, cc = (tid & 15) * 2;
  const int hsld = sc_stride(a.I);
  bool bad = false;
  for (int q = 0; q < n; q += 16) {
    const int tok = q + l < n ? rows[q + l] / a.k : -1;
    f32x4 acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = f32x4{0, 0, 0, 0};
    for (int c = 0; c < steps; c += chunk) {
      if (c > 0 || (q > 0 && steps > chunk)) load_w(c + wave * per);  // otherwise the registers hold it
      Frag xf[kGuSteps];
#pragma unroll
      for (int i = 0; i < kGuSteps; ++i) xf[i] = load_frag(x, i < per ? tok : -1, (c + wave * per + i) * 4 + g);
#pragma unroll
      for (int i = 0; i < kGuSteps; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[t] = mfma16(w[i][t], xf[i], acc[t]);
    }
    // sum over the waves, SwiGLU, re-quantise: thread = token slot of 16, two columns
    if (q) __syncthreads();
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) sh.part[wave][t * 4 + r][lane] = acc[t][r];
    __syncthreads();
    // column c sits in tile c / 16, lane (c % 16) / 4 * 16 + slot, register c % 4
    float h[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = cc + u, reg = (c >> 4) * 4 + (c & 3), at = ((c & 15) >> 2) * 16 + slot;
      float gate = 0, up = 0;
#pragma unroll
      for (int v = 0; v < kGuWaves; ++v) {
        gate += sh.part[v][reg][at];
        up += sh.part[v][reg + 8][at];
      }
      h[u] = gate * __builtin_amdgcn_rcpf(1.0f + __expf(-gate)) * up;
    }
    uint32_t m = max(__float_as_uint(h[0]) & 0x7FFFFFFFu, __float_as_uint(h[1]) & 0x7FFFFFFFu);
    m = oct_umax(m);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, false));  // row_mirror
    const uint32_t byte = mx_scale_byte(m, a.ceil_rule);
    uint32_t c = mx_pack_f32<0>(0u, h[0], h[1], mx_scale_value(byte));
    if (byte == kMxNan) c = 0u;
    if (q + slot < n) {
      bad |= byte == kMxNan;
      const int64_t r = rows[q + slot];
      ws.h_codes[r * (a.I / 2) + (c0 + cc) / 2] = (uint8_t)c;
      if ((tid & 15) == 0) ws.h_scales[r * hsld + c0 / 32] = (uint8_t)byte;
    }
  }
  if (bad && a.dev_status) atomicOr(a.dev_status, kDsNonFinite);
}

// ---------------------------------------------------------------- 3. down

constexpr int kDnWaves = 16, kDnSteps = 6;

// A wave's share: entries (experts in use, or assignments) wave / parts, + 16 / parts, ..; of
// each the steps part, part + parts, ..  (parts > 1 with fewer than 16 entries).  The weights of
// the next entry are loaded while this one is computed.
template <bool OUT_F32>
__global__ __launch_bounds__(kDnWaves * 64) void k_few_down(MxFewArgs a) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  extern __shared__ float table[];  // [wave][token][16 columns]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane & 15, g = lane >> 4;
  const int R = a.T * a.k;
  const bool direct = few_direct(a);
  const int na = direct ? R : __builtin_amdgcn_readfirstlane(*ws.n_active);
  const int parts = na > 8 ? 1 : na > 4 ? 2 : 4;
  const int part = wave % parts, stride = kDnWaves / parts;
  const int steps = (a.I + 127) / 128;
  const int c0 = blockIdx.x * 16;
  const int wrow = c0 + l < a.H ? c0 + l : -1;
  const Mat h = matrix(ws.h_codes, ws.h_scales, 0, R, a.I);
  float *mine = table + wave * a.T * 16;
  struct Entry {
    int e, r0, n;
  };
  const auto entry = [&](int i) __attribute__((always_inline)) {
    Entry n{-1, 0, 0};
    if (i < na) {
      if (direct) {
        n = Entry{ws.id[i], i, 1};
      } else {
        n.e = ws.act_e[i];
        n.r0 = ws.act_row[i];
        n.n = ws.act_row[i + 1] - n.r0;
      }
    }
    n.e = __builtin_amdgcn_readfirstlane(n.e);
    n.r0 = __builtin_amdgcn_readfirstlane(n.r0);
    n.n = __builtin_amdgcn_readfirstlane(n.e < 0 ? 0 : n.n);
    return n;
  };
  Frag w[kDnSteps];
  const auto load_w = [&](const Entry &n, int s0) __attribute__((always_inline)) {
    const Mat w2 = matrix(a.w2_codes, a.w2_scales, (int64_t)max(n.e, 0) * a.H, a.H, a.I);
#pragma unroll
    for (int s = 0; s < kDnSteps; ++s) w[s] = load_frag(w2, n.e < 0 ? -1 : wrow, (s0 + s * parts) * 4 + g);
  };
  Entry cur = entry(wave / parts);
  load_w(cur, part);
  for (int i = lane; i < a.T * 4; i += 64) reinterpret_cast<f32x4 *>(mine)[i] = f32x4{0, 0, 0, 0};
  for (int i = wave / parts; i < na; i += stride) {
    const Entry next = entry(i + stride);
    const bool once = steps <= parts * kDnSteps;  // the registers hold the whole row
    for (int q = 0; q < cur.n; q += 16) {
      const int f = q + l < cur.n ? (direct ? cur.r0 : ws.row_f[cur.r0 + q + l]) : -1;
      const float wt = f >= 0 ? ws.w[f] : 0.0f;
      f32x4 acc = f32x4{0, 0, 0, 0};
      for (int s0 = part; s0 < steps; s0 += parts * kDnSteps) {
        if (!once && (s0 != part || q > 0)) load_w(cur, s0);
        Frag x[kDnSteps];
#pragma unroll
        for (int s = 0; s < kDnSteps; ++s) x[s] = load_frag(h, f, (s0 + s * parts) * 4 + g);
#pragma unroll
        for (int s = 0; s < kDnSteps; ++s) acc = mfma16(w[s], x[s], acc);
      }
      // lane = row slot l, columns 4 g ..: an expert's rows are different tokens, so no two
      // lanes meet in the table
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (f >= 0) {
        f32x4 *p = reinterpret_cast<f32x4 *>(mine + f / a.k * 16 + g * 4);
        f32x4 v = *p;
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] += wt * acc[u];
        *p = v;
      }
    }
    load_w(next, part);
    cur = next;
  }
  __syncthreads();
  for (int i = tid; i < a.T * 16; i += kDnWaves * 64) {
    float s = 0;
#pragma unroll
    for (int v = 0; v < kDnWaves; ++v) s += table[v * a.T * 16 + i];
    const int t = i >> 4, c = c0 + (i & 15);
    if (c < a.H) {
      if constexpr (OUT_F32) static_cast<float *>(a.out)[t * a.ldo + c] = s;
      else reinterpret_cast<__bf16 *>(a.out)[t * a.ldo + c] = (__bf16)s;
    }
  }
}

template <int NPL, int LPT, bool F32>
void launch_route(const MxFewArgs &a, hipStream_t stream) {
  const int per = 4 * (kWave / LPT);  // tokens per routing workgroup
  const int nroute = a.logits ? (a.T + per - 1) / per : (a.T * a.k + 255) / 256;
  const int units = a.T * ((a.H + 127) / 128);
  k_few_route<NPL, LPT, F32><<<(unsigned)(nroute + (units + 15) / 16), 256, 0, stream>>>(a, nroute);
}
template <bool F32>
void launch_route(const MxFewArgs &a, hipStream_t stream) {
  if (a.E <= 64) launch_route<2, 32, F32>(a, stream);
  else if (a.E <= 128) launch_route<4, 32, F32>(a, stream);
  else if (a.E <= 256) launch_route<4, 64, F32>(a, stream);
  else if (a.E <= 512) launch_route<8, 64, F32>(a, stream);
  else launch_route<16, 64, F32>(a, stream);
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
  k_few_gate_up<<<1 + (unsigned)(a.I / 32) * (unsigned)most, kGuWaves * 64, 0, stream>>>(a);
  const unsigned lds = (unsigned)(kDnWaves * a.T * 16 * sizeof(float));
  const unsigned grid = (unsigned)((a.H + 15) / 16);
  if (a.out_is_f32) k_few_down<true><<<grid, kDnWaves * 64, lds, stream>>>(a);
  else k_few_down<false><<<grid, kDnWaves * 64, lds, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nv4
