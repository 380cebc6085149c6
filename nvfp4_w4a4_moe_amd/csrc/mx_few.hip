// A whole MXFP4 expert layer for a few tokens (T <= 64, a decode step) in two to four kernels.
//
// At this size the layer is bound by reading the chosen experts' weights once (0.53 bytes per
// element; 2.5 MB per expert at hidden size 2048 and expert size 768) and, below that, by
// launches and dependent latencies.  So: few launches, weight loads that wait for one table
// look-up only and are all under way at once, and no intermediate but the quantised rows.
//
//   1. k_few_route    routes the tokens (topk_device.h), a few per workgroup, and quantises x.
//                     Left out for one or two tokens (few_fused): there every workgroup of the
//                     next kernel routes and quantises for itself, in LDS (one token 19.3 -> 16.8
//                     us; at seven the repeated work costs 8 us more than the launch).
//   2. k_few_gate_up  one workgroup per (expert in use, 32 columns of I): gate and up products
//                     for all the expert's tokens, SwiGLU and re-quantisation: 32 columns are
//                     one MX block.  The K dimension is split over the eight waves.  Every wave
//                     finds its expert's rows itself from the T * k ids (ballots, no sorting).
//      With more assignments (few_grouped) k_few_group and the grouped GEMM (mx_gemm_kernel.h) take
//                     its place: the first lists the experts in use and their rows.
//   3. k_few_down     one workgroup per 16 columns of H: its waves walk over the assignments
//                     (few_grouped: the experts in use), add weight * product into a token table
//                     in LDS (one per wave), and the tables are summed in wave order.  Where there
//                     are few columns, several workgroups share a tile.  No atomics on sums: the
//                     result is deterministic.
// An assignment (token t, choice j) is numbered f = j * T + t.
//
// Products: v_mfma_scale_f32_16x16x128_f8f6f4 with weight rows as the first operand and up to
// 16 of the expert's tokens as the second: lane (row, g) holds the 16-byte block g of the row's
// 128-element step.  Tokens' rows come straight from global memory in that layout, through buffer
// loads, whose offsets behind the row's end or without a row give zeros without a branch.
// Weights pass through LDS: loaded in that layout 16 adjacent lanes ask for 16 rows, and a load
// costs the address unit 64 accesses instead of 16 (one token 16.4 -> 14.0 us, seven 41 -> 38, 64 of
// them 82 -> 78).  They are streamed (non-temporal) past the caches, where the other operands
// stay: eight layers in turn, as a decode step reads them, take 42.1 us each for seven tokens
// against 44.6; 64 tokens again and again 70 against 78, seven 39.9 against 38.2.
//
// Measured at H 2048, I 768, 8 of 128 experts a token, even routing, weights from memory: one token
// 14.9 us, seven 42 (2.8 TB/s), 64 tokens 74 us (4.2 TB/s, nearly every expert's weights).
#include <algorithm>
#include <type_traits>

#include "mx_device.h"
#include "mx_internal.h"
#include "mx_rows.h"
#include "nv4_internal.h"
#include "topk_device.h"
#include "../../include/nv4moe.h"

namespace nv4 {
namespace {

constexpr int kMaxT = 64;      // tokens (one bit each in an expert's mask)
constexpr int kMaxE = 1024;
constexpr int kMaxSplits = 4;  // workgroups that share a column tile of the down product
constexpr uint32_t kOut = 0xFFFFFF00u;  // a byte offset behind every buffer

// Workspace: per assignment f = j * T + t the expert (or -1) and its weight; the experts in use
// with the start of their rows, and the rows' tokens and weights (few_grouped); the down product's
// partial sums; the quantised x and SwiGLU rows.
struct FewWs {
  int32_t *id;
  float *w;
  int32_t *n_active, *act_e, *act_row;
  int32_t *offsets, *row_token;  // every expert's first row, the rows' tokens and weights
  float *row_w;
  int32_t *arrived;  // per column tile of the down product: workgroups that left their sums
  float *sums;       // [tile][split][token][16]
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
  w.row_w = reinterpret_cast<float *>(take(R * 4));
  w.offsets = reinterpret_cast<int32_t *>(take((E + 1) * 4));
  w.row_token = reinterpret_cast<int32_t *>(take(R * 4));
  const int64_t tiles = (H + 15) / 16;
  w.arrived = reinterpret_cast<int32_t *>(take(tiles * 4));
  w.sums = reinterpret_cast<float *>(take(tiles * kMaxSplits * T * 16 * 4));
  w.x_codes = reinterpret_cast<uint8_t *>(take(T * (H / 2)));
  w.x_scales = reinterpret_cast<uint8_t *>(take(T * sc_stride(H)));
  w.h_codes = reinterpret_cast<uint8_t *>(take(R * (I / 2)));
  w.h_scales = reinterpret_cast<uint8_t *>(take(R * sc_stride(I)));
  return at;
}

// token of an assignment: f mod T (f + 0.5 keeps the quotient away from an integer)
__device__ __forceinline__ int few_token(int f, int T) {
  return f - (int)(((float)f + 0.5f) * __builtin_amdgcn_rcpf((float)T)) * T;
}

// ---------------------------------------------------------------- 1. routing, x

// NPL, LPT: topk_token's.  The first `nroute` workgroups route, the others quantise 16 units of
// x each.
template <int NPL, int LPT, bool F32>
__global__ __launch_bounds__(256) void k_few_route(MxFewArgs a, int nroute) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (blockIdx.x == gridDim.x - 1)
    for (int i = tid; i < (a.H + 15) / 16; i += 256) ws.arrived[i] = 0;
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
      const int f = ll * a.T + t;
      ws.id[f] = id < a.E ? id : -1;  // every remaining logit was NaN: no expert
      ws.w[f] = w;
      if (a.topk_ids) a.topk_ids[t * a.k + ll] = id;
      if (a.topk_w) a.topk_w[t * a.k + ll] = w;
    }
    if (nan && lane == 0 && a.dev_status) atomicOr(a.dev_status, kDsNanLogit);
    return;
  }
  // the caller's ids may repeat within a token: the first takes the sum of the weights, in order
  const int R = a.T * a.k;
  for (int i = blockIdx.x * 256 + tid; i < R; i += nroute * 256) {
    const int t = i / a.k, j0 = i - t * a.k, id = a.topk_ids[i];
    const bool good = id >= 0 && id < a.E;
    bool first = true;
    float w = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      if (a.topk_ids[t * a.k + j] != id) continue;
      if (j < j0) first = false;
      w += a.topk_w[t * a.k + j];
    }
    ws.id[j0 * a.T + t] = good && first ? id : -1;
    ws.w[j0 * a.T + t] = w;
    if (!good && a.dev_status) atomicOr(a.dev_status, kDsBadExpert);
  }
}

// ---------------------------------------------------------------- products

// (device-only helpers: the buffer-resource type exists only on the GPU target)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u32x4 load16(const void *base, uint32_t bytes, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000), off, 0, 0);
}
__device__ __forceinline__ u32x2 load8(const void *base, uint32_t bytes, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b64(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000), off, 0, 0);
}
__device__ __forceinline__ const uint8_t *uniform_ptr(const uint8_t *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return reinterpret_cast<const uint8_t *>(((uint64_t)hi << 32) | lo);
}

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
// Block b of a row (row < 0: none): its 32 codes; zeros behind K.
__device__ __forceinline__ u32x4 load_codes(const Mat &m, int row, int b) {
  return load16(m.codes, m.cbytes, ((row >= 0) & (b < m.nb)) ? (uint32_t)(row * m.nb + b) * 16u : kOut);
}
// The scale bytes of two consecutive steps (8 blocks from block b0, a multiple of 4) of a row:
// dword i holds step i's four blocks, of which lane group g takes byte g (and b0 + 4 i + g < nb).
__device__ __forceinline__ u32x2 load_scales2(const Mat &m, int row, int b0) {
  return load8(m.scales, m.sbytes, row >= 0 && b0 < m.nb ? (uint32_t)(row * m.sld + b0) : kOut);
}
__device__ __forceinline__ uint32_t scale_of(uint32_t dword, int g, int b, int nb) {
  return b < nb ? dword >> (8 * g) : 0u;
}
__device__ __forceinline__ i32x8 operand(u32x4 v) {  // FP4 reads the first four of eight dwords
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}
__device__ __forceinline__ f32x4 mfma16(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(a), operand(b), c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// ---------------------------------------------------------------- 2. gate and up

constexpr int kGuWaves = 8, kGuSteps = 2;  // steps of K = 128 a wave holds at a time
constexpr int kGuThreads = kGuWaves * 64;
constexpr int kGuCodes = 64 * kGuSteps * 64, kGuSlot = kGuCodes + 64 * kGuSteps * 4;

constexpr int kMostRows = 128;  // assignments without few_grouped
constexpr int kIdChunks = kMostRows / 64;
constexpr int kFusedElems = 8192;                // tokens x H that a workgroup quantises for itself
constexpr int kFusedTokens = 2;

struct FewList {
  unsigned long long mask[kMaxE];
  int start[kMaxE];
  int wsum[4];
};
// few_grouped: the experts in use, all experts' first rows, the rows' assignments and tokens, for the
// grouped GEMM that takes k_few_gate_up's place and for k_few_down.
__global__ __launch_bounds__(kGuThreads) void k_few_group(MxFewArgs a) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  __shared__ FewList sh;
  const int *id = ws.id;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, R = a.T * a.k;
  for (int e = tid; e < kMaxE; e += kGuThreads) sh.mask[e] = 0ull;
  __syncthreads();
  for (int f = tid; f < R; f += kGuThreads)
    if (id[f] >= 0) atomicOr(&sh.mask[id[f]], 1ull << few_token(f, a.T));
  __syncthreads();
  // exclusive prefix over the experts of (in use, rows), packed (both stay below 2^16): four
  // experts for each of the first 256 threads
  const bool mine = tid < kMaxE / 4;
  int own[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = mine ? __popcll(sh.mask[tid * 4 + i]) : 0;
    own[i] = n | (n ? 1 << 16 : 0);
    sum += own[i];
  }
  int s = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(s, o, 64);
    if (lane >= o) s += x;
  }
  if (lane == 63 && mine) sh.wsum[wave] = s;
  __syncthreads();
  for (int w = 0; w < std::min(wave, 4); ++w) s += sh.wsum[w];
  int ex = s - sum;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (mine) sh.start[tid * 4 + i] = ex & 0xFFFF;
    if (mine && tid * 4 + i <= a.E) ws.offsets[tid * 4 + i] = ex & 0xFFFF;
    if (own[i]) {
      ws.act_e[ex >> 16] = tid * 4 + i;
      ws.act_row[ex >> 16] = ex & 0xFFFF;
    }
    ex += own[i];
  }
  if (tid == kMaxE / 4 - 1) {
    *ws.n_active = ex >> 16;
    if (a.E == kMaxE) ws.offsets[kMaxE] = ex & 0xFFFF;
    ws.act_row[ex >> 16] = ex & 0xFFFF;
  }
  __syncthreads();
  for (int f = tid; f < R; f += kGuThreads) {
    const int e = id[f];
    if (e < 0) continue;
    const int t = few_token(f, a.T), r = sh.start[e] + __popcll(sh.mask[e] & ((1ull << t) - 1ull));
    ws.row_w[r] = ws.w[f];
    ws.row_token[r] = t;
  }
}

// FUSED (few_fused): routes and quantises x as well;
// NPL, LPT as for topk_token, F32 the type of x.
template <bool FUSED, int NPL, int LPT, bool F32>
__global__ __launch_bounds__(kGuThreads) void k_few_gate_up(MxFewArgs a) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  // a wave's part of W13: 64 rows of kGuSteps steps, and their scale bytes; afterwards its sums
  __shared__ __attribute__((aligned(1024))) uint8_t slots[kGuWaves * kGuSlot];
  const auto part = [&](int v, int reg) __attribute__((always_inline)) {
    return reinterpret_cast<float *>(slots + v * kGuSlot) + reg * 64;
  };
  __shared__ int rows[kGuWaves][kMaxT];  // one list per wave: no barrier between finding and using it
  __shared__ int s_id[FUSED ? kFusedTokens * 32 : 1];
  __shared__ float s_w[FUSED ? kFusedTokens * 32 : 1];
  __shared__ __attribute__((aligned(16))) uint8_t s_xc[FUSED ? kFusedElems / 2 : 16];
  __shared__ uint32_t s_xs[FUSED ? kFusedElems / 32 : 1];  // (a row of H = 32 has a whole dword)
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int R = a.T * a.k;
  const int steps = (a.H + 127) / 128;
  const int *id = ws.id;
  if constexpr (FUSED) {
    // the first waves route, the others quantise meanwhile
    constexpr int TPW = kWave / LPT;
    const int l16 = lane & 15, units = a.T * steps, nroute = (a.T + TPW - 1) / TPW;
    for (int u0 = (wave - nroute) * 4; u0 < units && wave >= nroute; u0 += (kGuWaves - nroute) * 4) {
      const int u = u0 + (lane >> 4), row = u / steps, seg = u - row * steps, col = seg * 128 + l16 * 8;
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
        if (col < a.H) *reinterpret_cast<uint32_t *>(s_xc + row * (a.H / 2) + col / 2) = c;
        if (l16 == 0) s_xs[u] = d;
      }
      if (bad && a.dev_status && blockIdx.x == 0) atomicOr(a.dev_status, kDsNonFinite);
    }
    if (wave < nroute) {
      const int sub = lane / LPT, ll = lane % LPT;
      const int t = wave * TPW + sub;
      const bool valid = t < a.T;
      int e;
      float w;
      const bool nan = topk_token<NPL, LPT>(a.logits + (int64_t)t * a.E, valid, a.E, a.k, a.flags, lane, sub, ll, e, w);
      if (valid && ll < a.k) {
        s_id[ll * a.T + t] = e < a.E ? e : -1;
        s_w[ll * a.T + t] = w;
        if (blockIdx.x == 0) {
          if (a.topk_ids) a.topk_ids[t * a.k + ll] = e;
          if (a.topk_w) a.topk_w[t * a.k + ll] = w;
        }
      }
      if (nan && lane == 0 && a.dev_status && blockIdx.x == 0) atomicOr(a.dev_status, kDsNanLogit);
    }
    __syncthreads();
    id = s_id;
  }
  if (FUSED && blockIdx.x == 0) {
    for (int f = tid; f < R; f += kGuThreads) {
      ws.id[f] = s_id[f];
      ws.w[f] = s_w[f];
    }
    for (int i = tid; i < (a.H + 15) / 16; i += kGuThreads) ws.arrived[i] = 0;
  }
  const int tiles = a.I / 32;
  const int y = (int)blockIdx.x / tiles, c0 = ((int)blockIdx.x - y * tiles) * 32;
  // y counts assignments or, when there are fewer of them, experts
  const bool by_f = R <= a.E;
  const int e = by_f ? __builtin_amdgcn_readfirstlane(id[y]) : y;
  if (e < 0) return;
  int n = 0, owner = -1;
  int ids[kIdChunks];  // all under way at once
#pragma unroll
  for (int c = 0; c < kIdChunks; ++c) ids[c] = id[std::min(c * 64 + lane, R - 1)];
#pragma unroll
  for (int c = 0; c < kIdChunks; ++c) {
    const int f = c * 64 + lane;
    const bool hit = f < R && ids[c] == e;
    const unsigned long long m = __ballot(hit);
    if (hit) rows[wave][n + __popcll(m & ((1ull << lane) - 1ull))] = f;
    if (m && owner < 0) owner = c * 64 + __builtin_ctzll(m);
    n += __popcll(m);
  }
  n = __builtin_amdgcn_readfirstlane(n);
  // nobody's expert, or an earlier assignment's workgroup has it
  if (n == 0 || (by_f && owner != y)) return;
  const int l = lane & 15, g = lane >> 4;
  const Mat w13 = matrix(a.w13_codes, a.w13_scales, (int64_t)e * 2 * a.I, 2 * a.I, a.H);
  const Mat x = matrix(ws.x_codes, ws.x_scales, 0, a.T, a.H);
  const int per = min(kGuSteps, (steps + kGuWaves - 1) / kGuWaves);  // consecutive steps of a wave
  const int chunk = per * kGuWaves;
  static_assert(kGuSteps == 2, "128 bytes of codes and two dwords of scale bytes a row");
  // LDS position 16 p of the codes (p = 64 i + lane) holds block (p % 8) ^ (row / 2 % 8) of row p / 8:
  // the 16 rows of one read then lie in different banks
  uint8_t *mine = slots + wave * kGuSlot;
  const auto load_w = [&](int s0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kGuCodes / 1024; ++i) {
      const int r = i * 8 + (lane >> 3), b = (lane & 7) ^ ((r >> 1) & 7);
      const int row = c0 + (r & 31) + (r >> 5) * a.I;
      const bool in = (b < per * 4) & (s0 * 4 + b < w13.nb);
      mx_dma16<true>(w13.codes, w13.cbytes, mine + i * 1024, in ? (uint32_t)(row * w13.nb + s0 * 4 + b) * 16u : kOut);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = j * 32 + (lane >> 1), d = lane & 1;
      const int row = c0 + (r & 31) + (r >> 5) * a.I;
      const bool in = (d < per) & (s0 + d < steps);
      mx_dma4(w13.scales, w13.sbytes, mine + kGuCodes + j * 256, in ? (uint32_t)(row * w13.sld + (s0 + d) * 4) : kOut);
    }
  };
  load_w(wave * per);
  const int slot = tid >> 4, cc = (tid & 15) * 2;
  const int hsld = sc_stride(a.I);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  for (int q = 0; q < n; q += 16) {
    if (q) {
      __syncthreads();  // the sums of the rows before have been read
      load_w(wave * per);
    }
    const int tok = q + l < n ? few_token(rows[wave][q + l], a.T) : -1;
    f32x4 acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = f32x4{0, 0, 0, 0};
    for (int c = 0; c < steps; c += chunk) {
      const int s0 = c + wave * per;
      if (c > 0) load_w(s0);
      u32x4 xc[kGuSteps];
      uint32_t xs[kGuSteps];
      u32x2 xs2 = {0, 0};
      if constexpr (!FUSED) xs2 = load_scales2(x, tok, s0 * 4);
#pragma unroll
      for (int i = 0; i < kGuSteps; ++i) {
        const int b = (s0 + i) * 4 + g;
        if constexpr (FUSED) {
          const bool live = tok >= 0 && i < per && b < x.nb;
          xc[i] = live ? *reinterpret_cast<const u32x4 *>(s_xc + (tok * x.nb + b) * 16) : u32x4{0, 0, 0, 0};
          xs[i] = live ? s_xs[tok * steps + s0 + i] >> (8 * g) : 0u;
        } else {
          xc[i] = load_codes(x, i < per ? tok : -1, b);
          xs[i] = scale_of(xs2[i], g, i < per ? b : x.nb, x.nb);
        }
      }
      mx_wait_vm<0>();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int r = t * 16 + l;  // gate columns c0.., c0 + 16.., then the up rows
        const u32x2 wsc = *reinterpret_cast<const u32x2 *>(mine + kGuCodes + r * 8);
#pragma unroll
        for (int i = 0; i < kGuSteps; ++i) {
          const int b = (s0 + i) * 4 + g;
          const u32x4 w = *reinterpret_cast<const u32x4 *>(mine + (r * 8 + ((i * 4 + g) ^ ((r >> 1) & 7))) * 16);
          acc[t] = mfma16(w, scale_of(wsc[i], g, i < per ? b : w13.nb, w13.nb), xc[i], xs[i], acc[t]);
        }
      }
      mx_wait_lds();  // the next steps or the sums take the place
    }
    // sum over the waves, SwiGLU, re-quantise: thread = token slot of 16, two columns
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) part(wave, t * 4 + r)[lane] = acc[t][r];
    __syncthreads();
    if (tid < 256) {
      // column c sits in tile c / 16, lane (c % 16) / 4 * 16 + slot, register c % 4
      float h[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = cc + u, reg = (c >> 4) * 4 + (c & 3), at = ((c & 15) >> 2) * 16 + slot;
        float gate = 0, up = 0;
#pragma unroll
        for (int v = 0; v < kGuWaves; ++v) {
          gate += part(v, reg)[at];
          up += part(v, reg + 8)[at];
        }
        // (mx_swiglu's steps, and its error)
        h[u] = gate * __builtin_amdgcn_rcpf(1.0f + __expf(-gate)) * up;
      }
      uint32_t m = max(__float_as_uint(h[0]) & 0x7FFFFFFFu, __float_as_uint(h[1]) & 0x7FFFFFFFu);
      m = oct_umax(m);
      m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x140, 0xF, 0xF, false));  // row_mirror
      const uint32_t byte = mx_scale_byte(m, a.ceil_rule);
      uint32_t c = mx_pack_f32<0>(0u, h[0], h[1], mx_scale_value(byte));
      if (byte == kMxNan) c = 0u;
      if (q + slot < n) {
        const int64_t r = rows[wave][q + slot];
        ws.h_codes[r * (a.I / 2) + (c0 + cc) / 2] = (uint8_t)c;
        if ((tid & 15) == 0) ws.h_scales[r * hsld + c0 / 32] = (uint8_t)byte;
      }
    }
  }
}

// ---------------------------------------------------------------- 3. down

constexpr int kDnWaves = 8, kDnSteps = 6;
constexpr int kDnCodes = 16 * kDnSteps * 64;  // 16 rows of a window of kDnSteps steps
constexpr int kDnSlot = kDnCodes + 512;       // and their scale bytes, kDnSteps dwords a row
constexpr int kDnDma = kDnCodes / 1024 + 2;

// Workgroup (column tile, split): the tile's entries (experts in use, or assignments) are dealt to
// the waves of its `splits` workgroups in turn, each in windows of up to kDnSteps steps.  Of an
// entry a wave takes a `parts`-th of the steps (parts > 1 with at most four entries).
// W2's 16 rows of a window go straight to the wave's own part of LDS, the next window's while
// this one is computed, with no barrier.  Taken to registers in the products' layout they cost
// the address unit one access a lane, since 16 adjacent lanes hold 16 rows (64 tokens: 29 us, here 25).
// With several splits each workgroup leaves its sums in the workspace, and the last one to
// arrive adds them up, in split order whoever it is.
// The SwiGLU rows are in assignment order, or (grouped) in expert order.
template <bool OUT_F32, bool GROUPED>
__global__ __launch_bounds__(kDnWaves * 64) void k_few_down(MxFewArgs a, int splits) {
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  extern __shared__ float table[];  // [wave][token][16 columns]
  // (two arrays: the compiler then knows that reads of one do not depend on the loads into the other)
  __shared__ __attribute__((aligned(1024))) uint8_t ring0[kDnWaves * kDnSlot], ring1[kDnWaves * kDnSlot];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane & 15, g = lane >> 4;
  const int R = a.T * a.k;
  const int most = GROUPED ? min(a.E, R) : R;  // entries
  const int parts = most > 4 || splits > 1 ? 1 : most > 2 ? 2 : 4;
  const int tile = blockIdx.x / splits, split = blockIdx.x - tile * splits;
  const int part = wave % parts, stride = splits * kDnWaves / parts;
  const int steps = (a.I + 127) / 128;
  const int per = min(kDnSteps, (steps + parts - 1) / parts);  // consecutive steps of a wave's window
  const int windows = (steps + parts * per - 1) / (parts * per);
  const int c0 = tile * 16;
  const Mat h = matrix(ws.h_codes, ws.h_scales, 0, R, a.I);
  float *mine = table + wave * a.T * 16;
  // the wave's entries, 64 at a time, one per lane: expert, first row, rows
  int le = -1, lr = 0, ln = 0;
  const int first = (split * kDnWaves + wave) / parts;
  const auto load_entries = [&](int from) __attribute__((always_inline)) {
    const int i = first + (from + lane) * stride;
    if (i < most) {
      if (!GROUPED) {
        le = ws.id[i];
        lr = i;
        ln = le < 0 ? 0 : 1;
      } else {  // (behind the experts in use: not written, not used)
        le = ws.act_e[i];
        lr = ws.act_row[i];
        ln = ws.act_row[i + 1] - lr;
      }
    }
  };
  load_entries(0);
  const int na = GROUPED ? __builtin_amdgcn_readfirstlane(*ws.n_active) : R;
  const int count = (first < na ? (na - first + stride - 1) / stride : 0) * windows;
  for (int i = lane; i < a.T * 4; i += 64) reinterpret_cast<f32x4 *>(mine)[i] = f32x4{0, 0, 0, 0};
  // LDS position 16 p (p = 64 i + lane) holds block (p % 24) ^ (row / 2 % 8) of row p / 24: the 16
  // rows' same block then lies in 16 different groups of banks
  constexpr int kRow = kDnSteps * 4;
  int at_row[kDnCodes / 1024], at_b[kDnCodes / 1024];
#pragma unroll
  for (int i = 0; i < kDnCodes / 1024; ++i) {
    const int p = i * 64 + lane, r = p / kRow;
    at_row[i] = c0 + r < a.H ? r : -1;
    at_b[i] = (p - r * kRow) ^ ((r >> 1) & 7);
  }
  struct Item {
    int e, r0, n, s0;
  };
  // item c: entry c / windows, window c % windows (counted up alongside, ic and iw)
  int ic = 0, iw = 0;
  const auto next_item = [&]() __attribute__((always_inline)) -> Item {
    const int i = ic & 63;
    if (i == 0 && ic > 0 && iw == 0) load_entries(ic);
    const Item it{__builtin_amdgcn_readlane(le, i), __builtin_amdgcn_readlane(lr, i),
                  __builtin_amdgcn_readlane(ln, i), (iw * parts + part) * per};
    if (++iw == windows) iw = 0, ++ic;
    return it;
  };
  const auto dma = [&](uint8_t *ring, const Item &it) __attribute__((always_inline)) {
    const Mat w2 = matrix(a.w2_codes, a.w2_scales, (int64_t)max(it.e, 0) * a.H + c0, min(16, a.H - c0), a.I);
    uint8_t *dst = ring + wave * kDnSlot;
    const bool live = it.e >= 0;
#pragma unroll
    for (int i = 0; i < kDnCodes / 1024; ++i) {
      const int b = it.s0 * 4 + at_b[i];
      const bool in = live & (at_row[i] >= 0) & (at_b[i] < per * 4) & (b < w2.nb);
      mx_dma16<true>(w2.codes, w2.cbytes, dst + i * 1024, in ? (uint32_t)(at_row[i] * w2.nb + b) * 16u : kOut);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int p = j * 64 + lane, r = p / kDnSteps, d = p - r * kDnSteps;
      const bool in = live & (r < 16) & (c0 + r < a.H) & (d < per) & (it.s0 + d < steps);
      mx_dma4(w2.scales, w2.sbytes, dst + kDnCodes + j * 256,
              in ? (uint32_t)(r * w2.sld + (it.s0 + d) * 4) : kOut);
    }
  };
  // rows q .. q + 15 of an entry: row slot l's steps from s0 on, weight and token
  struct Rows {
    u32x4 c[kDnSteps];
    u32x4 lo;
    u32x2 hi;
    float w;
    int t;
  };
  const auto load_rows = [&](Rows &x, const Item &it, int q) __attribute__((always_inline)) {
    const int row = q + l < it.n ? it.r0 + q + l : -1;
#pragma unroll
    for (int s = 0; s < kDnSteps; ++s) x.c[s] = load_codes(h, s < per ? row : -1, (it.s0 + s) * 4 + g);
    const uint32_t at = ((row >= 0) & (it.s0 < steps)) ? (uint32_t)(row * h.sld + it.s0 * 4) : kOut;
    x.lo = load16(h.scales, h.sbytes, at);
    x.hi = load8(h.scales, h.sbytes, per > 4 ? at + 16 : kOut);
    x.w = (GROUPED ? ws.row_w : ws.w)[max(row, 0)];
    x.t = GROUPED ? ws.row_token[max(row, 0)] : few_token(max(row, 0), a.T);
  };
  Item it = count > 0 ? next_item() : Item{-1, 0, 0, 0};
  Rows x[2];
  dma(ring0, it);
  load_rows(x[0], it, 0);
  const auto item = [&](auto P, int c) __attribute__((always_inline)) {
    constexpr int p = decltype(P)::value;
    const bool more = c + 1 < count;
    const Item cur = it;
    // W2's window and the rows of this item were asked for before the next window
    if (more) {
      it = next_item();
      dma(p ? ring0 : ring1, it);
      mx_wait_vm<kDnDma>();
      load_rows(x[1 - p], it, 0);
    } else {
      mx_wait_vm<0>();
    }
    const uint8_t *w = (p ? ring1 : ring0) + wave * kDnSlot;
    for (int q = 0; q < cur.n; q += 16) {
      if (q > 0) load_rows(x[p], cur, q);
      const uint32_t xs[kDnSteps] = {x[p].lo[0], x[p].lo[1], x[p].lo[2], x[p].lo[3], x[p].hi[0], x[p].hi[1]};
      f32x4 acc = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < kDnSteps; ++s) {
        const int b = s < per ? (cur.s0 + s) * 4 + g : h.nb;
        const u32x4 wc = *reinterpret_cast<const u32x4 *>(w + (l * kRow + ((s * 4 + g) ^ ((l >> 1) & 7))) * 16);
        const uint32_t wsc = *reinterpret_cast<const uint32_t *>(w + kDnCodes + (l * kDnSteps + s) * 4);
        acc = mfma16(wc, scale_of(wsc, g, b, h.nb), x[p].c[s], scale_of(xs[s], g, b, h.nb), acc);
      }
      // The products of all lanes: without this the compiler moves them, and the scales that they
      // take from every lane, under the condition below.
      asm volatile("" : "+v"(acc));
      // lane = row slot l, columns 4 g ..: an expert's rows are different tokens, so no two
      // lanes meet in the table
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (q + l < cur.n) {
        f32x4 *dst = reinterpret_cast<f32x4 *>(mine + x[p].t * 16 + g * 4);
        f32x4 v = *dst;
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] += x[p].w * acc[u];
        *dst = v;
      }
    }
  };
  for (int c = 0; c < count; c += 2) {
    item(std::integral_constant<int, 0>{}, c);
    if (c + 1 < count) item(std::integral_constant<int, 1>{}, c + 1);
  }
  mx_wait_vm<0>();  // loads into this workgroup's LDS end before it does
  __syncthreads();
  const auto store = [&](int i, float v) __attribute__((always_inline)) {
    const int t = i >> 4, c = c0 + (i & 15);
    if (c < a.H) {
      if constexpr (OUT_F32) static_cast<float *>(a.out)[t * a.ldo + c] = v;
      else reinterpret_cast<__bf16 *>(a.out)[t * a.ldo + c] = (__bf16)v;
    }
  };
  float *sums = ws.sums + (int64_t)tile * splits * a.T * 16;
  for (int i = tid; i < a.T * 16; i += kDnWaves * 64) {
    float v = 0;
#pragma unroll
    for (int k = 0; k < kDnWaves; ++k) v += table[k * a.T * 16 + i];
    if (splits == 1) store(i, v);
    else __hip_atomic_store(sums + split * a.T * 16 + i, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (splits == 1) return;
  // The sums were stored past this XCD's L2 and are loaded past the reader's (agent scope): it is
  // enough that they have arrived before this workgroup counts as arrived.  A fence at that scope
  // would write back and invalidate the whole L2.
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0)
    s_last = __hip_atomic_fetch_add(ws.arrived + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == splits - 1;
  __syncthreads();
  if (!s_last) return;
  for (int i = tid; i < a.T * 16; i += kDnWaves * 64) {
    float v = 0;
    for (int k = 0; k < splits; ++k)
      v += __hip_atomic_load(sums + k * a.T * 16 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    store(i, v);
  }
}

// The smallest batches: one kernel less (see the top) when they are routed here.
bool few_smallest(const MxFewArgs &a) { return a.T <= kFusedTokens && (int64_t)a.T * a.H <= kFusedElems; }
bool few_fused(const MxFewArgs &a) { return a.logits && few_smallest(a); }

// Listing the experts costs 5 us, which pay once experts have several rows each: the GEMM, and the
// down product by experts, then read their weights once.  (Not the smallest batches: the same routing
// has the same bits whether it is computed here or given.)  The host knows the number of assignments
// and experts, not the routing: the rule takes it to be even.  Measured in us, layers in turn, even
// routing, one by one / grouped, by assignments:
//   8 experts (H 4096, I 14336)    8  106 / 113   12  143 / 130   16  163 / 141   32  240 / 151
//   8 (H 4096, I 1536)            16 31.4 / 31.0  32 39.5 / 39.0  48 47.4 / 39.4
//   16 (H 4096, I 4096)           16 70.2 / 77.6  24 86.3 / 88.2  32 99.7 / 88.7
//   32 (H 2880, I 2880)           24 74.6 / 79.8  40  102 / 100   64  135 / 117
//   64 (H 2048, I 1408)           48 51.5 / 53.5  60 58.8 / 55.7  96 71.9 / 66.8
//   64 (H 2048, I 1024)           48 44.4 / 51.2  72 51.4 / 52.9  96 58.8 / 55.2
//   128 (H 2048, I 768)           72 47.2 / 51.1  96 54.2 / 54.3 112 58.7 / 55.0
//   256 (H 2048, I 512)           64 39.2 / 42.8  96 49.0 / 55.1 128 58.1 / 59.6
// The border moves with I as well, which the rule leaves out: at 8 experts it is below 12 assignments
// for I 14336 and at 16 for 1536, and the rule takes 12.  On the other side of it a batch loses at
// most 10 % (8 experts, I 14336, 12; 16 experts, 24: 88.2 for 86.3).  Every token at the same experts
// is the rule's worst case: one by one the down product reads an expert's weights once per token
// (64 tokens of 2 of 256 experts, I 512: 38.0 / 29.3; 64 of 1 of 128, I 768: 29.5 / 28.3), which still
// takes less than even routing (54.0 and 42.6).
bool few_grouped(const MxFewArgs &a) {
  return !few_smallest(a) && a.T * a.k > std::min({a.E + 4, 64 + a.E / 4, kMostRows});
}

template <int NPL, int LPT, bool F32>
hipError_t launch_first(const MxFewArgs &a, hipStream_t stream) {
  const unsigned grid = (unsigned)(a.I / 32) * (unsigned)std::min(a.E, a.T * a.k);  // experts in use
  if (few_fused(a)) {
    k_few_gate_up<true, NPL, LPT, F32><<<grid, kGuThreads, 0, stream>>>(a);
    return hipSuccess;
  }
  const int per = 4 * (kWave / LPT);  // tokens per routing workgroup
  const int nroute = a.logits ? (a.T + per - 1) / per : (a.T * a.k + 255) / 256;
  const int units = a.T * ((a.H + 127) / 128);
  k_few_route<NPL, LPT, F32><<<(unsigned)(nroute + (units + 15) / 16), 256, 0, stream>>>(a, nroute);
  if (!few_grouped(a)) {
    k_few_gate_up<false, 1, 64, false><<<grid, kGuThreads, 0, stream>>>(a);
    return hipSuccess;
  }
  k_few_group<<<1, kGuThreads, 0, stream>>>(a);
  FewWs ws;
  few_ws(a.ws, a.T, a.E, a.k, a.H, a.I, ws);
  MxGemmArgs g{};
  g.a_codes = ws.x_codes;
  g.a_scales = ws.x_scales;
  g.a_rows = a.T;
  g.K = a.H;
  g.a_rows_index = ws.row_token;
  g.b_codes = a.w13_codes;
  g.b_scales = a.w13_scales;
  g.b_rows = (int64_t)a.E * 2 * a.I;
  g.offsets = ws.offsets;
  g.E = a.E;
  g.M_cap = a.T * a.k;
  g.N = a.I;
  g.group_mode = NV4_GROUP_M;
  g.epilogue = NV4_EPI_SWIGLU;
  g.q_codes = ws.h_codes;
  g.q_scales = ws.h_scales;
  g.ceil_rule = a.ceil_rule;
  return launch_mx_gemm(g, stream);
}
template <bool F32>
hipError_t launch_first(const MxFewArgs &a, hipStream_t stream) {
  if (a.E <= 64) return launch_first<2, 32, F32>(a, stream);
  if (a.E <= 128) return launch_first<4, 32, F32>(a, stream);
  if (a.E <= 256) return launch_first<4, 64, F32>(a, stream);
  if (a.E <= 512) return launch_first<8, 64, F32>(a, stream);
  return launch_first<16, 64, F32>(a, stream);
}

}  // namespace

size_t mx_few_workspace_bytes(int64_t T, int E, int k, int64_t H, int64_t I) {
  FewWs w;
  return few_ws(nullptr, T, E, k, H, I, w);
}

hipError_t launch_mx_few(const MxFewArgs &a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const hipError_t first = a.x_is_f32 ? launch_first<true>(a, stream) : launch_first<false>(a, stream);
  if (first != hipSuccess) return first;
  const unsigned lds = (unsigned)(kDnWaves * a.T * 16 * sizeof(float));
  const int tiles = (a.H + 15) / 16, entries = std::min(a.E, a.T * a.k);
  // workgroups for the whole chip, at least an entry for each of their waves
  const int splits = std::max(1, std::min({kMaxSplits, device_cu_count() / tiles, entries / kDnWaves}));
  const unsigned grid = (unsigned)(tiles * splits);
  const bool grouped = few_grouped(a);
  const auto kernel = a.out_is_f32 ? (grouped ? k_few_down<true, true> : k_few_down<true, false>)
                                   : (grouped ? k_few_down<false, true> : k_few_down<false, false>);
  kernel<<<grid, kDnWaves * 64, lds, stream>>>(a, splits);
  return hipGetLastError();
}

}  // namespace nv4
