// The router's balance and z losses, per-expert counts, and the gradient of the logits for gfx950.
//
//   p = softmax(l), lse = log sum exp(l);  over the n tokens of a segment c_e assignments, P_e = sum p_e:
//   balance_s = E / (k n^2) sum_e c_e P_e,  z_s = 1/n sum lse^2,  the losses their means over the segments.
//   d balance / d l_j = E / (nseg k n^2) p_j (c_j - sum_i c_i p_i),  d z / d l_j = 2 / (nseg n) lse p_j.
//
// Both passes are bound by the logits (4 bytes read; backward also 4 written), with an exp and some
// twenty other operations for each.
//
// Loss: a workgroup takes a chunk of consecutive tokens, a half-wave (or wave) a token at a time, each
// lane summing its own experts' probabilities in registers over the tokens; where a segment ends inside
// the chunk, and at its end, the waves' sums meet in LDS and leave as one partial.  Chunk b's part of
// segment s goes to slot b + s: the pairs that occur form a staircase, so no slot is used twice.  A
// second kernel adds a segment's slots in their order and forms the losses; no sum depends on the order in which
// workgroups run.
#include <algorithm>

#include "nv4_device.h"
#include "nv4_internal.h"
#include "router_internal.h"
#include "topk_device.h"

namespace nv4 {
namespace {

constexpr int kMaxE = 1024;
constexpr int kBalThreads = 256;
constexpr int kBalWaves = kBalThreads / 64;

// tokens of a chunk: enough chunks to fill the chip, few enough for the second kernel's sums
__host__ __device__ inline int64_t bal_chunk(int64_t T) { return T <= 32 * 1024 ? 32 : (T + 1023) / 1024; }
inline int64_t bal_chunks(int64_t T) { return (T + bal_chunk(T) - 1) / bal_chunk(T); }

// workspace: partial sums by slot, then by segment
struct BalWs {
  float *psum;     // [slots][E]
  int32_t *count;  // [slots][E]
  float *z;        // [slots]
  int32_t *n;      // [slots]
  float *seg;      // [nseg][2]: a segment's balance and z
  uint32_t *done;  // segments that the second kernel has finished
};
inline size_t bal_align(size_t b) { return (b + 255) & ~(size_t)255; }
inline BalWs bal_ws(void *ws, int64_t T, int E, int nseg, size_t *bytes) {
  const size_t slots = (size_t)(bal_chunks(T) + nseg);
  size_t at = 0;
  const auto take = [&](size_t b) {
    const uintptr_t r = reinterpret_cast<uintptr_t>(ws) + at;
    at += bal_align(b);
    return r;
  };
  BalWs w;
  w.psum = reinterpret_cast<float *>(take(slots * E * 4));
  w.count = reinterpret_cast<int32_t *>(take(slots * E * 4));
  w.z = reinterpret_cast<float *>(take(slots * 4));
  w.n = reinterpret_cast<int32_t *>(take(slots * 4));
  w.seg = reinterpret_cast<float *>(take((size_t)nseg * 8));
  w.done = reinterpret_cast<uint32_t *>(take(4));
  *bytes = at;
  return w;
}

// a segment border, inside [0, T] whatever the array holds
__device__ __forceinline__ int64_t bal_border(const int32_t *off, int s, int64_t T) {
  return off ? std::min<int64_t>(std::max<int64_t>(off[s], 0), T) : s ? T : 0;
}
// the last segment that starts at or before t, -1 without one
__device__ __forceinline__ int bal_segment(const int32_t *off, int nseg, int64_t t) {
  if (!off) return 0;
  int lo = -1, hi = nseg;  // off[lo] <= t < off[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// One token's softmax on its LPT lanes: v[i] = exp(l - max) (0 behind E), their sum, and lse.  A token
// whose logits are all -infinity has v = 0 and sum 0.
template <int NPL, int LPT>
__device__ __forceinline__ void bal_softmax(const float *lg, bool valid, int E, int ll, float (&v)[NPL], float &sum,
                                            float &lse, bool &bad) {
  float mx = -INFINITY;
  bad = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = ll + LPT * i;
    v[i] = -INFINITY;
    if (valid && e < E) v[i] = lg[e];
    bad |= !(v[i] < INFINITY);  // NaN or +infinity
    mx = fmaxf(mx, v[i]);
  }
  mx = wave_max_dpp<LPT>(mx);
  const bool none = mx == -INFINITY;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    v[i] = none ? (v[i] != v[i] ? v[i] : 0.0f) : expf(v[i] - mx);
    sum += v[i];
  }
  sum = wave_sum_dpp<LPT>(sum);
  lse = sum == 0.0f ? 0.0f : mx + logf(sum);
}

template <int NPL, int LPT>
__global__ __launch_bounds__(kBalThreads) void k_balance(BalanceArgs a, BalWs w, int64_t chunk) {
  constexpr int TPW = 64 / LPT, TPB = kBalWaves * TPW;  // tokens at a time
  __shared__ int cnt[kMaxE];
  __shared__ float ps[kBalWaves][NPL * LPT];
  __shared__ float zs[kBalWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sub = lane / LPT, ll = lane % LPT;
  if (blockIdx.x == 0 && tid == 0) *w.done = 0;
  const int64_t end = std::min<int64_t>((blockIdx.x + 1) * chunk, a.T);
  int64_t t = blockIdx.x * chunk;
  int s = bal_segment(a.seg_offsets, a.nseg, t);
  bool bad = false, badid = false;
  if (s < 0) {
    s = 0;
    t = std::max<int64_t>(t, bal_border(a.seg_offsets, 0, a.T));
  }
  for (; s < a.nseg && t < end; ++s) {
    const int64_t hi = std::min<int64_t>(bal_border(a.seg_offsets, s + 1, a.T), end);
    if (hi <= t) continue;
    __syncthreads();
    for (int e = tid; e < a.E; e += kBalThreads) cnt[e] = 0;
    __syncthreads();
    float acc[NPL], z = 0.0f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) acc[i] = 0.0f;
    for (int64_t t0 = t; t0 < hi; t0 += TPB) {  // (the same count for every wave)
      const int64_t tt = t0 + wave * TPW + sub;
      const bool live = tt < hi && (!a.mask || a.mask[tt]);
      float v[NPL], sum, lse;
      bool b;
      bal_softmax<NPL, LPT>(a.logits + tt * a.E, live, a.E, ll, v, sum, lse, b);
      if (!live) continue;
      bad |= b;
      if (sum != 0.0f) {
#pragma unroll
        for (int i = 0; i < NPL; ++i) acc[i] += v[i] / sum;
        z = __builtin_fmaf(lse, lse, z);
      }
      ++n;
      if (ll < a.k) {
        const int id = a.topk_ids[tt * a.k + ll];
        if (id >= 0 && id < a.E) atomicAdd(&cnt[id], 1);
        else badid = true;
      }
    }
    // the wave's two tokens, then the waves
    if (LPT == 32) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) acc[i] += __shfl_xor(acc[i], 32, 64);
      z += __shfl_xor(z, 32, 64);
      n += __shfl_xor(n, 32, 64);
    }
    if (sub == 0) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) ps[wave][ll + LPT * i] = acc[i];
    }
    if (lane == 0) zs[wave][0] = z, zs[wave][1] = __int_as_float(n);
    __syncthreads();
    const int64_t slot = blockIdx.x + s;
    for (int e = tid; e < a.E; e += kBalThreads) {
      float p = ps[0][e];
#pragma unroll
      for (int i = 1; i < kBalWaves; ++i) p += ps[i][e];
      w.psum[slot * a.E + e] = p;
      w.count[slot * a.E + e] = cnt[e];
    }
    if (tid == 0) {
      float zz = zs[0][0];
      int nn = __float_as_int(zs[0][1]);
#pragma unroll
      for (int i = 1; i < kBalWaves; ++i) zz += zs[i][0], nn += __float_as_int(zs[i][1]);
      w.z[slot] = zz;
      w.n[slot] = nn;
    }
    t = hi;
  }
  if (a.dev_status) {
    if (bad) atomicOr(a.dev_status, kDsNanLogit);
    if (badid) atomicOr(a.dev_status, kDsBadExpert);
  }
}

// One workgroup of 1024 a segment: its slots' sums, 16 at a time for 64 experts, and its losses; the
// last workgroup adds the segments' losses.
__global__ __launch_bounds__(1024) void k_balance_sum(BalanceArgs a, BalWs w, int64_t chunk) {
  __shared__ float sp[16][64];
  __shared__ int sc[16][64];
  __shared__ float s_dot[16], s_z[16];
  __shared__ int s_n[16];
  __shared__ bool s_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, s = blockIdx.x;
  const int64_t lo = bal_border(a.seg_offsets, s, a.T), hi = bal_border(a.seg_offsets, s + 1, a.T);
  const int64_t first = lo / chunk + s, last = hi > lo ? (hi - 1) / chunk + s : first - 1;
  float dot = 0.0f;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const int e = e0 + lane;
    float p = 0.0f;
    int c = 0;
    if (e < a.E) {
#pragma unroll 4
      for (int64_t b = first + wave; b <= last; b += 16) {
        p += w.psum[b * a.E + e];
        c += w.count[b * a.E + e];
      }
    }
    sp[wave][lane] = p;
    sc[wave][lane] = c;
    __syncthreads();
    if (wave == 0 && e < a.E) {
#pragma unroll
      for (int i = 1; i < 16; ++i) p += sp[i][lane], c += sc[i][lane];
      a.prob_sums[(int64_t)s * a.E + e] = p;
      a.counts[(int64_t)s * a.E + e] = c;
      dot = __builtin_fmaf((float)c, p, dot);
    }
    __syncthreads();
  }
  float z = 0.0f;
  int n = 0;
  for (int64_t b = first + tid; b <= last; b += 1024) z += w.z[b], n += w.n[b];
  z = wave_sum_dpp(z);
  n = (int)wave_reduce_u32((uint32_t)n, [](uint32_t x, uint32_t y) { return x + y; });
  dot = wave_sum_dpp(dot);
  if (lane == 0) s_dot[wave] = dot, s_z[wave] = z, s_n[wave] = n;
  __syncthreads();
  if (tid == 0) {
    z = s_z[0], n = s_n[0];
    for (int i = 1; i < 16; ++i) z += s_z[i], n += s_n[i];
    a.tokens[s] = n;
    // (n^2 as FP32 factors: 65536 tokens squared leave 32 bits)
    const float fn = (float)n;
    w.seg[2 * s] = n ? (float)a.E / (float)a.k / fn * (s_dot[0] / fn) : 0.0f;
    w.seg[2 * s + 1] = n ? z / fn : 0.0f;
    __threadfence();
    s_last = atomicAdd(w.done, 1u) == (uint32_t)a.nseg - 1u;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // thread i adds segments i, i + 1024, ..; then a fixed tree
  float b = 0.0f, zz = 0.0f;
  for (int i = tid; i < a.nseg; i += 1024) {
    b += __hip_atomic_load(&w.seg[2 * i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    zz += __hip_atomic_load(&w.seg[2 * i + 1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  b = wave_sum_dpp(b);
  zz = wave_sum_dpp(zz);
  __syncthreads();
  if (lane == 0) s_dot[wave] = b, s_z[wave] = zz;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < 16; ++i) b += s_dot[i], zz += s_z[i];
    a.loss[0] = b / (float)a.nseg;
    a.loss[1] = zz / (float)a.nseg;
  }
}

// The gradient of a token's logits on its LPT lanes.  With q_j = sum of dw_m over the choices m of expert
// j and m_j how many there are, the weights' part is p_j (q_j - sum_i p_i q_i), or with renormalised
// weights r_j = p_j / sum_i m_i p_i:  r_j (q_j - m_j sum_i r_i q_i).
template <int NPL, int LPT>
__global__ __launch_bounds__(kBalThreads) void k_balance_backward(BalanceBackwardArgs a) {
  constexpr int TPW = 64 / LPT;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / LPT, ll = lane % LPT;
  const int64_t t = ((int64_t)blockIdx.x * kBalWaves + wave) * TPW + sub;
  const bool valid = t < a.T;
  float dw = 0.0f;
  int id = -1;
  if (valid && a.dtopk_w && ll < a.k) {
    dw = a.dtopk_w[t * a.k + ll];
    id = a.topk_ids[t * a.k + ll];
    if (id < 0 || id >= a.E) {
      id = -1;
      if (a.dev_status) atomicOr(a.dev_status, kDsBadExpert);
    }
  }
  bool counted = valid && a.dloss && (!a.mask || a.mask[t]);
  int s = 0;
  float fn = 0.0f;
  if (counted) {
    s = bal_segment(a.seg_offsets, a.nseg, t);
    counted = s >= 0 && t < bal_border(a.seg_offsets, s + 1, a.T);
    if (counted) fn = (float)a.tokens[s];
    counted = counted && fn > 0.0f;
  }
  // whether the weights' gradient reaches the token: some dw that is not 0 (NaN included)
  const uint64_t any = __ballot(!(dw == 0.0f));
  const bool weighted = LPT == 64 ? any != 0 : (uint32_t)(any >> (32 * sub)) != 0;
  const bool live = counted || weighted;
  float v[NPL], sum, lse;
  bool bad;
  bal_softmax<NPL, LPT>(a.logits + t * a.E, live, a.E, ll, v, sum, lse, bad);
  if (bad && live && a.dev_status) atomicOr(a.dev_status, kDsNanLogit);
  float cb = 0.0f, cz = 0.0f;
  if (counted) {
    cb = a.dloss[0] * ((float)a.E / (float)a.k / (float)a.nseg / fn) / fn;
    cz = a.dloss[1] * 2.0f / (float)a.nseg / fn * lse;
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  float c[NPL], q[NPL], m[NPL], cp = 0.0f, pq = 0.0f, mp = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = ll + LPT * i;
    v[i] *= inv;
    c[i] = counted && e < a.E ? (float)a.counts[(int64_t)s * a.E + e] : 0.0f;
    q[i] = m[i] = 0.0f;
    cp = __builtin_fmaf(c[i], v[i], cp);
  }
  if (a.dtopk_w) {
    for (int j = 0; j < a.k; ++j) {
      const int idj = __shfl(id, sub * LPT + j, 64);
      const float dwj = __shfl(dw, sub * LPT + j, 64);
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (idj == ll + LPT * i) q[i] += dwj, m[i] += 1.0f;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      pq = __builtin_fmaf(v[i], q[i], pq);
      mp = __builtin_fmaf(v[i], m[i], mp);
    }
    pq = wave_sum_dpp<LPT>(pq);
    if (a.renorm) mp = wave_sum_dpp<LPT>(mp);
  }
  cp = wave_sum_dpp<LPT>(cp);
  const float rz = a.renorm ? (mp == 0.0f ? 0.0f : 1.0f / mp) : 1.0f, D = pq * rz;
  if (!valid) return;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = ll + LPT * i;
    if (e >= a.E) continue;
    float d = v[i] * __builtin_fmaf(cb, c[i] - cp, cz);
    if (weighted) d = __builtin_fmaf(v[i] * rz, q[i] - (a.renorm ? m[i] * D : D), d);
    a.dlogits[t * a.E + e] = live ? d : 0.0f;
  }
}

template <class F>
void by_experts(int E, F f) {
  if (E <= 32) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 32>{});
  else if (E <= 64) f(std::integral_constant<int, 2>{}, std::integral_constant<int, 32>{});
  else if (E <= 128) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 32>{});
  else if (E <= 256) f(std::integral_constant<int, 4>{}, std::integral_constant<int, 64>{});
  else if (E <= 512) f(std::integral_constant<int, 8>{}, std::integral_constant<int, 64>{});
  else f(std::integral_constant<int, 16>{}, std::integral_constant<int, 64>{});
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int E, int nseg) {
  size_t bytes;
  bal_ws(nullptr, T, E, nseg, &bytes);
  return bytes;
}

hipError_t launch_balance_loss(const BalanceArgs &a, hipStream_t stream) {
  size_t bytes;
  const BalWs w = bal_ws(a.ws, a.T, a.E, a.nseg, &bytes);
  const int64_t chunk = bal_chunk(a.T);
  // (without a token one workgroup still clears the count of finished segments)
  const unsigned grid = (unsigned)std::max<int64_t>(bal_chunks(a.T), 1);
  by_experts(a.E, [&](auto npl, auto lpt) {
    k_balance<decltype(npl)::value, decltype(lpt)::value><<<grid, kBalThreads, 0, stream>>>(a, w, chunk);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_balance_sum<<<a.nseg, 1024, 0, stream>>>(a, w, chunk);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceBackwardArgs &a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  by_experts(a.E, [&](auto npl, auto lpt) {
    constexpr int tokens = kBalWaves * 64 / decltype(lpt)::value;
    k_balance_backward<decltype(npl)::value, decltype(lpt)::value>
        <<<(unsigned)((a.T + tokens - 1) / tokens), kBalThreads, 0, stream>>>(a);
  });
  return hipGetLastError();
}

}  // namespace nv4
