// The router's balance and z losses, per-expert counts, and the gradient of the logits for gfx950.
//
//   p = softmax(l), lse = log sum exp(l);  over the n tokens of a segment c_e assignments, P_e = sum p_e:
//   balance_s = E / (k n^2) sum_e c_e P_e,  z_s = 1/n sum lse^2,  the losses their means over the segments.
//   d balance / d l_j = E / (nseg k n^2) p_j (c_j - sum_i c_i p_i),  d z / d l_j = 2 / (nseg n) lse p_j.
//
// A logit is 4 bytes read (backward: and 4 written), an exp and some twenty other operations, so that both
// passes are bound by the VALU before memory.  65536 tokens of 128 experts: loss 15 us (VALU busy 67 %, 2.4 TB/s), the
// segments' sums 13, backward 23 (84 %, 3.0 TB/s).
//
// Loss: a workgroup takes a chunk of consecutive tokens, a half-wave (or wave) a token at a time, each
// lane summing its own experts' probabilities in registers over the tokens; where a segment ends inside
// the chunk, and at its end, the waves' sums meet in LDS and leave as one partial.  Chunk b's part of
// segment s goes to slot b + s: the pairs that occur form a staircase, so no slot is used twice.  A
// second kernel adds a segment's slots in their order and forms the losses; no sum depends on the order in which
// workgroups run.
#include <algorithm>

#include "many_groups.h"
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

// Tokens that a half-wave (wave) loads at once: as the registers last, or one where tokens are few (257 tokens
// of 60 experts, backward: 9.5 us with four, 4.9 with one; 65536 of 128, loss: 15.9 and 23).
__host__ __device__ constexpr int bal_at(int npl, bool many) { return !many ? 1 : npl <= 4 ? 4 : npl <= 8 ? 2 : 1; }
inline bool bal_many(int64_t T) { return T >= 16384; }

// a segment border, inside [0, T] whatever the array holds
__device__ __forceinline__ int64_t bal_border(const int32_t *off, int s, int64_t T) {
  return off ? std::min<int64_t>(std::max<int64_t>(off[s], 0), T) : s ? T : 0;
}
// the last segment that starts at or before t, -1 without one: among lo .. hi, off[lo] <= t < off[hi]
__device__ __forceinline__ int bal_segment(const int32_t *off, int lo, int hi, int64_t t) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}
// The same by the whole wave for one t, 64 borders at a time: a load for 64 segments where halving would
// take six, one behind the other.
__device__ __forceinline__ int bal_segment_wave(const int32_t *off, int nseg, int64_t t) {
  if (!off) return 0;
  const int lane = threadIdx.x & 63;
  int lo = -1, hi = nseg;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) / 64, i = lo + (lane + 1) * step;
    const int n = __popcll(__ballot(i < hi && off[min(i, nseg)] <= t));
    const int next = lo + n * step;
    hi = min(hi, next + step);
    lo = next;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// e^x for x <= 0 to two steps of FP32: the hardware's 2^y for y = x log2(e) rounded, times 1 + what the
// rounding left.  Below 2^-126 it may be 0.
__device__ __forceinline__ float bal_exp(float x) {
  const float c = __builtin_elementwise_maximum(x, -104.0f);  // (a NaN stays)
  const float y = c * 0x1.715476p+0f;
  const float left = __builtin_fmaf(c, 0x1.4ae0cp-26f, __builtin_fmaf(c, 0x1.715476p+0f, -y));
  const float r = __builtin_amdgcn_exp2f(y);
  return __builtin_fmaf(r, left * 0x1.62e43p-1f, r);
}

// A token's logits on its LPT lanes: four consecutive ones of every 4 LPT on a lane where it has that
// many, else every LPT-th
template <int NPL, int LPT>
__device__ __forceinline__ int bal_expert(int ll, int i) {
  return NPL % 4 == 0 ? i / 4 * 4 * LPT + ll * 4 + i % 4 : ll + LPT * i;
}
// (-infinity behind E and where there is no token; wide: E and the array allow 16-byte loads)
template <int NPL, int LPT, class T>
__device__ __forceinline__ void bal_load(const T *row, bool valid, bool wide, int E, int ll, T none, T (&v)[NPL]) {
#pragma unroll
  for (int i = 0; i < NPL; ++i) v[i] = none;
  if (!valid) return;
  if (NPL % 4 == 0 && wide) {
    typedef T T4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
      const int e = bal_expert<NPL, LPT>(ll, i);
      if (e >= E) continue;
      const T4 x = *reinterpret_cast<const T4 *>(row + e);
#pragma unroll
      for (int r = 0; r < 4; ++r) v[(i + r) % NPL] = x[r];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = bal_expert<NPL, LPT>(ll, i);
      if (e < E) v[i] = row[e];
    }
  }
}
template <class T>
__device__ __forceinline__ bool bal_wide(const T *p, int E) {
  return E % 4 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0;
}

// One token's softmax: v[i] = exp(l - max) in the logits' place, 1 / their sum, and lse.  A token whose logits
// are all -infinity has v = 0 and inv = 0; a NaN or +infinity among them makes all three NaN.
template <int NPL, int LPT>
__device__ __forceinline__ void bal_softmax(float (&v)[NPL], float &inv, float &lse, bool &bad) {
  float mx = v[0];
#pragma unroll
  for (int i = 1; i < NPL; ++i) mx = fmaxf(mx, v[i]);
  mx = wave_max_dpp<LPT>(mx);
  mx = mx == -INFINITY ? 0.0f : mx;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    v[i] = bal_exp(v[i] - mx);
    sum += v[i];
  }
  sum = wave_sum_dpp<LPT>(sum);
  bad = sum != sum;
  lse = sum == 0.0f ? 0.0f : mx + logf(sum);
  inv = sum == 0.0f ? 0.0f : 1.0f / sum;
}

template <int NPL, int LPT, bool MANY>
__global__ __launch_bounds__(kBalThreads) void k_balance(BalanceArgs a, BalWs w, int64_t chunk) {
  constexpr int TPW = 64 / LPT, TPB = kBalWaves * TPW;  // tokens at a time
  constexpr int AT = bal_at(NPL, MANY);                  // times as many under way
  __shared__ int cnt[kMaxE];
  __shared__ float ps[kBalWaves][NPL * LPT];
  __shared__ float zs[kBalWaves][2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sub = lane / LPT, ll = lane % LPT;
  if (blockIdx.x == 0 && tid == 0) *w.done = 0;
  const int64_t end = std::min<int64_t>((blockIdx.x + 1) * chunk, a.T);
  int64_t t = blockIdx.x * chunk;
  int s = bal_segment_wave(a.seg_offsets, a.nseg, t);
  const bool wide = bal_wide(a.logits, a.E);
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
    for (int64_t t0 = t; t0 < hi; t0 += AT * TPB) {  // (the same count for every wave)
      float v[AT][NPL];
      int id[AT];
      bool live[AT];
#pragma unroll
      for (int u = 0; u < AT; ++u) {
        const int64_t tt = t0 + u * TPB + wave * TPW + sub;
        bal_load<NPL, LPT>(a.logits + tt * a.E, tt < hi, wide, a.E, ll, -INFINITY, v[u]);
        live[u] = tt < hi && (!a.mask || a.mask[tt]);
        id[u] = tt < hi && ll < a.k ? a.topk_ids[tt * a.k + ll] : 0;
      }
#pragma unroll
      for (int u = 0; u < AT; ++u) {
        float inv, lse;
        bool b;
        bal_softmax<NPL, LPT>(v[u], inv, lse, b);
        if (!live[u]) continue;
        bad |= b;
#pragma unroll
        for (int i = 0; i < NPL; ++i) acc[i] = __builtin_fmaf(v[u][i], inv, acc[i]);
        z = __builtin_fmaf(lse, lse, z);
        ++n;
        if (ll < a.k) {
          if (id[u] >= 0 && id[u] < a.E) atomicAdd(&cnt[id[u]], 1);
          else badid = true;
        }
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
      for (int i = 0; i < NPL; ++i) ps[wave][bal_expert<NPL, LPT>(ll, i)] = acc[i];
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

// One workgroup of 1024 a segment: its slots' sums, 1024 / P at a time (P: the power of two from E on, 64 at
// least), and its losses; the last workgroup adds the segments' losses.
__global__ __launch_bounds__(1024) void k_balance_sum(BalanceArgs a, BalWs w, int64_t chunk) {
  __shared__ float sp[1024];
  __shared__ int sc[1024];
  __shared__ float s_dot[16], s_z[16];
  __shared__ int s_n[16];
  __shared__ bool s_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, s = blockIdx.x;
  const int64_t lo = bal_border(a.seg_offsets, s, a.T), hi = bal_border(a.seg_offsets, s + 1, a.T);
  const int64_t first = lo / chunk + s, last = hi > lo ? (hi - 1) / chunk + s : first - 1;
  const int P = a.E <= 64 ? 64 : 1 << (32 - __clz(a.E - 1)), e = tid & (P - 1), groups = 1024 / P;
  float dot = 0.0f, p = 0.0f, z = 0.0f;
  int c = 0, n = 0;
  for (int64_t b = first + tid; b <= last; b += 1024) z += w.z[b], n += w.n[b];
  if (e < a.E) {
#pragma unroll 8
    for (int64_t b = first + tid / P; b <= last; b += groups) {
      p += w.psum[b * a.E + e];
      c += w.count[b * a.E + e];
    }
  }
  sp[tid] = p;
  sc[tid] = c;
  __syncthreads();
  if (tid < a.E) {  // (P >= E: the first group's threads)
#pragma unroll 4
    for (int i = 1; i < groups; ++i) p += sp[i * P + tid], c += sc[i * P + tid];
    a.prob_sums[(int64_t)s * a.E + tid] = p;
    a.counts[(int64_t)s * a.E + tid] = c;
    dot = (float)c * p;
  }
  z = wave_sum_dpp(z);
  n = (int)wave_reduce_u32((uint32_t)n, [](uint32_t x, uint32_t y) { return x + y; });
  dot = wave_sum_dpp(dot);
  if (lane == 0) s_dot[wave] = dot, s_z[wave] = z, s_n[wave] = n;
  __syncthreads();
  if (tid == 0) {
    dot = s_dot[0], z = s_z[0], n = s_n[0];
    for (int i = 1; i < 16; ++i) dot += s_dot[i], z += s_z[i], n += s_n[i];
    a.tokens[s] = n;
    // (n^2 as FP32 factors: 65536 tokens squared leave 32 bits)
    const float fn = (float)n;
    const float bal = n ? (float)a.E / (float)a.k / fn * (dot / fn) : 0.0f;
    const float zz = n ? z / fn : 0.0f;
    s_last = false;
    if (a.nseg == 1) {
      a.loss[0] = bal;
      a.loss[1] = zz;
    } else {
      w.seg[2 * s] = bal;
      w.seg[2 * s + 1] = zz;
      __threadfence();
      s_last = atomicAdd(w.done, 1u) == (uint32_t)a.nseg - 1u;
    }
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

// A token's row in LDS, this lane's experts of it: a wave's own accesses to LDS keep their order, and volatile ones
// the program's.
template <class T>
using LdsRow = volatile __attribute__((address_space(3))) T *;
template <int NPL, int LPT, class T>
__device__ __forceinline__ void bal_clear_row(LdsRow<T> row, int ll) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  if constexpr (NPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NPL; i += 4) *(LdsRow<T4>)(row + bal_expert<NPL, LPT>(ll, i)) = T4{0, 0, 0, 0};
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) row[bal_expert<NPL, LPT>(ll, i)] = 0;
  }
}
template <int NPL, int LPT, class T>
__device__ __forceinline__ void bal_read_row(LdsRow<T> row, int ll, T (&v)[NPL]) {
  typedef T T4 __attribute__((ext_vector_type(4)));
  if constexpr (NPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
      const T4 x = *(LdsRow<T4>)(row + bal_expert<NPL, LPT>(ll, i));
#pragma unroll
      for (int r = 0; r < 4; ++r) v[i + r] = x[r];
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = row[bal_expert<NPL, LPT>(ll, i)];
  }
}

// The gradient of a token's logits on its LPT lanes.  With q_j = sum of dw_m over the choices m of expert
// j and m_j how many there are, the weights' part is p_j (q_j - sum_i p_i q_i), or with renormalised
// weights r_j = p_j / sum_i m_i p_i:  r_j (q_j - m_j sum_i r_i q_i).  Where no choice has the row's largest logit
// that sum may leave FP32's range: r_j is then taken from the choices' own softmax, exp(l_j - the largest chosen
// logit).  The logits are read again for it, by the few waves that meet such a token.
template <int NPL, int LPT, bool MANY, bool RENORM>
__global__ __launch_bounds__(kBalThreads) void k_balance_backward(BalanceBackwardArgs a) {
  constexpr int TPW = 64 / LPT, AT = bal_at(NPL, MANY);
  const int lane = threadIdx.x & 63, sub = lane / LPT, ll = lane % LPT;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  __shared__ __attribute__((aligned(16))) int places[kBalWaves][TPW][NPL * LPT];
  __shared__ __attribute__((aligned(16))) float weights[kBalWaves][TPW][NPL * LPT];
  const LdsRow<int> place = (LdsRow<int>)places[wave][sub];
  const LdsRow<float> weight = (LdsRow<float>)weights[wave][sub];
  // AT times TPW consecutive tokens a wave
  const int64_t first = ((int64_t)group_index() * kBalWaves + wave) * (AT * TPW);
  if (first >= a.T) return;
  const int64_t last = std::min<int64_t>(first + AT * TPW, a.T) - 1;
  const bool wide = bal_wide(a.logits, a.E), wide_c = bal_wide(a.counts, a.E), wide_d = bal_wide(a.dlogits, a.E);
  float l[AT][NPL], dw[AT];
  int id[AT];
  bool counted[AT];
#pragma unroll
  for (int u = 0; u < AT; ++u) {
    const int64_t t = first + u * TPW + sub;
    const bool valid = t < a.T;
    bal_load<NPL, LPT>(a.logits + t * a.E, valid, wide, a.E, ll, -INFINITY, l[u]);
    dw[u] = 0.0f;
    id[u] = -1;
    if (valid && a.dtopk_w && ll < a.k) {
      dw[u] = a.dtopk_w[t * a.k + ll];
      id[u] = a.topk_ids[t * a.k + ll];
    }
    counted[u] = valid && a.dloss && (!a.mask || a.mask[t]);
  }
  // a segment's coefficients: of p_j (c_j - sum) and of lse p_j
  const auto coefficients = [&](int s, float &cb, float &cz) {
    const float n = s >= 0 ? (float)a.tokens[s] : 0.0f;
    cb = n > 0.0f ? a.dloss[0] * ((float)a.E / (float)a.k / (float)a.nseg / n) / n : 0.0f;
    cz = n > 0.0f ? a.dloss[1] * 2.0f / (float)a.nseg / n : 0.0f;
    return n > 0.0f;
  };
  int s0 = 0, s1 = 0;
  float cb0 = 0.0f, cz0 = 0.0f;
  bool any0 = false;
  int64_t end0 = 0;
  if (a.dloss) {
    s0 = bal_segment_wave(a.seg_offsets, a.nseg, first);
    s1 = !a.seg_offsets || (s0 >= 0 && s0 + 1 < a.nseg && last < a.seg_offsets[s0 + 1]) || s0 == a.nseg - 1
             ? s0 : bal_segment_wave(a.seg_offsets, a.nseg, last);
    end0 = bal_border(a.seg_offsets, s0 + 1, a.T);
    any0 = coefficients(s0, cb0, cz0);
  }
  // counts of the segment that all of the wave's tokens lie in
  float c[NPL];
  int ci[NPL];
  const auto load_counts = [&](int s, bool in) {
    bal_load<NPL, LPT>(a.counts + (int64_t)max(s, 0) * a.E, in, wide_c, a.E, ll, 0, ci);
#pragma unroll
    for (int i = 0; i < NPL; ++i) c[i] = (float)ci[i];
  };
  load_counts(s0, any0 && s1 == s0);
#pragma unroll
  for (int u = 0; u < AT; ++u) {
    const int64_t t = first + u * TPW + sub;
    const bool valid = t < a.T;
    if (id[u] < -1 || id[u] >= a.E || (id[u] == -1 && valid && a.dtopk_w && ll < a.k)) {
      if (a.dev_status) atomicOr(a.dev_status, kDsBadExpert);
      id[u] = -1;
      dw[u] = 0.0f;
    }
    int s = s0;
    float cb = cb0, cz = cz0;
    bool in = any0;
    int64_t end = end0;
    if (s1 != s0 && counted[u]) {
      s = bal_segment(a.seg_offsets, s0, s1 + 1, t);
      end = bal_border(a.seg_offsets, s + 1, a.T);
      in = coefficients(s, cb, cz);
    }
    in = in && counted[u] && t < end;
    if (s1 != s0) load_counts(s, in);
    float cf[NPL];
    // whether the weights' gradient reaches the token: some dw that is not 0 (NaN included)
    const uint64_t any = __ballot(!(dw[u] == 0.0f));
    const bool weighted = LPT == 64 ? any != 0 : (uint32_t)(any >> (32 * sub)) != 0;
    const bool live = in || weighted;
    float (&v)[NPL] = l[u];
    float inv, lse;
    bool bad;
    bal_softmax<NPL, LPT>(v, inv, lse, bad);
    if (bad && live && a.dev_status) atomicOr(a.dev_status, kDsNanLogit);
    cb = in ? cb : 0.0f;
    cz = in ? cz * lse : 0.0f;
    float q[NPL], m[NPL], r[NPL], cp = 0.0f, pq = 0.0f, mp = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      v[i] *= inv;
      q[i] = m[i] = r[i] = 0.0f;
      cp = __builtin_fmaf(c[i], v[i], cp);
    }
    if (a.dtopk_w) {
      // A choice leaves its weight's gradient with its expert, whose lane fetches it.  (One that does not find its own
      // lane in the expert's place has the same expert as another one: those are compared one by one.)
      bal_clear_row<NPL, LPT, float>(weight, ll);
      if (RENORM) bal_clear_row<NPL, LPT, int>(place, ll);
      if (id[u] >= 0) {
        place[id[u]] = ll + 1;
        weight[id[u]] = dw[u];
      }
      const bool twice = id[u] >= 0 && place[id[u]] != ll + 1;
      if (__ballot(twice) == 0) {
        bal_read_row<NPL, LPT, float>(weight, ll, q);
        if (RENORM) {
          int j[NPL];
          bal_read_row<NPL, LPT, int>(place, ll, j);
#pragma unroll
          for (int i = 0; i < NPL; ++i) m[i] = j[i] ? 1.0f : 0.0f;
        }
      } else for (int j = 0; j < a.k; ++j) {
        const int idj = __shfl(id[u], sub * LPT + j, 64);
        const float dwj = __shfl(dw[u], sub * LPT + j, 64);
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          const bool hit = idj == bal_expert<NPL, LPT>(ll, i);
          q[i] += hit ? dwj : 0.0f;
          if (RENORM) m[i] += hit ? 1.0f : 0.0f;
        }
      }
      if (RENORM) {
        bool largest = false;  // (exp of the largest logit is 1, its probability inv)
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
          r[i] = v[i];
          largest |= m[i] != 0.0f && v[i] == inv;
        }
        const uint64_t found = __ballot(largest);
        const bool far = weighted && (LPT == 64 ? found == 0 : (uint32_t)(found >> (32 * sub)) == 0);
        if (__ballot(far) != 0) {
          float x[NPL], mx = -INFINITY;
          bal_load<NPL, LPT>(a.logits + t * a.E, valid, wide, a.E, ll, -INFINITY, x);
#pragma unroll
          for (int i = 0; i < NPL; ++i) mx = fmaxf(mx, m[i] != 0.0f ? x[i] : -INFINITY);
          mx = wave_max_dpp<LPT>(mx);
          mx = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
          for (int i = 0; i < NPL; ++i)
            if (far) r[i] = m[i] != 0.0f ? bal_exp(x[i] - mx) : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        pq = __builtin_fmaf(RENORM ? r[i] : v[i], q[i], pq);
        if (RENORM) mp = __builtin_fmaf(r[i], m[i], mp);
      }
      pq = wave_sum_dpp<LPT>(pq);
      if (RENORM) mp = wave_sum_dpp<LPT>(mp);
    }
    cp = wave_sum_dpp<LPT>(cp);
    const float rz = RENORM ? (mp == 0.0f ? 0.0f : 1.0f / mp) : 1.0f, D = pq * rz;
    if (!valid) continue;
    const float base = __builtin_fmaf(-cb, cp, cz) - (!RENORM && weighted ? D : 0.0f);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      float d = v[i] * (RENORM ? __builtin_fmaf(cb, c[i], base) : __builtin_fmaf(cb, c[i], base) + q[i]);
      if (RENORM && weighted) d = __builtin_fmaf(r[i] * rz, q[i] - m[i] * D, d);
      cf[i] = live ? d : 0.0f;
    }
    float *out = a.dlogits + t * a.E;
    if (NPL % 4 == 0 && wide_d) {
#pragma unroll
      for (int i = 0; i < NPL; i += 4) {
        const int e = bal_expert<NPL, LPT>(ll, i);
        if (e < a.E)
          *reinterpret_cast<f32x4 *>(out + e) = f32x4{cf[i], cf[(i + 1) % NPL], cf[(i + 2) % NPL], cf[(i + 3) % NPL]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < NPL; ++i) {
        const int e = bal_expert<NPL, LPT>(ll, i);
        if (e < a.E) out[e] = cf[i];
      }
    }
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
    constexpr int N = decltype(npl)::value, L = decltype(lpt)::value;
    if (bal_many(a.T)) k_balance<N, L, true><<<grid, kBalThreads, 0, stream>>>(a, w, chunk);
    else k_balance<N, L, false><<<grid, kBalThreads, 0, stream>>>(a, w, chunk);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_balance_sum<<<a.nseg, 1024, 0, stream>>>(a, w, chunk);
  return hipGetLastError();
}

hipError_t launch_balance_backward(const BalanceBackwardArgs &a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  by_experts(a.E, [&](auto npl, auto lpt) {
    constexpr int N = decltype(npl)::value, L = decltype(lpt)::value;
    const bool many = bal_many(a.T), renorm = a.renorm && a.dtopk_w;
    const int tokens = kBalWaves * 64 / L * bal_at(N, many);
    const dim3 grid = many_groups((a.T + tokens - 1) / tokens);
    if (many && renorm) k_balance_backward<N, L, true, true><<<grid, kBalThreads, 0, stream>>>(a);
    else if (many) k_balance_backward<N, L, true, false><<<grid, kBalThreads, 0, stream>>>(a);
    else if (renorm) k_balance_backward<N, L, false, true><<<grid, kBalThreads, 0, stream>>>(a);
    else k_balance_backward<N, L, false, false><<<grid, kBalThreads, 0, stream>>>(a);
  });
  return hipGetLastError();
}

}  // namespace nv4
