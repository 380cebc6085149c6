// Top-k routing of one token on LPT lanes of a wave, shared by moe_permute's routing kernel and
// the few-token layer (the two give the same ids and weights bit for bit).
#pragma once

#include "nv4_device.h"
#include "../../include/nv4moe.h"

namespace nv4 {

// Wave-wide reductions over 64 lanes without LDS: DPP within rows of 16 lanes (the
// pairs (i, i^1), (i, i^2), then the half-row and row mirrors), then the gfx950
// row swaps across 16 and 32 lanes.  Every lane ends with the result.
template <int LANES = 64, class F>
__device__ __forceinline__ uint32_t wave_reduce_u32(uint32_t v, F op) {
  static_assert(LANES == 32 || LANES == 64, "reductions over 32-lane halves or the wave");
  v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
  v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
  v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));  // row_half_mirror
  v = op(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));  // row_mirror
  const auto s16 = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = op(s16[0], s16[1]);
  if (LANES == 32) return v;  // each 32-lane half holds its own result
  const auto s32 = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return op(s32[0], s32[1]);
}
template <int LANES = 64>
__device__ __forceinline__ float wave_max_dpp(float v) {
  return __uint_as_float(wave_reduce_u32<LANES>(__float_as_uint(v), [](uint32_t x, uint32_t y) {
    return __float_as_uint(fmaxf(__uint_as_float(x), __uint_as_float(y)));
  }));
}
template <int LANES = 64>
__device__ __forceinline__ float wave_sum_dpp(float v) {
  return __uint_as_float(wave_reduce_u32<LANES>(__float_as_uint(v), [](uint32_t x, uint32_t y) {
    return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
  }));
}
template <int LANES = 64>
__device__ __forceinline__ int wave_min_dpp(int v) {
  return (int)wave_reduce_u32<LANES>((uint32_t)v, [](uint32_t x, uint32_t y) { return (uint32_t)min((int)x, (int)y); });
}

// LPT lanes per token (64: one token per wave; 32: two, one per half-wave), NPL
// logits per lane (expert e = lane-in-token + LPT * i): softmax statistics, then k
// rounds of an argmax over the token's lanes.  Each round: every lane's best untaken
// candidate (larger logit first, then lower id), the token's maximum value, and among
// the lanes holding it the lowest id (a ballot; a second reduction only when several
// lanes tie).  Lane j of the token keeps round j's id and logit; the k softmax
// weights are formed after the rounds, one per lane.  The kernel is bound by its VALU
// work: an exp and a division in every round cost a third of it (78 -> 60 us on the
// learner batch), and two tokens per wave share every reduction's instructions.
// On return lane ll < k of the token holds its ll-th choice in my_id (0x7FFFFFFF when every
// remaining logit is NaN) and its weight in my_w; the result is whether any lane of the wave
// met a NaN.  lane, sub, ll: the lane, its token within the wave, its lane within the token.
template <int NPL, int LPT>
__device__ __forceinline__ bool topk_token(const float *lg, bool valid, int E, int k, int flags, int lane, int sub,
                                           int ll, int &my_id, float &my_w) {
  float lv[NPL];
  float mx = -INFINITY;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = ll + LPT * i;
    lv[i] = -INFINITY;
    if (valid && e < E) {
      lv[i] = lg[e];
      nan |= lv[i] != lv[i];
      mx = fmaxf(mx, lv[i]);
    }
  }
  mx = wave_max_dpp<LPT>(mx);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = ll + LPT * i;
    if (valid && e < E) s += expf(lv[i] - mx);
  }
  s = wave_sum_dpp<LPT>(s);
  uint32_t taken = 0;
  my_id = 0;
  float my_v = -INFINITY;
  for (int j = 0; j < k; ++j) {
    float bv = -INFINITY;
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = ll + LPT * i;
      // ids of one lane increase with i, so the first of equal values has the lowest id
      if (e < E && !((taken >> i) & 1u) && (lv[i] > bv || (bi == 0x7FFFFFFF && lv[i] == bv))) { bv = lv[i]; bi = e; }
    }
    const float vmax = wave_max_dpp<LPT>(bv);
    const uint64_t cand = __ballot(bi != 0x7FFFFFFF && bv == vmax);
    int wid;
    if (LPT == 64) {
      if (cand == 0) {
        wid = 0x7FFFFFFF;  // every remaining logit is NaN
      } else if ((cand & (cand - 1)) == 0) {
        wid = __builtin_amdgcn_readlane(bi, (int)__builtin_ctzll(cand));
      } else {
        wid = wave_min_dpp(((cand >> lane) & 1) ? bi : 0x7FFFFFFF);
      }
    } else {
      // the two halves' candidate lanes: one each (the usual case) is read directly
      const uint32_t c0 = (uint32_t)cand, c1 = (uint32_t)(cand >> 32);
      if ((c0 & (c0 - 1)) == 0 && (c1 & (c1 - 1)) == 0) {
        const int w0 = c0 ? __builtin_amdgcn_readlane(bi, (int)__builtin_ctz(c0)) : 0x7FFFFFFF;
        const int w1 = c1 ? __builtin_amdgcn_readlane(bi, 32 + (int)__builtin_ctz(c1)) : 0x7FFFFFFF;
        wid = sub ? w1 : w0;
      } else {
        wid = wave_min_dpp<LPT>(((cand >> lane) & 1) ? bi : 0x7FFFFFFF);
      }
    }
    if (wid < E && (wid % LPT) == ll) taken |= 1u << (wid / LPT);
    if (ll == j) { my_id = wid; my_v = vmax; }
  }
  my_w = 0.0f;
  if (ll < k) my_w = expf(my_v - mx) / s;
  if (flags & NV4_RENORM) my_w = my_w / wave_sum_dpp<LPT>(my_w);  // lanes >= k hold 0
  return __ballot(nan) != 0;  // any lane's (each lane held only its own experts' logits)
}

}  // namespace nv4
