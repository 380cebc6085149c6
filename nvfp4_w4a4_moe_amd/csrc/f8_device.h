// Device helpers of the FP8 kernels (OCP E4M3 codes with an FP32 scale for each block of 128).
#pragma once

#include "mx_device.h"
#include "topk_device.h"

namespace nv4 {

// S and G of a block from the bit pattern of its largest |v| (NaN and infinity order above
// every finite value): the factor before rounding and the scale that is kept.
//   448 / A: a quotient of 448 and FP32's smallest subnormal is 2^157, so S is capped at 2^126,
//   whose reciprocal is normal.
//   A power of two: 448 = 1.75 * 2^8, so with A = f * 2^e, 1 <= f < 2, the largest t with
//   A * 2^t <= 448 is 8 - e, or 7 - e where f > 1.75.  A subnormal A has e <= -127: t is capped.
struct F8Scale {
  float S, G;
  bool bad;
};
__device__ __forceinline__ F8Scale f8_scale(uint32_t amax_bits, int pow2) {
  F8Scale r;
  r.bad = amax_bits >= 0x7F800000u;
  if (pow2) {
    // exponent field of 2^t: 127 + 8 - (field - 127), at most that of 2^126
    const int t = 262 - (int)(amax_bits >> 23) - ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    const int s = amax_bits == 0 ? 127 : min(t, 253);
    r.S = __uint_as_float((uint32_t)s << 23);
    r.G = __uint_as_float((uint32_t)(254 - s) << 23);
  } else {
    r.S = amax_bits == 0 ? 1.0f : fminf(__fdiv_rn(448.0f, __uint_as_float(amax_bits)), 0x1p126f);
    r.G = __fdiv_rn(1.0f, r.S);
  }
  if (r.bad) {
    r.S = 0.0f;
    r.G = __uint_as_float(0x7FC00000u);
  }
  return r;
}

typedef int i32x4 __attribute__((ext_vector_type(4)));
// eight codes as FP16, exactly
__device__ __forceinline__ f16x8 f8_to_f16(int lo, int hi) {
  const f16x2 a = e4m3x2_to_f16(lo), b = e4m3x2_to_f16<true>(lo), c = e4m3x2_to_f16(hi), d = e4m3x2_to_f16<true>(hi);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// four values times S as E4M3 codes (gfx950's converter rounds to nearest even)
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d, float S) {
  const uint32_t lo = __builtin_amdgcn_cvt_pk_fp8_f32(a * S, b * S, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(c * S, d * S, lo, true);
}
__device__ __forceinline__ float bf16_lo(uint32_t pair) { return __uint_as_float(pair << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t pair) { return __uint_as_float(pair & 0xFFFF0000u); }

// 16 bytes of input: |v| maximum as FP32 bits
template <bool F32>
__device__ __forceinline__ uint32_t f8_amax(uint4 v) {
  if constexpr (F32) {
    const uint32_t m = 0x7FFFFFFFu;
    return max(max(v.x & m, v.y & m), max(v.z & m, v.w & m));
  } else {
    const uint32_t m = 0x7FFF7FFFu;
    const uint32_t p = pk_umax16(pk_umax16(v.x & m, v.y & m), pk_umax16(v.z & m, v.w & m));
    return max(p << 16, p & 0xFFFF0000u);
  }
}
// their codes: one dword (FP32: 4 values) or two (BF16: 8)
__device__ __forceinline__ uint32_t f8_pack_f32(uint4 v, float S) {
  return f8_pack4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w), S);
}
__device__ __forceinline__ uint2 f8_pack_bf16(uint4 v, float S) {
  return make_uint2(f8_pack4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y), S),
                    f8_pack4(bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w), S));
}

// max over a row of 16 lanes; over 32 lanes
__device__ __forceinline__ uint32_t row16_umax(uint32_t v) {
  v = oct_umax(v);
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));  // row_mirror
}
__device__ __forceinline__ uint32_t half_umax(uint32_t v) {
  v = row16_umax(v);
  const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max(s[0], s[1]);
}

}  // namespace nv4
