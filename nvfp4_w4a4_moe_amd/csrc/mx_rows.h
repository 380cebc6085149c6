// MXFP4 quantisation along rows, shared by the quantiser and the few-token layer.
//
// 16 lanes take one unit: 128 elements of a row, four blocks, one dword of scale bytes; each
// lane 8 of them.  |v| maxima are taken on the bit patterns (integers order as the magnitudes
// do, with NaN and infinity on top), two BF16 at a time.
#pragma once

#include "mx_device.h"

namespace nv4 {

// 8 BF16 (one uint4): |v| maximum as FP32 bits, and their codes
__device__ __forceinline__ uint32_t mx_amax8_bf16(uint4 v) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t p = pk_umax16(pk_umax16(v.x & m, v.y & m), pk_umax16(v.z & m, v.w & m));
  return max(p << 16, p & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t mx_pack8_bf16(uint4 v, float s) {
  uint32_t c = mx_pack_bf16<0>(0u, v.x, s);
  c = mx_pack_bf16<1>(c, v.y, s);
  c = mx_pack_bf16<2>(c, v.z, s);
  return mx_pack_bf16<3>(c, v.w, s);
}
// 4 FP32 (one uint4)
__device__ __forceinline__ uint32_t mx_amax4_f32(uint4 v) {
  const uint32_t m = 0x7FFFFFFFu;
  return max(max(v.x & m, v.y & m), max(v.z & m, v.w & m));
}
__device__ __forceinline__ uint32_t mx_pack4_f32(uint4 v, float s) {
  const uint32_t c = mx_pack_f32<0>(0u, __uint_as_float(v.x), __uint_as_float(v.y), s);
  return mx_pack_f32<1>(c, __uint_as_float(v.z), __uint_as_float(v.w), s);
}

// A lane's 8 elements of a unit, already loaded (zeros behind K): its codes, and in every lane
// the unit's four scale bytes.  Lanes behind K hold zeros, whose bytes are the zeros a scale
// row is padded with.  Returns whether the lane's block holds a NaN or infinity.  Whole wave.
template <bool F32>
__device__ __forceinline__ bool mx_unit(const uint4 (&v)[F32 ? 2 : 1], int l16, int ceil_rule, uint32_t &codes,
                                        uint32_t &bytes) {
  uint32_t m;
  if constexpr (F32) m = max(mx_amax4_f32(v[0]), mx_amax4_f32(v[1]));
  else m = mx_amax8_bf16(v[0]);
  m = quad_umax(m);
  const uint32_t byte = mx_scale_byte(m, ceil_rule);
  const float s = mx_scale_value(byte);
  if constexpr (F32) codes = mx_pack4_f32(v[0], s) | (mx_pack4_f32(v[1], s) << 16);
  else codes = mx_pack8_bf16(v[0], s);
  if (byte == kMxNan) codes = 0u;
  // the four blocks' bytes meet in one dword (lanes 0, 4, 8, 12 of the 16)
  uint32_t d = byte << (8 * (l16 >> 2));
  d |= (uint32_t)__builtin_amdgcn_mov_dpp((int)d, 0x124, 0xF, 0xF, false);  // row_ror:4
  d |= (uint32_t)__builtin_amdgcn_mov_dpp((int)d, 0x128, 0xF, 0xF, false);  // row_ror:8
  bytes = d;
  return byte == kMxNan;
}

}  // namespace nv4
