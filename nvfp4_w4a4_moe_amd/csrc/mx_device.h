// Device helpers of the MXFP4 kernels (OCP Microscaling v1.0: blocks of 32 E2M1 codes
// under one E8M0 scale).
#pragma once

#include "nv4_device.h"

namespace nv4 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kMxBlock = 32;
constexpr int kMxSegment = 128;  // NV4_MX_SEGMENT
constexpr uint32_t kMxNan = 255;

// E8M0 byte of a block from the bit pattern of its largest |v| (FP32; NaN and infinity
// order above every finite value).  floor(log2 A) is the exponent field - 127, so the OCP
// exponent floor(log2 A) - 2 has byte field - 2; a field below 2 clamps to byte 0.
// NV4_MX_CEIL takes the next power of two when A > 6 * 2^e, i.e. A's significand > 1.5.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax_bits, int ceil_rule) {
  const uint32_t field = amax_bits >> 23;
  if (field == 255u) return kMxNan;
  if (field < 2u) return 0u;
  return field - 2u + ((ceil_rule && (amax_bits & 0x7FFFFFu) > 0x400000u) ? 1u : 0u);
}

// 2^(byte - 127) as FP32 (2^-127 is subnormal; 255 maps to infinity)
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Four / two values to E2M1 codes of v / scale.  gfx950's converters round to nearest even,
// saturate at 6 and keep the sign; with a power-of-two scale (2^-127 included) every step
// before the rounding is exact.
template <int SEL>
__device__ __forceinline__ uint32_t mx_pack_f32(uint32_t old, float a, float b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, SEL);
}
template <int SEL>
__device__ __forceinline__ uint32_t mx_pack_bf16(uint32_t old, uint32_t pair, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2, pair), scale, SEL);
}

// max over the lanes i, i^1, i^2, i^3 of a quad, and over a 16-lane row
__device__ __forceinline__ uint32_t quad_umax(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));  // quad_perm [1,0,3,2]
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));  // quad_perm [2,3,0,1]
}
__device__ __forceinline__ uint32_t quad_or(uint32_t v) {
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false);
  return v | (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false);
}
// max over the 8 lanes of a half row: the quad's, then the half-row mirror
__device__ __forceinline__ uint32_t oct_umax(uint32_t v) {
  v = quad_umax(v);
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));
}

// largest |v| of the BF16 pairs of a dword, both halves at once
__device__ __forceinline__ uint32_t pk_umax16(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// Loads straight into LDS: lane i of the wave brings 16 (4) bytes at byte offset voff to
// dst + 16 i (4 i); an offset behind the buffer brings zeros.
// STREAM: a line that nobody else reads (non-temporal).
constexpr int kStream = 2;
typedef __attribute__((address_space(3))) void *mx_lds_ptr;
template <bool STREAM = false>
__device__ __forceinline__ void mx_dma16(const void *base, uint32_t bytes, uint8_t *dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000), (mx_lds_ptr)dst,
      16, voff, 0, 0, STREAM ? kStream : 0);
}
__device__ __forceinline__ void mx_dma4(const void *base, uint32_t bytes, uint8_t *dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000), (mx_lds_ptr)dst, 4,
      voff, 0, 0, 0);
}

// wait until at most N vector-memory operations of this wave are outstanding
template <int N>
__device__ __forceinline__ void mx_wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  asm volatile("" ::: "memory");
}
// wait for this wave's LDS operations (lgkmcnt(0) only)
__device__ __forceinline__ void mx_wait_lds() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
  asm volatile("" ::: "memory");
}

}  // namespace nv4
