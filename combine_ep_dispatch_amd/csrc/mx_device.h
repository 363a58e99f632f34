// MXFP4 device helpers (gfx950): 32 channels to E2M1 codes and one E8M0
// scale, and back.  Internal header: not part of the C ABI.
#pragma once

#include "ep_device.h"

namespace ep {

constexpr int kMxGroup = 32;  // channels per MXFP4 scale

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// (by value: a bit cast applied to a vector's element itself reads element 0)
__device__ __forceinline__ bf16x2 as_bf16x2(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }

// binary32 value of an E8M0 scale byte: 2^(b - 127), NaN for 255.
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
  const uint32_t bits = b << 23;
  return __uint_as_float(b == 0 ? 0x00400000u : (b == 255 ? 0x7FC00000u : bits));
}

// The group's scale byte for its largest magnitude (BF16 bits): e = floor(log2
// amax) - 2 is the BF16 exponent field minus 2; with that the largest
// magnitude lands in [4, 8) and saturates at 6.  255 for an infinity or a NaN.
__device__ __forceinline__ uint32_t mx_scale(uint32_t top) {
  const uint32_t code = static_cast<uint32_t>(max(static_cast<int>(top >> 7) - 2, 0));
  return top >= 0x7F80u ? 255u : (top == 0 ? 127u : code);
}

// Largest magnitude (BF16 bits; they order as numbers) of eight channels.
__device__ __forceinline__ uint32_t amax8_bf16(u32x4 a) {
  u16x2 m = {0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, a[j] & 0x7FFF7FFFu));
  return m.x > m.y ? m.x : m.y;
}

// Eight channels to E2M1 codes.  gfx950's convert divides by the scale, rounds
// to nearest even and saturates; x / 2^e is exact, so that one rounding is the
// only one (checked for every BF16 value at scales from 2^-127 to 2^125).
__device__ __forceinline__ uint32_t codes8_mxfp4(u32x4 a, uint32_t scale) {
  const float s = __uint_as_float(scale == 0 ? 0x00400000u : scale << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a[0]), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a[1]), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a[2]), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a[3]), s, 3);
  return scale == 255 ? 0u : w;
}

// A group's 32 channels in one lane (four 16-byte vectors of BF16 bits) ->
// 16 bytes of codes and the scale byte.
__device__ __forceinline__ u32x4 quantize32_mxfp4(const u32x4 (&a)[4], uint32_t& scale_byte) {
  scale_byte = mx_scale(max(max(amax8_bf16(a[0]), amax8_bf16(a[1])), max(amax8_bf16(a[2]), amax8_bf16(a[3]))));
  return u32x4{codes8_mxfp4(a[0], scale_byte), codes8_mxfp4(a[1], scale_byte), codes8_mxfp4(a[2], scale_byte),
               codes8_mxfp4(a[3], scale_byte)};
}

// The same for a group held by the 4 aligned lanes 4j..4j+3, 8 channels each
// (all 4 must call this): each lane's codes, and the scale byte in all.
__device__ __forceinline__ uint32_t quantize8_mxfp4(u32x4 a, uint32_t& scale_byte) {
  uint32_t m = amax8_bf16(a);
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0xB1, 0xF, 0xF, false)));
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x4E, 0xF, 0xF, false)));
  scale_byte = mx_scale(m);
  return codes8_mxfp4(a, scale_byte);
}

}  // namespace ep
