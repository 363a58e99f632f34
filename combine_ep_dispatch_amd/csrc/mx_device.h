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

// The 32 channels of one group, held by one lane as BF16 bits (four 16-byte
// vectors, channel order) -> 16 bytes of E2M1 codes and the scale byte.
// e = floor(log2 amax) - 2 is the BF16 exponent field of amax, minus 2: with
// that the largest magnitude lands in [4, 8) and saturates at 6.  BF16
// magnitudes order as their bit patterns, so amax is an integer maximum.
// gfx950's convert divides by the scale, rounds to nearest even and
// saturates; x / 2^e is exact, so that one rounding is the only one (checked
// for every BF16 value at scales from 2^-127 to 2^125).
__device__ __forceinline__ u32x4 quantize32_mxfp4(const u32x4 (&a)[4], uint32_t& scale_byte) {
  u16x2 m = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, a[i][j] & 0x7FFF7FFFu));
  const uint32_t top = m.x > m.y ? m.x : m.y;
  const int e = static_cast<int>(top >> 7);
  uint32_t code = static_cast<uint32_t>(max(e - 2, 0));
  code = top == 0 ? 127u : code;
  const float s = __uint_as_float(code == 0 ? 0x00400000u : code << 23);
  u32x4 q;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a[i][0]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a[i][1]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a[i][2]), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, as_bf16x2(a[i][3]), s, 3);
    q[i] = w;
  }
  const bool finite = top < 0x7F80u;
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = finite ? q[i] : 0u;
  scale_byte = finite ? code : 255u;
  return q;
}

}  // namespace ep
