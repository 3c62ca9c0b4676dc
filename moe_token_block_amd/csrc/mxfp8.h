// MXFP8 block helpers: the power of two of a 32-element block and its E4M3
// bytes, shared by the pack and the activation checkpoint.
#pragma once

#include "common.h"

namespace mtb {

// The block exponent: the least e with a <= 448 * 2^e, within [-127, 127].
__device__ __forceinline__ int mx_exponent(float a) {
  if (!(a > 0.0f)) return 0;
  int sub = 0;
  if (a < 0x1p-126f) { a *= 0x1p64f; sub = 64; }
  int E = __builtin_amdgcn_frexp_expf(a) - 1 - sub;
  float m = __builtin_amdgcn_frexp_mantf(a) * 2.0f;
  int e = E - 8 + (m > 1.75f ? 1 : 0);  // least e with a <= 448 * 2^e
  return e < -127 ? -127 : (e > 127 ? 127 : e);
}

__device__ __forceinline__ uint32_t fp8x4_from_bf16(uint32_t w0, uint32_t w1, float scale) {
  i16x2 r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, w0), scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, w1), scale, true);
  return __builtin_bit_cast(uint32_t, r);
}

// Tiny blocks (e < -126): scale the inputs by 2^64 first so that the
// converter's power of two stays a normal float.
__device__ __forceinline__ uint32_t fp8x4_from_bf16_tiny(uint32_t w0, uint32_t w1, float scale) {
  i16x2 r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, bf16lo(w0) * 0x1p64f, bf16hi(w0) * 0x1p64f, scale, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, bf16lo(w1) * 0x1p64f, bf16hi(w1) * 0x1p64f, scale, true);
  return __builtin_bit_cast(uint32_t, r);
}

}  // namespace mtb
