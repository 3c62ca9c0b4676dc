// Helpers of the kernels that pass over rows once: accesses past the caches at any
// byte address, and the blocks of 32 that a lane quad shares.
#pragma once

#include "common.h"

namespace mtb {

template <typename T>
__device__ __forceinline__ T ld_once(const void* p) {
  typedef T any __attribute__((aligned(1)));
  return __builtin_nontemporal_load(reinterpret_cast<const any*>(p));
}
template <typename T>
__device__ __forceinline__ void st_once(void* p, T v) {
  typedef T any __attribute__((aligned(1)));
  __builtin_nontemporal_store(v, reinterpret_cast<any*>(p));
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// E8M0 byte -> the power of two it stands for (255: NaN).
__device__ __forceinline__ float e8m0(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(1.0f, (int)b - 127);
}

__device__ __forceinline__ u32x4 pack8(const float* v) {
  return u32x4{bf16pair(v[0], v[1]), bf16pair(v[2], v[3]), bf16pair(v[4], v[5]), bf16pair(v[6], v[7])};
}

// The largest of a lane quad.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));  // lane ^ 1
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));  // lane ^ 2
}

}  // namespace mtb
