// Matrix operand types, and the exchange within a lane quad that turns coalesced
// loads (four lanes on 64 contiguous bytes of a row) into the matrix instructions'
// order (a lane per row).
#pragma once

#include "common.h"

namespace mtb {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The neighbour's value (lane ^ 1 or lane ^ 2) where `take`, else own.
template <int CTRL>
__device__ __forceinline__ uint32_t quad_mix(bool take, uint32_t other, uint32_t own) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)other, CTRL, 0xF, 0xF, true);
  return take ? o : own;
}

// c[j] of lane i of a quad becomes c[i] of lane j.
__device__ __forceinline__ void quad_transpose(u32x4* c) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
  for (int p = 0; p < 4; p += 2)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = c[p][w], y = c[p + 1][w];
      c[p][w] = quad_mix<0xB1>(odd, y, x);
      c[p + 1][w] = quad_mix<0xB1>(!odd, x, y);
    }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = c[p][w], y = c[p + 2][w];
      c[p][w] = quad_mix<0x4E>(high, y, x);
      c[p + 2][w] = quad_mix<0x4E>(!high, x, y);
    }
}

}  // namespace mtb
