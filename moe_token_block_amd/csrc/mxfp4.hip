// BF16 rows to MXFP4 and back: E2M1 codes and one E8M0 scale per 32 values, the
// layout of the rowwise operand of ep_mxfp4_direct_receive.
#include "common.h"
#include "launch.h"
#include "stream.h"

namespace mtb {

// The block exponent: the least e with a <= 6 * 2^e, within [-127, 127].
__device__ __forceinline__ int mx4_exponent(float a) {
  if (!(a > 0.0f)) return 0;
  int sub = 0;
  if (a < 0x1p-126f) { a *= 0x1p64f; sub = 64; }
  const int E = __builtin_amdgcn_frexp_expf(a) - 1 - sub;
  const float m = __builtin_amdgcn_frexp_mantf(a) * 2.0f;
  const int e = E - 2 + (m > 1.5f ? 1 : 0);
  return e < -127 ? -127 : e;
}

// Eight values of a block as E2M1 codes, the first in the lowest nibble.  scale:
// 2^e, the values lifted by 2^64 with it where 2^e is no normal number.
__device__ __forceinline__ uint32_t e2m1x8(u32x4 v, float lift, float scale) {
  uint32_t o = fp4_pack2<0>(v[0], bf16lo(v[0]) * lift, bf16hi(v[0]) * lift, scale);  // the other bytes: overwritten next
  o = fp4_pack2<1>(o, bf16lo(v[1]) * lift, bf16hi(v[1]) * lift, scale);
  o = fp4_pack2<2>(o, bf16lo(v[2]) * lift, bf16hi(v[2]) * lift, scale);
  return fp4_pack2<3>(o, bf16lo(v[3]) * lift, bf16hi(v[3]) * lift, scale);
}

// One lane per 8 values, four to a block: every access of a wave is contiguous.  Bound
// by memory: 297 MB in 51 us at 16384 x 7168, 5.8 TB/s.  A block with an infinity or a NaN gets
// E8M0's NaN, so that every value of it reads back as one.
__global__ __launch_bounds__(256) void k_mxfp4_pack(const uint16_t* __restrict__ x, int64_t chunks,
                                                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;  // whole quads: chunks is a multiple of 4
  const u32x4 v = ld_once<u32x4>(x + 8 * i);
  const uint32_t m = quad_max(absmax_bf16x8(make_uint4(v[0], v[1], v[2], v[3])));
  const int e = mx4_exponent(__uint_as_float(m << 16));
  const bool tiny = e < -62;
  const uint32_t o = e2m1x8(v, tiny ? 0x1p64f : 1.0f, pow2f(tiny ? e + 64 : e));
  st_once(codes + 4 * i, o);
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)(m < 0x7F80u ? e + 127 : 255);
}

// One lane per 8 values: 297 MB in 55 us at 16384 x 7168, 5.4 TB/s.
__global__ __launch_bounds__(256) void k_mxfp4_unpack(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, int64_t chunks,
                                                      uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const uint32_t w = ld_once<uint32_t>(codes + 4 * i);
  const float s = e8m0(scales[i >> 2]);
  const f32x2 a = fp4_unpack2<0>(w, 1.0f), b = fp4_unpack2<1>(w, 1.0f), c = fp4_unpack2<2>(w, 1.0f),
              d = fp4_unpack2<3>(w, 1.0f);
  const u32x4 o = {bf16pair(a[0] * s, a[1] * s), bf16pair(b[0] * s, b[1] * s), bf16pair(c[0] * s, c[1] * s),
                   bf16pair(d[0] * s, d[1] * s)};
  st_once(out + 8 * i, o);
}

}  // namespace mtb

using namespace mtb;

namespace {
int32_t check(int64_t rows, int64_t hidden) {
  if (rows < 0 || hidden <= 0 || hidden % 32 != 0) return EP_ERR_SHAPE;
  // one lane per 8 values, fewer than 2^31 lanes: a grid has less than 2^32
  if (hidden > (1 << 24) || rows > (((int64_t)1 << 34) - 1) / hidden) return EP_ERR_RANGE;
  return EP_OK;
}
}  // namespace

MTB_EXPORT int32_t ep_mxfp4_pack(const uint16_t* x, int64_t rows, int64_t hidden, uint8_t* codes, uint8_t* scales,
                                 void* stream) {
  const int32_t st = check(rows, hidden);
  if (st != EP_OK) return st;
  if (rows == 0) return EP_OK;
  if (!x || !codes || !scales) return EP_ERR_NULL;
  const int64_t chunks = rows * (hidden / 8);
  hipLaunchKernelGGL(k_mxfp4_pack, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, (hipStream_t)stream, x, chunks,
                     codes, scales);
  return launch_status();
}

MTB_EXPORT int32_t ep_mxfp4_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t hidden, uint16_t* out,
                                   void* stream) {
  const int32_t st = check(rows, hidden);
  if (st != EP_OK) return st;
  if (rows == 0) return EP_OK;
  if (!codes || !scales || !out) return EP_ERR_NULL;
  const int64_t chunks = rows * (hidden / 8);
  hipLaunchKernelGGL(k_mxfp4_unpack, dim3((unsigned)((chunks + 255) / 256)), dim3(256), 0, (hipStream_t)stream, codes,
                     scales, chunks, out);
  return launch_status();
}
