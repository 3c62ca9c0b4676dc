// SwiGLU with its pre-activation kept in 8 bits for the backward pass: MXFP8
// (E4M3 bytes and one E8M0 scale per 32 columns, the format of the pack), 33
// bytes per 32 values instead of 64, written while the values are in registers
// and decoded in registers by the gradient.
#include "common.h"
#include "launch.h"
#include "mxfp8.h"
#include "stream.h"

// Every value here is read or written once: accesses past the caches (14841 x 2048:
// the forward 45 -> 41 us, forward and read-back 72.2 -> 71.5, the gradient 54.7 ->
// 50.0).
namespace mtb {

// Eight E4M3 bytes times a power of two: exact in FP32.
__device__ __forceinline__ void decode_e4m3x8(u32x2 v, float s, float* o) {
  o[0] = __builtin_amdgcn_cvt_f32_fp8((int)v.x, 0) * s;
  o[1] = __builtin_amdgcn_cvt_f32_fp8((int)v.x, 1) * s;
  o[2] = __builtin_amdgcn_cvt_f32_fp8((int)v.x, 2) * s;
  o[3] = __builtin_amdgcn_cvt_f32_fp8((int)v.x, 3) * s;
  o[4] = __builtin_amdgcn_cvt_f32_fp8((int)v.y, 0) * s;
  o[5] = __builtin_amdgcn_cvt_f32_fp8((int)v.y, 1) * s;
  o[6] = __builtin_amdgcn_cvt_f32_fp8((int)v.y, 2) * s;
  o[7] = __builtin_amdgcn_cvt_f32_fp8((int)v.y, 3) * s;
}

__device__ __forceinline__ float silu(float a, float& s) {
  s = __builtin_amdgcn_rcpf(1.0f + __expf(-a));
  return a * s;
}

// Eight values of a 32-value block, whose largest magnitude is m, as E4M3 bytes;
// the block's scale byte.  A block with an infinity or a NaN gets E8M0's NaN: its
// exponent would be made up and the infinity kept as a finite value, so that the
// gradient hid what the output shows.
__device__ __forceinline__ u32x2 quantize8(u32x4 v, uint32_t m, uint8_t& scale) {
  const int e = mx_exponent(__uint_as_float(m << 16));
  scale = (uint8_t)(m < 0x7F80u ? e + 127 : 255);
  if (e >= -126) {
    const float s = pow2f(e);
    return u32x2{fp8x4_from_bf16(v[0], v[1], s), fp8x4_from_bf16(v[2], v[3], s)};
  }
  const float s = pow2f(e + 64);
  return u32x2{fp8x4_from_bf16_tiny(v[0], v[1], s), fp8x4_from_bf16_tiny(v[2], v[3], s)};
}

// One lane per 8 columns of a and of b: four neighbouring lanes share a block of
// 32, and every access of a wave is contiguous (a lane per whole block, 64 bytes
// apart: 66 us).  Bound by memory: 245 MB in 41 us at 14841 x 2048, 6.0 TB/s.
__global__ __launch_bounds__(256) void k_swiglu_checkpoint(const uint16_t* __restrict__ preact, uint32_t chunks,
                                                           uint32_t nch, uint16_t* __restrict__ act,
                                                           uint8_t* __restrict__ data, uint8_t* __restrict__ scales) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= chunks) return;  // whole quads: chunks is a multiple of 4
  const size_t ca = (size_t)i + (size_t)(i / nch) * nch, cb = ca + nch;  // chunks of a and b within [T, 2F/8]
  const u32x4 a = ld_once<u32x4>(preact + 8 * ca), b = ld_once<u32x4>(preact + 8 * cb);
  uint8_t ea, eb;
  const u32x2 da = quantize8(a, quad_max(absmax_bf16x8(make_uint4(a[0], a[1], a[2], a[3]))), ea);
  const u32x2 db = quantize8(b, quad_max(absmax_bf16x8(make_uint4(b[0], b[1], b[2], b[3]))), eb);
  st_once(data + 8 * ca, da);
  st_once(data + 8 * cb, db);
  if ((i & 3) == 0) {
    scales[ca >> 2] = ea;
    scales[cb >> 2] = eb;
  }
  u32x4 y;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    float s;
    y[v] = bf16pair(silu(bf16lo(a[v]), s) * bf16lo(b[v]), silu(bf16hi(a[v]), s) * bf16hi(b[v]));
  }
  st_once(act + 8 * (size_t)i, y);
}

// One lane per 8 columns of a, b and dy.  Bound by memory: 306 MB in 49 us at
// 14841 x 2048, 6.2 TB/s; the exponential and reciprocal of a value serve da, db
// and act.
__global__ __launch_bounds__(256) void k_dswiglu_checkpoint(const uint8_t* __restrict__ data,
                                                            const uint8_t* __restrict__ scales,
                                                            const uint16_t* __restrict__ dy, uint32_t chunks, uint32_t nch,
                                                            uint16_t* __restrict__ dx, uint16_t* __restrict__ act) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= chunks) return;
  const size_t ca = (size_t)i + (size_t)(i / nch) * nch, cb = ca + nch;  // chunks of a and b within [T, 2F/8]
  float a[8], b[8], da[8], db[8], y[8];
  decode_e4m3x8(ld_once<u32x2>(data + 8 * ca), e8m0(scales[ca >> 2]), a);
  decode_e4m3x8(ld_once<u32x2>(data + 8 * cb), e8m0(scales[cb >> 2]), b);
  const u32x4 gw = ld_once<u32x4>(dy + 8 * (size_t)i);
  for (int u = 0; u < 8; ++u) {
    const float d = u & 1 ? bf16hi(gw[u >> 1]) : bf16lo(gw[u >> 1]);
    float s;
    const float sa = silu(a[u], s);
    da[u] = d * b[u] * s * (1.0f + a[u] * (1.0f - s));
    db[u] = d * sa;
    y[u] = sa * b[u];
  }
  st_once(dx + 8 * ca, pack8(da));
  st_once(dx + 8 * cb, pack8(db));
  if (act) st_once(act + 8 * (size_t)i, pack8(y));
}

// MXFP8 -> BF16, one lane per 8 elements: 184 MB in 28-31 us at 14841 x 4096.
__global__ __launch_bounds__(256) void k_mxfp8_unpack(const uint8_t* __restrict__ data,
                                                      const uint8_t* __restrict__ scales, uint32_t chunks,
                                                      uint16_t* __restrict__ out) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= chunks) return;
  float v[8];
  decode_e4m3x8(ld_once<u32x2>(data + 8 * (size_t)i), e8m0(scales[i >> 2]), v);
  st_once(out + 8 * (size_t)i, pack8(v));
}

}  // namespace mtb

using namespace mtb;

namespace {
// tokens * width stays below 2^34, so that a grid of one lane per 8 values fits.
int32_t check_sizes(int64_t tokens, int64_t width) {
  if (tokens < 0 || width <= 0 || width % 32 != 0) return EP_ERR_SHAPE;
  if (width > (1 << 24) || tokens > (((int64_t)1 << 34) - 1) / width) return EP_ERR_RANGE;
  return EP_OK;
}
unsigned grid_of(int64_t lanes) { return (unsigned)((lanes + 255) / 256); }
}  // namespace

MTB_EXPORT int32_t swiglu_mxfp8_checkpoint(const uint16_t* preact, int64_t tokens, int64_t ffn, uint16_t* act,
                                           uint8_t* data, uint8_t* scales, void* stream) {
  const int32_t st = check_sizes(tokens, ffn);
  if (st != EP_OK) return st;
  if (tokens == 0) return EP_OK;
  if (!preact || !act || !data || !scales) return EP_ERR_NULL;
  const int64_t chunks = tokens * (ffn / 8);
  hipLaunchKernelGGL(k_swiglu_checkpoint, dim3(grid_of(chunks)), dim3(256), 0, (hipStream_t)stream, preact,
                     (uint32_t)chunks, (uint32_t)(ffn / 8), act, data, scales);
  return launch_status();
}

MTB_EXPORT int32_t dswiglu_mxfp8_checkpoint(const uint8_t* data, const uint8_t* scales, const uint16_t* dy,
                                            int64_t tokens, int64_t ffn, uint16_t* dx, uint16_t* act, void* stream) {
  const int32_t st = check_sizes(tokens, ffn);
  if (st != EP_OK) return st;
  if (tokens == 0) return EP_OK;
  if (!data || !scales || !dy || !dx) return EP_ERR_NULL;
  const int64_t chunks = tokens * (ffn / 8);
  hipLaunchKernelGGL(k_dswiglu_checkpoint, dim3(grid_of(chunks)), dim3(256), 0, (hipStream_t)stream, data, scales, dy,
                     (uint32_t)chunks, (uint32_t)(ffn / 8), dx, act);
  return launch_status();
}

MTB_EXPORT int32_t ep_mxfp8_unpack(const uint8_t* data, const uint8_t* scales, int64_t rows, int64_t hidden,
                                   uint16_t* out, void* stream) {
  const int32_t st = check_sizes(rows, hidden);
  if (st != EP_OK) return st;
  if (rows == 0) return EP_OK;
  if (!data || !scales || !out) return EP_ERR_NULL;
  const int64_t chunks = rows * (hidden / 8);
  hipLaunchKernelGGL(k_mxfp8_unpack, dim3(grid_of(chunks)), dim3(256), 0, (hipStream_t)stream, data, scales,
                     (uint32_t)chunks, out);
  return launch_status();
}
