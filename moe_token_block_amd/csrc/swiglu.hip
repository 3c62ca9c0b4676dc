// SwiGLU with its pre-activation kept in 8 bits for the backward pass: MXFP8
// (E4M3 bytes and one E8M0 scale per 32 columns, the format of the pack), 33
// bytes per 32 values instead of 64, written while the values are in registers
// and decoded in registers by the gradient.
#include "common.h"
#include "launch.h"
#include "mxfp8.h"

namespace mtb {

// E8M0 byte -> the power of two it stands for (255: NaN).
__device__ __forceinline__ float e8m0(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(1.0f, (int)b - 127);
}

// Eight E4M3 bytes times a power of two: exact in FP32.
__device__ __forceinline__ void decode_e4m3x8(uint2 v, float s, float* o) {
  o[0] = __builtin_amdgcn_cvt_f32_fp8((int)v.x, 0) * s;
  o[1] = __builtin_amdgcn_cvt_f32_fp8((int)v.x, 1) * s;
  o[2] = __builtin_amdgcn_cvt_f32_fp8((int)v.x, 2) * s;
  o[3] = __builtin_amdgcn_cvt_f32_fp8((int)v.x, 3) * s;
  o[4] = __builtin_amdgcn_cvt_f32_fp8((int)v.y, 0) * s;
  o[5] = __builtin_amdgcn_cvt_f32_fp8((int)v.y, 1) * s;
  o[6] = __builtin_amdgcn_cvt_f32_fp8((int)v.y, 2) * s;
  o[7] = __builtin_amdgcn_cvt_f32_fp8((int)v.y, 3) * s;
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(bf16pair(v[0], v[1]), bf16pair(v[2], v[3]), bf16pair(v[4], v[5]), bf16pair(v[6], v[7]));
}

__device__ __forceinline__ float silu(float a, float& s) {
  s = __builtin_amdgcn_rcpf(1.0f + __expf(-a));
  return a * s;
}

// One lane per 32-column block of a and the matching block of b.
__global__ __launch_bounds__(256) void k_swiglu_checkpoint(const uint16_t* __restrict__ preact, int64_t blocks, int nb,
                                                           uint16_t* __restrict__ act, uint8_t* __restrict__ data,
                                                           uint8_t* __restrict__ scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= blocks) return;
  const int64_t row = i / nb;
  const int c = (int)(i % nb);
  const size_t ba = (size_t)row * 2 * nb + c;  // block index of a within [T, 2F/32]; b's is ba + nb
  uint4 q[2][4];
  for (int h = 0; h < 2; ++h) {
    const size_t blk = ba + (h ? nb : 0);
    const uint16_t* p = preact + 32 * blk;
    uint32_t m = 0;
    for (int u = 0; u < 4; ++u) {
      q[h][u] = ld_any<uint4>(p + 8 * u);
      m = max(m, absmax_bf16x8(q[h][u]));
    }
    const int e = mx_exponent(__uint_as_float(m << 16));
    uint8_t* d = data + 32 * blk;
    for (int u = 0; u < 4; ++u)
      st_any(d + 8 * u, e >= -126 ? make_uint2(fp8x4_from_bf16(q[h][u].x, q[h][u].y, pow2f(e)),
                                               fp8x4_from_bf16(q[h][u].z, q[h][u].w, pow2f(e)))
                                  : make_uint2(fp8x4_from_bf16_tiny(q[h][u].x, q[h][u].y, pow2f(e + 64)),
                                               fp8x4_from_bf16_tiny(q[h][u].z, q[h][u].w, pow2f(e + 64))));
    scales[blk] = (uint8_t)(e + 127);
  }
  uint16_t* o = act + 32 * (size_t)i;
  for (int u = 0; u < 4; ++u) {
    const uint32_t a[4] = {q[0][u].x, q[0][u].y, q[0][u].z, q[0][u].w};
    const uint32_t b[4] = {q[1][u].x, q[1][u].y, q[1][u].z, q[1][u].w};
    float y[8], s;
    for (int v = 0; v < 4; ++v) {
      y[2 * v] = silu(bf16lo(a[v]), s) * bf16lo(b[v]);
      y[2 * v + 1] = silu(bf16hi(a[v]), s) * bf16hi(b[v]);
    }
    st_any(o + 8 * u, pack8(y));
  }
}

// One lane per 8 columns of a, b and dy.
__global__ __launch_bounds__(256) void k_dswiglu_checkpoint(const uint8_t* __restrict__ data,
                                                            const uint8_t* __restrict__ scales,
                                                            const uint16_t* __restrict__ dy, int64_t chunks, int nch,
                                                            uint16_t* __restrict__ dx, uint16_t* __restrict__ act) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const int64_t row = i / nch;
  const size_t ca = (size_t)(i + row * nch), cb = ca + nch;  // chunks of a and b within [T, 2F/8]
  float a[8], b[8], da[8], db[8], y[8];
  decode_e4m3x8(ld_any<uint2>(data + 8 * ca), e8m0(scales[ca >> 2]), a);
  decode_e4m3x8(ld_any<uint2>(data + 8 * cb), e8m0(scales[cb >> 2]), b);
  const uint4 g = ld_any<uint4>(dy + 8 * i);
  const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
  for (int u = 0; u < 8; ++u) {
    const float d = u & 1 ? bf16hi(gw[u >> 1]) : bf16lo(gw[u >> 1]);
    float s;
    const float sa = silu(a[u], s);
    da[u] = d * b[u] * s * (1.0f + a[u] * (1.0f - s));
    db[u] = d * sa;
    y[u] = sa * b[u];
  }
  st_any(dx + 8 * ca, pack8(da));
  st_any(dx + 8 * cb, pack8(db));
  if (act) st_any(act + 8 * i, pack8(y));
}

// MXFP8 -> BF16, one lane per 8 elements.
__global__ __launch_bounds__(256) void k_mxfp8_unpack(const uint8_t* __restrict__ data,
                                                      const uint8_t* __restrict__ scales, int64_t chunks,
                                                      uint16_t* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  float v[8];
  decode_e4m3x8(ld_any<uint2>(data + 8 * i), e8m0(scales[i >> 2]), v);
  st_any(out + 8 * i, pack8(v));
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
  const int64_t blocks = tokens * (ffn / 32);
  hipLaunchKernelGGL(k_swiglu_checkpoint, dim3(grid_of(blocks)), dim3(256), 0, (hipStream_t)stream, preact, blocks,
                     (int)(ffn / 32), act, data, scales);
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
                     chunks, (int)(ffn / 8), dx, act);
  return launch_status();
}

MTB_EXPORT int32_t ep_mxfp8_unpack(const uint8_t* data, const uint8_t* scales, int64_t rows, int64_t hidden,
                                   uint16_t* out, void* stream) {
  const int32_t st = check_sizes(rows, hidden);
  if (st != EP_OK) return st;
  if (rows == 0) return EP_OK;
  if (!data || !scales || !out) return EP_ERR_NULL;
  const int64_t chunks = rows * (hidden / 8);
  hipLaunchKernelGGL(k_mxfp8_unpack, dim3(grid_of(chunks)), dim3(256), 0, (hipStream_t)stream, data, scales, chunks,
                     out);
  return launch_status();
}
