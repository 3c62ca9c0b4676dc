// BF16 token rows to their experts and back (P2, review comments: one routing
// serves the dispatch and the combine): the copy into grouped rows, the
// weighted sum of a token's expert rows, and the gradients of both.
#include "common.h"
#include "launch.h"

namespace mtb {

// Eight BF16 values: a row of an odd width starts at any 2-byte boundary.
__device__ __forceinline__ u32x4 ld8(const uint16_t* p) { return ld_any<u32x4>(p); }
__device__ __forceinline__ void st8(uint16_t* p, u32x4 v) { st_any(p, v); }

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f32_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// out[g] = x[src_row[g]], zeros for padding: one wave per grouped row.
__global__ __launch_bounds__(256) void k_bf16_dispatch(const uint16_t* __restrict__ x, int tokens, int H,
                                                       const int32_t* __restrict__ src_row, int r_cap,
                                                       uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int g = (int)(blockIdx.x * 4u + (threadIdx.x >> 6));
  if (g >= r_cap) return;
  const int src = src_row[g];
  const bool pad = src < 0 || src >= tokens;
  const uint16_t* p = x + (size_t)(pad ? 0 : src) * H;
  uint16_t* o = out + (size_t)g * H;
  const int nch = H >> 3;
  for (int c = lane; c < nch; c += 64) st8(o + 8 * c, pad ? u32x4{0u, 0u, 0u, 0u} : ld8(p + 8 * c));
  const int i = 8 * nch + lane;
  if (i < H) o[i] = pad ? (uint16_t)0 : p[i];
}

// out[t] = sum over slots j, in order, of w[t, j] * rows[dst_row[t, j]], in
// FP32, rounded once.  One wave per token and 512 columns.
__global__ __launch_bounds__(64) void k_bf16_combine(const uint16_t* __restrict__ rows, int r_cap, int H, int k,
                                                     const int32_t* __restrict__ dst_row,
                                                     const float* __restrict__ weights, uint16_t* __restrict__ out) {
  const int t = blockIdx.x, lane = threadIdx.x;
  const int32_t* d = dst_row + (size_t)t * k;
  const float* w = weights ? weights + (size_t)t * k : nullptr;
  const int c0 = 8 * (int)(blockIdx.y * 64u + lane);
  if (c0 >= H) return;
  const int n = min(8, H - c0);
  float acc[8] = {};
  for (int j = 0; j < k; ++j) {
    const int g = d[j];
    if ((uint32_t)g >= (uint32_t)r_cap) continue;
    const float wj = w ? w[j] : 1.0f;
    const uint16_t* p = rows + (size_t)g * H + c0;
    for (int i = 0; i < n; ++i) acc[i] = __builtin_fmaf(wj, bf16_f32(p[i]), acc[i]);
  }
  uint16_t* o = out + (size_t)t * H + c0;
  for (int i = 0; i < n; ++i) o[i] = f32_bf16(acc[i]);
}

// Gradients of the combine: drows[dst] = w * dout, dw = <dout, rows[dst]>.
// One wave per token; waves past the tokens clear the padding rows.
__global__ __launch_bounds__(64) void k_bf16_combine_bwd(const uint16_t* __restrict__ dout,
                                                         const uint16_t* __restrict__ rows, int T, int H, int k,
                                                         int r_cap, const int32_t* __restrict__ dst_row,
                                                         const int32_t* __restrict__ src_row,
                                                         const float* __restrict__ weights,
                                                         uint16_t* __restrict__ drows, float* __restrict__ dweights) {
  const int lane = threadIdx.x;
  if ((int)blockIdx.x >= T) {
    const int g = (int)blockIdx.x - T;
    const int s = src_row[g];
    if (s >= 0 && s < T) return;
    for (int c = lane; c < H; c += 64) drows[(size_t)g * H + c] = 0;
    return;
  }
  const int t = blockIdx.x;
  const uint16_t* d = dout + (size_t)t * H;
  for (int j = 0; j < k; ++j) {
    const int g = dst_row[(size_t)t * k + j];
    float dot = 0.0f;
    if ((uint32_t)g < (uint32_t)r_cap) {
      const float w = weights[(size_t)t * k + j];
      const uint16_t* y = rows + (size_t)g * H;
      uint16_t* o = drows + (size_t)g * H;
      for (int c = lane; c < H; c += 64) {
        const float v = bf16_f32(d[c]);
        dot = __builtin_fmaf(v, bf16_f32(y[c]), dot);
        o[c] = f32_bf16(w * v);
      }
#pragma unroll
      for (int s = 32; s > 0; s >>= 1) dot += __shfl_xor(dot, s, kWave);
    }
    if (lane == 0) dweights[(size_t)t * k + j] = dot;
  }
}

}  // namespace mtb

using namespace mtb;

namespace {
// Sizes every call here checks first: hidden from 1 to 2^20; tokens and grouped
// rows up to 2^25, so that a wave for each fits one grid.
int32_t check_sizes(int64_t tokens, int64_t hidden, int64_t top_k, int64_t r_cap) {
  if (tokens < 0 || hidden <= 0 || top_k < 1 || r_cap < 0) return EP_ERR_SHAPE;
  if (tokens >= (1 << 25) || r_cap >= (1 << 25) || hidden > (1 << 20) || top_k > 1024 || tokens * top_k > INT32_MAX / 4)
    return EP_ERR_RANGE;
  return EP_OK;
}
}  // namespace

MTB_EXPORT int32_t ep_bf16_dispatch(const uint16_t* x, int64_t tokens, int64_t hidden, int64_t r_cap,
                                    const int32_t* src_row, uint16_t* out, void* stream) {
  const int32_t st = check_sizes(tokens, hidden, 1, r_cap);
  if (st != EP_OK) return st;
  if (r_cap == 0) return EP_OK;
  if (!src_row || !out || (tokens > 0 && !x)) return EP_ERR_NULL;
  hipLaunchKernelGGL(k_bf16_dispatch, dim3((unsigned)((r_cap + 3) / 4)), dim3(256), 0, (hipStream_t)stream, x,
                     (int)tokens, (int)hidden, src_row, (int)r_cap, out);
  return launch_status();
}

MTB_EXPORT int32_t ep_bf16_combine(const uint16_t* rows, int64_t r_cap, int64_t hidden, int64_t tokens,
                                   int64_t top_k, const int32_t* dst_row, const float* weights, uint16_t* out,
                                   void* stream) {
  const int32_t st = check_sizes(tokens, hidden, top_k, r_cap);
  if (st != EP_OK) return st;
  if (tokens == 0) return EP_OK;
  if (!dst_row || !out || (r_cap > 0 && !rows)) return EP_ERR_NULL;
  hipLaunchKernelGGL(k_bf16_combine, dim3((unsigned)tokens, (unsigned)((hidden + 511) / 512)), dim3(64), 0,
                     (hipStream_t)stream, rows, (int)r_cap, (int)hidden, (int)top_k, dst_row, weights, out);
  return launch_status();
}

MTB_EXPORT int32_t ep_bf16_combine_bwd(const uint16_t* dout, const uint16_t* rows, int64_t tokens, int64_t hidden,
                                       int64_t top_k, int64_t r_cap, const int32_t* dst_row, const int32_t* src_row,
                                       const float* weights, uint16_t* drows, float* dweights, void* stream) {
  const int32_t st = check_sizes(tokens, hidden, top_k, r_cap);
  if (st != EP_OK) return st;
  if (tokens == 0 && r_cap == 0) return EP_OK;
  if (r_cap > 0 && (!rows || !drows || !src_row)) return EP_ERR_NULL;
  if (tokens > 0 && (!dout || !dst_row || !weights || !dweights)) return EP_ERR_NULL;
  hipLaunchKernelGGL(k_bf16_combine_bwd, dim3((unsigned)(tokens + r_cap)), dim3(64), 0, (hipStream_t)stream, dout,
                     rows, (int)tokens, (int)hidden, (int)top_k, (int)r_cap, dst_row, src_row, weights, drows,
                     dweights);
  return launch_status();
}
