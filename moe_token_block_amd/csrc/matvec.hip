// Few token rows times the NVFP4 weights of their experts: the products of an
// expert layer that serves single tokens, where each weight byte is used once
// or a few times and the time is that of reading it.
#include "common.h"
#include "launch.h"

namespace mtb {

__device__ __forceinline__ float dot_row(const uint16_t* __restrict__ x, const uint8_t* __restrict__ w, int K) {
  const int lane = threadIdx.x & 63;
  const float t = ld_any<float>(w + K / 2 + K / 16);
  float acc = 0.0f;
  for (int b = lane; b < K / 16; b += 64) {  // one 16-element block per lane
    // the whole weight before the product: a sum of code * x alone could pass
    // FP32's range where t brings it back
    const float s = e4m3_decode(w[K / 2 + b]) * t;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t cw = ld_any<uint32_t>(w + 8 * b + 4 * h);
      const f32x2 p[4] = {fp4_unpack2<0>(cw, 1.0f), fp4_unpack2<1>(cw, 1.0f), fp4_unpack2<2>(cw, 1.0f),
                          fp4_unpack2<3>(cw, 1.0f)};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xv = __uint_as_float((uint32_t)x[16 * b + 8 * h + i] << 16);
        acc = __builtin_fmaf(p[i >> 1][i & 1] * s, xv, acc);
      }
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) acc += __shfl_xor(acc, o, kWave);
  return acc;
}

// One wave per entry (t, j) and output column.
template <typename IDX>
__global__ __launch_bounds__(64) void k_nvfp4_matvec(const uint16_t* __restrict__ x, int K, int per_entry,
                                                     const uint8_t* __restrict__ weight, int E, int N,
                                                     const IDX* __restrict__ ids, int k, int swiglu,
                                                     uint16_t* __restrict__ out, int32_t* __restrict__ d_error) {
  const int n = blockIdx.x, entry = blockIdx.y;
  const int NO = swiglu ? N / 2 : N;
  int64_t e = ids ? (int64_t)ids[entry] : 0;
  uint16_t* o = out + (size_t)entry * NO + n;
  if (e < 0 || e >= E) {
    if (threadIdx.x == 0) {
      *o = 0;
      if (e != -1 && d_error && n == 0) atomicOr(d_error, EP_DEVERR_EXPERT_ID);
    }
    return;
  }
  const size_t rb = (size_t)(9 * K / 16 + 4);
  const uint16_t* xr = x + (size_t)(per_entry ? entry : entry / k) * K;
  const uint8_t* w = weight + (size_t)e * N * rb;
  float y = dot_row(xr, w + n * rb, K);
  if (swiglu) {
    const float b = dot_row(xr, w + (size_t)(n + NO) * rb, K);
    y = y * __builtin_amdgcn_rcpf(1.0f + __expf(-y)) * b;
  }
  if (threadIdx.x == 0) *o = __builtin_bit_cast(uint16_t, (__bf16)y);
}

}  // namespace mtb

using namespace mtb;

MTB_EXPORT int32_t ep_nvfp4_expert_matvec(const uint16_t* x, int64_t tokens, int64_t hidden, int32_t x_per_entry,
                                          const uint8_t* weight, int64_t num_experts, int64_t width,
                                          const void* topk_idx, int32_t idx_dtype, int64_t top_k, int32_t swiglu,
                                          uint16_t* out, int32_t* d_error, void* stream) {
  if (tokens < 0 || hidden <= 0 || hidden % 64 != 0 || num_experts < 1 || num_experts > 1024 || width < 1 ||
      top_k < 1 || (swiglu && width % 2 != 0))
    return EP_ERR_SHAPE;
  if (!topk_idx && (num_experts != 1 || top_k != 1)) return EP_ERR_SHAPE;
  if (idx_dtype != EP_IDX_INT32 && idx_dtype != EP_IDX_INT64) return EP_ERR_DTYPE;
  if (tokens >= kSizeLimit || top_k > 1024 || hidden > (1 << 20) || width > (1 << 24) || tokens * top_k > 4096)
    return EP_ERR_RANGE;
  if (tokens == 0) return EP_OK;
  if (!x || !weight || !out) return EP_ERR_NULL;
  const dim3 grid((unsigned)(swiglu ? width / 2 : width), (unsigned)(tokens * top_k));
  if (idx_dtype == EP_IDX_INT64)
    hipLaunchKernelGGL(k_nvfp4_matvec<int64_t>, grid, dim3(64), 0, (hipStream_t)stream, x, (int)hidden, x_per_entry,
                       weight, (int)num_experts, (int)width, (const int64_t*)topk_idx, (int)top_k, swiglu, out,
                       d_error);
  else
    hipLaunchKernelGGL(k_nvfp4_matvec<int32_t>, grid, dim3(64), 0, (hipStream_t)stream, x, (int)hidden, x_per_entry,
                       weight, (int)num_experts, (int)width, (const int32_t*)topk_idx, (int)top_k, swiglu, out,
                       d_error);
  return launch_status();
}
