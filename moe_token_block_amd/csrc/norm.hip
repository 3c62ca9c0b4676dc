// The root-mean-square norm in front of an expert layer: the residual's addition,
// the norm and its MXFP8 quantization in one pass, and the gradient.
//   h = bf16(x + residual), r = 1 / sqrt(mean(h^2) + eps), y = h r w
//   dx = r (g - h r^2 mean(g h)) + dh, g = w dy;  dw = sum over rows of dy h r
// All in FP32; what is stored is rounded once.
#include "common.h"
#include "launch.h"
#include "mxfp8.h"
#include "stream.h"

namespace mtb {

typedef float f32x4 __attribute__((ext_vector_type(4)));

// A row is a workgroup's: thread i has its chunks of 8 values i, i + THREADS, ...
// (NB of them), kept in registers between the sum and its use.
template <int THREADS, typename T>
__device__ __forceinline__ T block_sum(T v, T* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if (THREADS == 64) return v;
  const int wave = threadIdx.x >> 6;
  __syncthreads();  // the last sum has been read
  if ((threadIdx.x & 63) == 0) red[wave] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < THREADS / 64; ++i) v += red[i];
  return v;
}

__device__ __forceinline__ void unpack8(u32x4 v, float* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[2 * i] = bf16lo(v[i]);
    o[2 * i + 1] = bf16hi(v[i]);
  }
}

// Eight values of a block of 32 (its largest magnitude's bits m) as E4M3 bytes.
__device__ __forceinline__ u32x2 e4m3x8(const float* y, uint32_t m, uint8_t& scale) {
  const int e = mx_exponent(__uint_as_float(m));
  scale = (uint8_t)(m < 0x7F800000u ? e + 127 : 255);
  // below 2^-126 the power is no normal number: the values are lifted by 2^64 first
  const bool tiny = e < -126;
  const float lift = tiny ? 0x1p64f : 1.0f, s = pow2f(tiny ? e + 64 : e);
  u32x2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    i16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, y[4 * i] * lift, y[4 * i + 1] * lift, s, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, y[4 * i + 2] * lift, y[4 * i + 3] * lift, s, true);
    o[i] = __builtin_bit_cast(uint32_t, r);
  }
  return o;
}

// A workgroup a row: one pass over memory, 820 MB in 136 us at 16384 x 7168 (6.0 TB/s);
// one row of 4096 2.8 us, two memory latencies and the sum's exchange.
// h_out may be x or res: a chunk is read before its sum is written, by one thread.
template <int THREADS, int NB, bool RES>
__global__ __launch_bounds__(THREADS) void k_rmsnorm_mxfp8(const uint16_t* x, const uint16_t* res,
                                                           const uint16_t* __restrict__ weight, int H, float eps,
                                                           uint16_t* h_out, uint8_t* __restrict__ data,
                                                           uint8_t* __restrict__ scales, float* __restrict__ rstd) {
  __shared__ double red[THREADS / 64];
  const int tid = threadIdx.x, nch = H >> 3;
  const int64_t row = blockIdx.x, c0 = row * nch;
  u32x4 v[NB], q[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int c = tid + b * THREADS;
    v[b] = q[b] = u32x4{0u, 0u, 0u, 0u};
    if (c < nch) {
      v[b] = ld_once<u32x4>(x + 8 * (c0 + c));
      if (RES) q[b] = ld_once<u32x4>(res + 8 * (c0 + c));
    }
  }
  double ss = 0.0;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int c = tid + b * THREADS;
    if (RES) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[b][i] = bf16pair(bf16lo(v[b][i]) + bf16lo(q[b][i]), bf16hi(v[b][i]) + bf16hi(q[b][i]));
      if (c < nch) st_once(h_out + 8 * (c0 + c), v[b]);
    }
    float f[8], part = 0.0f;
    unpack8(v[b], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) part = __builtin_fmaf(f[i], f[i], part);
    ss += part;
  }
  // eight squares at a time in FP32, their sums in FP64: rstd is the nearest FP32 number
  // but for a few in a thousand rows, and with it nearly every byte what exact
  // arithmetic gives
  ss = block_sum<THREADS>(ss, red);
  const float r = (float)(1.0 / sqrt(ss / H + (double)eps));
  if (tid == 0) rstd[row] = r;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int c = tid + b * THREADS;
    if (c >= nch) continue;  // whole quads: nch is a multiple of 4
    float f[8], w[8];
    unpack8(v[b], f);
    unpack8(ld_any<u32x4>(weight + 8 * c), w);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = f[i] * r * w[i];
      m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    }
    uint8_t s;
    const u32x2 d = e4m3x8(f, quad_max(m), s);
    st_once(data + 8 * (c0 + c), d);
    if ((c & 3) == 0) scales[(c0 + c) >> 2] = s;
  }
}

// The gradient of rows blockIdx.x, + gridDim.x, ...: dx of each, and the
// workgroup's share of dw, one row of `part`.  A row's loads are in flight while the
// row before is taken, and the columns' sums stay in registers: 486 MB in 79 us at 14841
// x 4096 (6.1 TB/s), the join of the 512 parts 5 us more.
template <int THREADS, int NB, bool DH>
__global__ __launch_bounds__(THREADS) void k_drmsnorm(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ h,
                                                      const uint16_t* __restrict__ weight,
                                                      const float* __restrict__ rstd, const uint16_t* __restrict__ dh,
                                                      int rows, int H, uint16_t* __restrict__ dx,
                                                      float* __restrict__ part) {
  __shared__ float red[THREADS / 64];
  const int tid = threadIdx.x, nch = H >> 3;
  const float inv = 1.0f / (float)H;
  float dw[NB][8];
  u32x4 w[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int c = tid + b * THREADS;
    w[b] = c < nch ? ld_any<u32x4>(weight + 8 * c) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[b][i] = 0.0f;
  }
  struct Row {
    u32x4 g[NB], h[NB], d[NB];
    float r;
  };
  auto load = [&](int row, Row& q) {
    const int64_t c0 = (int64_t)row * nch;
    q.r = rstd[row];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int c = tid + b * THREADS;
      q.g[b] = q.h[b] = q.d[b] = u32x4{0u, 0u, 0u, 0u};
      if (c < nch) {
        q.g[b] = ld_once<u32x4>(dy + 8 * (c0 + c));
        q.h[b] = ld_once<u32x4>(h + 8 * (c0 + c));
        if (DH) q.d[b] = ld_once<u32x4>(dh + 8 * (c0 + c));
      }
    }
  };
  auto step = [&](int row, const Row& q) {
    float dot = 0.0f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float g[8], f[8], ww[8];
      unpack8(q.g[b], g);
      unpack8(q.h[b], f);
      unpack8(w[b], ww);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot = __builtin_fmaf(g[i] * ww[i], f[i], dot);
        dw[b][i] = __builtin_fmaf(g[i], f[i] * q.r, dw[b][i]);
      }
    }
    const float k = block_sum<THREADS>(dot, red) * inv * q.r * q.r;
    const int64_t c0 = (int64_t)row * nch;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int c = tid + b * THREADS;
      if (c >= nch) continue;
      float g[8], f[8], ww[8], d[8];
      unpack8(q.g[b], g);
      unpack8(q.h[b], f);
      unpack8(w[b], ww);
      unpack8(q.d[b], d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = q.r * (g[i] * ww[i] - f[i] * k);
        d[i] = DH ? v + d[i] : v;
      }
      st_once(dx + 8 * (c0 + c), pack8(d));
    }
  };
  Row cur;
  load(blockIdx.x, cur);
  for (int row = blockIdx.x; row < rows; row += gridDim.x) {
    Row next;
    const bool more = rows - row > (int)gridDim.x;
    if (more) load(row + gridDim.x, next);
    step(row, cur);
    if (more) cur = next;
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int c = tid + b * THREADS;
    if (c >= nch) continue;
    float* o = part + ((int64_t)blockIdx.x * nch + c) * 8;
    st_any<f32x4>(o, f32x4{dw[b][0], dw[b][1], dw[b][2], dw[b][3]});
    st_any<f32x4>(o + 4, f32x4{dw[b][4], dw[b][5], dw[b][6], dw[b][7]});
  }
}

// dw = the sum of the parts, 32 threads a column, each its run of them in order, eight
// loads at a time.
__global__ __launch_bounds__(1024) void k_drmsnorm_weight(const float* __restrict__ part, int parts, int H,
                                                          float* __restrict__ dw) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), q = threadIdx.x >> 5;  // H is a multiple of 32
  const int each = (parts + 31) >> 5, lo = q * each, hi = min(parts, lo + each);
  float v = 0.0f;
  int p = lo;
  for (; p + 8 <= hi; p += 8) {
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = part[(int64_t)(p + i) * H + c];
#pragma unroll
    for (int i = 0; i < 8; ++i) v += a[i];
  }
  for (; p < hi; ++p) v += part[(int64_t)p * H + c];
  s[q][threadIdx.x & 31] = v;
  __syncthreads();
  if (q) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) v += s[i][threadIdx.x];
  dw[c] = v;
}

}  // namespace mtb

using namespace mtb;

namespace {

int32_t check_sizes(int64_t rows, int64_t hidden) {
  if (rows < 0 || hidden < 32 || hidden % 32 != 0 || hidden > 16384) return EP_ERR_SHAPE;
  if (rows >= ((int64_t)1 << 23)) return EP_ERR_RANGE;  // a row has up to 512 of the grid's 2^32 threads
  return EP_OK;
}

// f(threads, chunks a thread): one wave where a row has few chunks.
template <typename F>
void by_width(int64_t hidden, F&& f) {
  if (hidden <= 512) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (hidden <= 1024) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  else if (hidden <= 2048) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  else if (hidden <= 4096) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  else if (hidden <= 8192) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 512>{}, std::integral_constant<int, 4>{});
}

// Up to so many rows one workgroup takes them all and its sums are dw: one launch.
constexpr int64_t kOneBlockRows = 4;

// Workgroups of the gradient, and rows of its workspace.
int64_t grad_parts(int64_t rows, int64_t hidden) {
  if (rows <= kOneBlockRows) return rows > 0;
  const int64_t most = hidden <= 1024 ? 2048 : 512;
  return rows < most ? rows : most;
}

}  // namespace

MTB_EXPORT int32_t rmsnorm_mxfp8(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, int64_t rows,
                                 int64_t hidden, float eps, uint16_t* h, uint8_t* data, uint8_t* scales, float* rstd,
                                 void* stream) {
  const int32_t st = check_sizes(rows, hidden);
  if (st != EP_OK) return st;
  // from here on squares that FP32 loses below its range are nothing beside eps
  if (!(eps >= 0x1p-100f && eps <= 1e30f)) return EP_ERR_SHAPE;
  if (rows == 0) return EP_OK;
  if (!x || !weight || !data || !scales || !rstd || (residual && !h)) return EP_ERR_NULL;
  by_width(hidden, [&](auto threads, auto nb) {
    constexpr int TH = decltype(threads)::value, NB = decltype(nb)::value;
    if (residual)
      hipLaunchKernelGGL((k_rmsnorm_mxfp8<TH, NB, true>), dim3((unsigned)rows), dim3(TH), 0, (hipStream_t)stream, x, residual,
                         weight, (int)hidden, eps, h, data, scales, rstd);
    else
      hipLaunchKernelGGL((k_rmsnorm_mxfp8<TH, NB, false>), dim3((unsigned)rows), dim3(TH), 0, (hipStream_t)stream, x,
                         residual, weight, (int)hidden, eps, h, data, scales, rstd);
  });
  return launch_status();
}

MTB_EXPORT size_t drmsnorm_workspace_bytes(int64_t rows, int64_t hidden) {
  if (check_sizes(rows, hidden) != EP_OK || rows <= kOneBlockRows) return 0;
  return (size_t)(grad_parts(rows, hidden) * hidden) * 4;
}

MTB_EXPORT int32_t drmsnorm(const uint16_t* dy, const uint16_t* h, const uint16_t* weight, const float* rstd,
                            const uint16_t* dh, int64_t rows, int64_t hidden, uint16_t* dx, float* dweight,
                            void* workspace, size_t workspace_bytes, void* stream) {
  const int32_t st = check_sizes(rows, hidden);
  if (st != EP_OK) return st;
  if (!dweight || (rows > 0 && (!dy || !h || !weight || !rstd || !dx))) return EP_ERR_NULL;
  const size_t need = drmsnorm_workspace_bytes(rows, hidden);
  if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15))) return EP_ERR_WORKSPACE;
  float* part = need ? (float*)workspace : dweight;
  const int parts = (int)grad_parts(rows, hidden);
  if (rows > 0)
    by_width(hidden, [&](auto threads, auto nb) {
      constexpr int TH = decltype(threads)::value, NB = decltype(nb)::value;
      if (dh)
        hipLaunchKernelGGL((k_drmsnorm<TH, NB, true>), dim3((unsigned)parts), dim3(TH), 0, (hipStream_t)stream, dy, h, weight,
                           rstd, dh, (int)rows, (int)hidden, dx, part);
      else
        hipLaunchKernelGGL((k_drmsnorm<TH, NB, false>), dim3((unsigned)parts), dim3(TH), 0, (hipStream_t)stream, dy, h, weight,
                           rstd, dh, (int)rows, (int)hidden, dx, part);
    });
  if (parts == 1) return launch_status();
  hipLaunchKernelGGL(k_drmsnorm_weight, dim3((unsigned)(hidden / 32)), dim3(1024), 0, (hipStream_t)stream,
                     (const float*)workspace, parts, (int)hidden, dweight);
  return launch_status();
}
