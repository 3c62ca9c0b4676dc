// Products of grouped MXFP4 or MXFP8 rows with MXFP4 weights:
//   out[g, n] = sum over blocks b of 32 of 2^(sa[g, b] - 127) 2^(sw[n, b] - 127)
//               sum_i a[g, 32 b + i] w[n, 32 b + i]
// on v_mfma_scale_f32_16x16x128_f8f6f4, which takes the codes and the blocks'
// scale bytes as they are stored: nothing is decoded.  Sums are FP32.  For MXFP4
// rows every product is exact and so is the sum of a block.  For MXFP8 rows the
// instruction adds eight neighbouring products at a time, each cut at 2^-13 of the
// largest of the eight (measured: 16 + 2^-9 is kept, 32 + 2^-9 is not; across the
// eights the sum has FP32's width), at most 2^-10 of the sum of the terms'
// magnitudes and a quarter of the result's own BF16 rounding where terms do not
// cancel.  Decoding to BF16 instead would be exact, at a quarter of the rate.
#include "common.h"
#include "grouped.h"
#include "launch.h"

namespace mtb {

constexpr int kE2M1 = 4, kE4M3 = 0;  // the instruction's operand formats

// Where chunk c (16 bytes) of a tile row lies in LDS, so that eight lanes reading
// one chunk of eight neighbouring rows meet every bank once.
template <int RB>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  if (RB == 128) return row * 128 + 16 * (c ^ (row & 7));
  return (row >> 1) * 128 + 16 * ((4 * (row & 1) + c) ^ ((row >> 1) & 3));
}

// Codes and scale bytes of C rows, one step of them: RB bytes of codes a row and
// SB scale bytes.
template <int C, int THREADS, int RB, int SB>
struct MxTile {
  static constexpr int kRowPieces = RB / 16, kPieces = C * kRowPieces / THREADS;
  static constexpr int kWords = C * SB / 4, kSc = (kWords + THREADS - 1) / THREADS;
  static constexpr int kBytes = C * (RB + SB);
  uint32_t off[kPieces], soff[kSc];
  u32x4 v[kPieces];
  uint32_t sv[kSc];

  __device__ __forceinline__ void init(int64_t row_bytes, int64_t row_blocks, int c_n) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = threadIdx.x + i * THREADS;
      off[i] = (uint32_t)(min(p / kRowPieces, c_n - 1) * (uint32_t)row_bytes + 16 * (p % kRowPieces));
    }
#pragma unroll
    for (int i = 0; i < kSc; ++i) {
      const int p = min((int)threadIdx.x + i * THREADS, kWords - 1);
      soff[i] = (uint32_t)(min(p / (SB / 4), c_n - 1) * (uint32_t)row_blocks + 4 * (p % (SB / 4)));
    }
  }
  // bytes and blocks: what is left of a row from the step's first value on.
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int bytes, int blocks) {
    const bool whole = blocks >= SB;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = threadIdx.x + i * THREADS;
      if (whole) v[i] = ld_any<u32x4>(codes + off[i]);
      else v[i] = 16 * (p % kRowPieces) < bytes ? ld_any<u32x4>(codes + off[i]) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < kSc; ++i) {
      const int p = min((int)threadIdx.x + i * THREADS, kWords - 1), n = blocks - 4 * (p % (SB / 4));
      if (whole) {
        sv[i] = ld_any<uint32_t>(scales + soff[i]);
      } else {
        uint32_t w = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (b < n) w |= (uint32_t)scales[soff[i] + b] << (8 * b);
        sv[i] = w;
      }
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = threadIdx.x + i * THREADS;
      *reinterpret_cast<u32x4*>(lds + chunk_at<RB>(p / kRowPieces, p % kRowPieces)) = v[i];
    }
#pragma unroll
    for (int i = 0; i < kSc; ++i) {
      const int p = threadIdx.x + i * THREADS;
      if (kWords % THREADS == 0 || p < kWords) *reinterpret_cast<uint32_t*>(lds + C * RB + 4 * p) = sv[i];
    }
  }
};

// One output tile of BM x BN per workgroup, 256 values (MXFP8 rows: 128) a step
// through two LDS buffers.
template <int BM, int BN, int WM, int WN, bool A8>
struct MxProduct {
  static constexpr int kThreads = 64 * WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int kStep = A8 ? 128 : 256, SB = kStep / 32, kRowW = kStep / 2;
  typedef MxTile<BM, kThreads, 128, SB> TileA;
  typedef MxTile<BN, kThreads, kRowW, SB> TileW;
  static constexpr int kBuf = TileA::kBytes + TileW::kBytes;
  static constexpr int kOut = WM * WN * MT * 2048, kLds = 2 * kBuf > kOut ? 2 * kBuf : kOut;
  f32x4 acc[MT][NT];

  static __device__ __forceinline__ i32x8 wide(u32x4 lo, u32x4 hi) {
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  }

  __device__ __forceinline__ void compute(const char* a_lds, const char* w_lds, int wm, int wn) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const u32x4 none = {0u, 0u, 0u, 0u};
    int sa[MT], sw[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const char* at = w_lds + BN * kRowW + (16 * (wn * NT + i) + r) * SB;
      sw[i] = A8 ? (int)*reinterpret_cast<const uint8_t*>(at + g) : (int)*reinterpret_cast<const uint16_t*>(at + 2 * g);
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const char* at = a_lds + BM * 128 + (16 * (wm * MT + j) + r) * SB;
      sa[j] = A8 ? (int)*reinterpret_cast<const uint8_t*>(at + g) : (int)*reinterpret_cast<const uint16_t*>(at + 2 * g);
    }
    if (A8) {
      // lane group g: weights 32 g .. + 31, row values 16 g .. + 15 and 64 + 16 g .. + 15,
      // the scale of values 32 g .. + 31, as the instruction has them
      u32x4 w[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i)
        w[i] = *reinterpret_cast<const u32x4*>(w_lds + chunk_at<kRowW>(16 * (wn * NT + i) + r, g));
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int row = 16 * (wm * MT + j) + r;
        const i32x8 a = wide(*reinterpret_cast<const u32x4*>(a_lds + chunk_at<128>(row, g)),
                             *reinterpret_cast<const u32x4*>(a_lds + chunk_at<128>(row, 4 + g)));
#pragma unroll
        for (int i = 0; i < NT; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(w[i], none), a, acc[j][i], kE2M1, kE4M3, 0,
                                                                       sw[i], 0, sa[j]);
      }
    } else {
      // which blocks of 32 a lane group takes is free: 2 g in the first half, 2 g + 1
      // in the second, so that one 16-bit read has both scales
#define MTB_HALF(S)                                                                                                  \
  do {                                                                                                               \
    u32x4 w[NT];                                                                                                     \
    _Pragma("unroll") for (int i = 0; i < NT; ++i) w[i] =                                                            \
        *reinterpret_cast<const u32x4*>(w_lds + chunk_at<kRowW>(16 * (wn * NT + i) + r, 2 * g + S));                 \
    _Pragma("unroll") for (int j = 0; j < MT; ++j) {                                                                 \
      const u32x4 a = *reinterpret_cast<const u32x4*>(a_lds + chunk_at<128>(16 * (wm * MT + j) + r, 2 * g + S));     \
      _Pragma("unroll") for (int i = 0; i < NT; ++i) acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(   \
          wide(w[i], none), wide(a, none), acc[j][i], kE2M1, kE2M1, S, sw[i], S, sa[j]);                             \
    }                                                                                                                \
  } while (0)
      MTB_HALF(0);
      MTB_HALF(1);
#undef MTB_HALF
    }
  }

  __device__ __forceinline__ void run(char* lds, const uint8_t* a, const uint8_t* as, int a_n, const uint8_t* w,
                                      const uint8_t* ws, int w_n, int K) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (K <= 0) return;
    TileA ta;
    TileW tw;
    ta.init(A8 ? K : K / 2, K / 32, a_n);
    tw.init(K / 2, K / 32, w_n);
    int left = K;
    auto load = [&]() {
      ta.load(a, as, A8 ? left : left / 2, left / 32);
      tw.load(w, ws, left / 2, left / 32);
      a += 128;
      as += SB;
      w += kRowW;
      ws += SB;
      left -= kStep;
    };
    load();
    ta.store(lds);
    tw.store(lds + TileA::kBytes);
    if (left > 0) load();
    const int steps = (K + kStep - 1) / kStep;
    __syncthreads();
    for (int t = 0; t < steps; ++t) {
      char* next = lds + ((t & 1) ? 0 : kBuf);
      if (t + 1 < steps) {
        ta.store(next);
        tw.store(next + TileA::kBytes);
        if (left > 0) load();
      }
      const char* buf = lds + ((t & 1) ? kBuf : 0);
      compute(buf, buf + TileA::kBytes, wm, wn);
      __syncthreads();
    }
  }
};

template <int BM, int BN, int WM, int WN, bool A8>
__global__ __launch_bounds__(64 * WM * WN) void k_mxfp4_grouped_gemm(const uint8_t* __restrict__ data,
                                                                     const uint8_t* __restrict__ scales, int K,
                                                                     const uint8_t* __restrict__ wcodes,
                                                                     const uint8_t* __restrict__ wscales, int64_t N,
                                                                     Groups gr, uint16_t* __restrict__ out) {
  typedef MxProduct<BM, BN, WM, WN, A8> P;
  extern __shared__ char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  Span s;
  int tn;
  if (!find_span<BM>(gr, (int)((N + BN - 1) / BN), s, tn, 8)) return;
  P prod;
  const int n0 = tn * BN;
  const int64_t row = s.row0, col = (int64_t)s.expert * N + n0;
  if (s.used > 0)
    prod.run(lds, data + row * (A8 ? K : K / 2), scales + row * (K / 32), s.used, wcodes + col * (K / 2),
             wscales + col * (K / 32), (int)min((int64_t)BN, N - n0), K);
  else
    prod.run(lds, data, scales, 1, wcodes, wscales, 1, 0);
  static_assert(P::NT == 4, "a wave stores 64 columns");
  const int m = wm * P::MT * 16, n = n0 + wn * 64;
  store_block64<P::MT>(prod.acc, lds + wave * P::MT * 2048, out + (row + m) * N + n, N, s.used - m, s.extent - m,
                       (int)min((int64_t)64, N - n));
}

}  // namespace mtb

using namespace mtb;

namespace {
template <bool A8>
int32_t mx_product(const uint8_t* data, const uint8_t* scales, int64_t r_cap, int64_t K, const uint8_t* wcodes,
                   const uint8_t* wscales, int64_t E, int64_t N, const int32_t* counts, const int32_t* offsets,
                   uint16_t* out, hipStream_t s) {
  constexpr int BM = 128, BN = 128, WM = 2, WN = 2;
  const Groups gr{counts, offsets, (int)E, (int)r_cap};
  const int64_t blocks = span_blocks(r_cap, E, !counts, BM, (N + BN - 1) / BN);
  if (blocks >= kSizeLimit) return EP_ERR_RANGE;
  const size_t lds = MxProduct<BM, BN, WM, WN, A8>::kLds;
  hipLaunchKernelGGL((k_mxfp4_grouped_gemm<BM, BN, WM, WN, A8>), dim3((unsigned)blocks), dim3(64 * WM * WN), lds, s, data,
                     scales, (int)K, wcodes, wscales, N, gr, out);
  return launch_status();
}
}  // namespace

MTB_EXPORT int32_t ep_mxfp4_grouped_gemm(const uint8_t* data, const uint8_t* scales, int32_t row_format, int64_t r_cap,
                                         int64_t hidden, const uint8_t* weight_codes, const uint8_t* weight_scales,
                                         int64_t num_experts, int64_t width, const int32_t* counts,
                                         const int32_t* offsets, int64_t entries, uint16_t* out, void* stream) {
  if (r_cap < 0 || hidden < 32 || hidden % 32 != 0 || width < 1 || num_experts < 1 || num_experts > 1024)
    return EP_ERR_SHAPE;
  if (entries < 0 || !counts != !offsets || (!counts && num_experts != 1)) return EP_ERR_SHAPE;
  if (row_format != EP_ROWS_MXFP4 && row_format != EP_ROWS_MXFP8) return EP_ERR_DTYPE;
  if (r_cap >= ((int64_t)1 << 25) || hidden > (1 << 20) || width > (1 << 20)) return EP_ERR_RANGE;
  if (r_cap == 0) return EP_OK;
  if (!data || !scales || !weight_codes || !weight_scales || !out) return EP_ERR_NULL;
  if (row_format == EP_ROWS_MXFP8)
    return mx_product<true>(data, scales, r_cap, hidden, weight_codes, weight_scales, num_experts, width, counts, offsets,
                            out, (hipStream_t)stream);
  return mx_product<false>(data, scales, r_cap, hidden, weight_codes, weight_scales, num_experts, width, counts, offsets,
                           out, (hipStream_t)stream);
}
