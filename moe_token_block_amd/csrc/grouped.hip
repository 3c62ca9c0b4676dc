// Products of the grouped BF16 rows with their experts' weights, and both
// gradients:
//   out[g, n]  = sum_k rows[g, k] W[e, n, k]
//   drows[g, k] = sum_n dout[g, n] W[e, n, k]
//   dW[e, n, k] = sum_g dout[g, n] rows[g, k]      over the rows g of expert e
// One kernel: an output tile of BM x BN per workgroup, the sum in steps of 64
// through two LDS buffers, v_mfma_f32_16x16x32_bf16 (products exact, sums FP32).
// The three differ in how an operand lies in memory: along the sum ("R": a tile
// row is 64 values of one output row or column), or across it ("T": a tile row is
// one term of the sum for all of the tile's output rows or columns), which LDS's
// transposing read turns into the instruction's operand.
#include "common.h"
#include "grouped.h"
#include "launch.h"

namespace mtb {

constexpr int kBK = 64;  // terms of the sum in one step

// An operand's tile: C output rows (or columns) by 64 terms, C * 128 bytes of LDS,
// staged through registers by THREADS threads.
template <int C, int THREADS, bool T>
struct Tile {
  static constexpr int kPieces = C * 8 / THREADS;  // 16-byte pieces a thread
  uint32_t off[kPieces];                           // bytes from the step's base
  u32x4 v[kPieces];

  // ld: values from one row of the matrix to the next; c_n: rows (R) or columns (T)
  // that exist from the tile's first on, at least 1.
  __device__ __forceinline__ void init(int64_t ld, int c_n) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = threadIdx.x + i * THREADS;
      if (T) off[i] = (uint32_t)((p / (C / 8)) * (uint32_t)ld + 8 * (p % (C / 8))) * 2u;
      else off[i] = (uint32_t)(min(p >> 3, c_n - 1) * (uint32_t)ld + 8 * (p & 7)) * 2u;
    }
  }
  // base: the step's first value; terms: how many of the step's 64 exist.  Rows (R)
  // that do not exist repeat the last; columns (T) that do not, and terms, are zeros.
  template <bool EDGE>
  __device__ __forceinline__ void load(const uint16_t* base, int terms, int c_n) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(base) + off[i]);
      const int p = threadIdx.x + i * THREADS;
      if (!EDGE) v[i] = ld_any<u32x4>(src);
      else if (T) v[i] = load8(src, p / (C / 8) < terms ? c_n - 8 * (p % (C / 8)) : 0);
      else v[i] = load8(src, terms - 8 * (p & 7));
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = threadIdx.x + i * THREADS;
      uint32_t at;
      if (T) {
        const int k = p / (C / 8), c = p % (C / 8);
        at = k * (2 * C) + 16 * (c ^ (2 * (k & 3)));
      } else {
        const int row = p >> 3, c = p & 7;
        at = row * 128 + 16 * (c ^ (row & 7));
      }
      *reinterpret_cast<u32x4*>(lds + at) = v[i];
    }
  }
  // The instruction's operand of the 16 output rows (columns) from c0 on and the 32
  // terms from 32 ks on: lane (r, g) holds terms 8 g .. 8 g + 7 of c0 + r.
  static __device__ __forceinline__ bf16x8 frag(const char* lds, int c0, int ks) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    if (T) {
      typedef short i16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
      const int k = 32 * ks + 8 * g + (r >> 2);  // this lane's row of the four that are transposed
      const uint32_t at = k * (2 * C) + ((2 * c0 + 8 * (r & 3)) ^ (32 * (k & 3)));
      i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(lds + at));
      i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(lds + at + 8 * C));
      typedef short i16x8 __attribute__((ext_vector_type(8)));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    const int row = c0 + r;
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(lds + row * 128 + 16 * ((4 * ks + g) ^ (row & 7))));
  }
};

// acc += P Q^T over `terms` terms: P (BM output rows) and Q (BN output columns) with
// first values p and q, and rows p_ld and q_ld values apart.
template <int BM, int BN, int WM, int WN, bool PT, bool QT>
struct Product {
  static constexpr int kThreads = 64 * WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int kBuf = (BM + BN) * 128, kLds = 2 * kBuf;
  f32x4 acc[MT][NT];

  __device__ __forceinline__ void run(char* lds, const uint16_t* p, int64_t p_ld, int p_n, const uint16_t* q,
                                      int64_t q_ld, int q_n, int terms) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (terms <= 0) return;
    Tile<BM, kThreads, PT> tp;
    Tile<BN, kThreads, QT> tq;
    tp.init(p_ld, p_n);
    tq.init(q_ld, q_n);
    const int64_t p_step = PT ? kBK * p_ld : kBK, q_step = QT ? kBK * q_ld : kBK;
    const bool p_cut = PT && p_n < BM, q_cut = QT && q_n < BN;
    int left = terms;  // terms that are not loaded yet
    auto load = [&]() {
      if (left >= kBK && !p_cut) tp.template load<false>(p, left, p_n);
      else tp.template load<true>(p, left, p_n);
      if (left >= kBK && !q_cut) tq.template load<false>(q, left, q_n);
      else tq.template load<true>(q, left, q_n);
      p += p_step;
      q += q_step;
      left -= kBK;
    };
    auto compute = [&](const char* buf) {
      const char* qb = buf + BM * 128;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        bf16x8 a[MT], b[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) b[i] = Tile<BN, kThreads, QT>::frag(qb, 16 * (wn * NT + i), ks);
#pragma unroll
        for (int j = 0; j < MT; ++j) a[j] = Tile<BM, kThreads, PT>::frag(buf, 16 * (wm * MT + j), ks);
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int i = 0; i < NT; ++i) acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[i], a[j], acc[j][i], 0, 0, 0);
      }
    };
    load();
    tp.store(lds);
    tq.store(lds + BM * 128);
    if (left > 0) load();
    const int steps = (terms + kBK - 1) / kBK;
    __syncthreads();
    for (int t = 0; t < steps; ++t) {
      char* next = lds + ((t & 1) ? 0 : kBuf);
      if (t + 1 < steps) {  // the next step's values, loaded a step ago, to the other buffer
        tp.store(next);
        tq.store(next + BM * 128);
        if (left > 0) load();
      }
      compute(lds + ((t & 1) ? kBuf : 0));
      __syncthreads();
    }
  }
};

// out[m, n] for grouped rows m: P the rows, Q the weights (QT: their transposes).
template <int BM, int BN, int WM, int WN, bool QT>
__global__ __launch_bounds__(64 * WM * WN) void k_bf16_grouped_gemm(const uint16_t* __restrict__ rows, int64_t K,
                                                                    const uint16_t* __restrict__ weight, int64_t N,
                                                                    Groups gr, uint16_t* __restrict__ out) {
  typedef Product<BM, BN, WM, WN, false, QT> P;
  extern __shared__ char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  Span s;
  int tn;
  if (!find_span<BM>(gr, (int)((N + BN - 1) / BN), s, tn, 8)) return;
  P prod;
  const int n0 = tn * BN;
  const int64_t ld = QT ? N : K;  // values of a weight row; K terms, N columns
  if (s.used > 0) {
    const uint16_t* w = weight + (int64_t)s.expert * N * K + (QT ? (int64_t)n0 : (int64_t)n0 * K);
    prod.run(lds, rows + (int64_t)s.row0 * K, K, s.used, w, ld, (int)min((int64_t)BN, N - n0), (int)K);
  } else {
    prod.run(lds, rows, K, 1, weight, ld, 1, 0);
  }
  static_assert(P::NT == 4, "a wave stores 64 columns");
  const int m = wm * P::MT * 16, n = n0 + wn * 64;
  store_block64<P::MT>(prod.acc, lds + wave * P::MT * 2048, out + (int64_t)(s.row0 + m) * N + n, N, s.used - m,
                       s.extent - m, (int)min((int64_t)64, N - n));
}

// dW of one expert: P dout's columns, Q the rows' columns, the sum over the expert's rows.
template <int BM, int BN, int WM, int WN, bool F32>
__global__ __launch_bounds__(64 * WM * WN) void k_bf16_grouped_wgrad(const uint16_t* __restrict__ dout, int64_t N,
                                                                     const uint16_t* __restrict__ rows, int64_t K,
                                                                     Groups gr, void* __restrict__ out) {
  typedef Product<BM, BN, WM, WN, true, true> P;
  extern __shared__ char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int e = blockIdx.z, m0 = blockIdx.y * BM, n0 = blockIdx.x * BN;
  int lo = 0, cnt = gr.r_cap;
  if (gr.counts) {
    lo = min(max(gr.offsets[e], 0), gr.r_cap);
    cnt = min(max(gr.counts[e], 0), gr.r_cap - lo);
  }
  P prod;
  prod.run(lds, dout + (int64_t)lo * N + m0, N, (int)min((int64_t)BM, N - m0), rows + (int64_t)lo * K + n0, K,
           (int)min((int64_t)BN, K - n0), cnt);
  const int m = m0 + wm * P::MT * 16, n = n0 + wn * 64;
  const int64_t at = ((int64_t)e * N + m) * K + n;
  if (!F32) {
    store_block64<P::MT>(prod.acc, lds + wave * P::MT * 2048, (uint16_t*)out + at, K, (int)(N - m), (int)(N - m),
                         (int)min((int64_t)64, K - n));
  } else {
    float* o = (float*)out + at;
#pragma unroll
    for (int j = 0; j < P::MT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * j + r, c = 16 * i + 4 * g;
        if (m + row >= N) continue;
        float* d = o + (int64_t)row * K + c;
        if (n + c + 4 <= K) st_any<f32x4>(d, prod.acc[j][i]);
        else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (n + c + q < K) d[q] = prod.acc[j][i][q];
        }
      }
  }
}

}  // namespace mtb

using namespace mtb;

namespace {

// Sizes of the three products: r_cap grouped rows, [width, depth] weights.
int32_t check_sizes(int64_t r_cap, int64_t depth, int64_t width, int64_t experts, const int32_t* counts,
                    const int32_t* offsets) {
  if (r_cap < 0 || depth < 1 || width < 1 || experts < 1 || experts > 1024) return EP_ERR_SHAPE;
  if (!counts != !offsets || (!counts && experts != 1)) return EP_ERR_SHAPE;
  // a tile's rows are addressed by 32 bits of bytes, the grid by 31 bits of tiles
  if (r_cap >= ((int64_t)1 << 25) || depth > (1 << 20) || width > (1 << 20)) return EP_ERR_RANGE;
  return EP_OK;
}

template <bool QT>
int32_t product(const uint16_t* rows, int64_t r_cap, int64_t K, const uint16_t* weight, int64_t E, int64_t N,
                const int32_t* counts, const int32_t* offsets, uint16_t* out, hipStream_t s) {
  if (r_cap == 0) return EP_OK;
  if (!rows || !weight || !out) return EP_ERR_NULL;
  const Groups gr{counts, offsets, (int)E, (int)r_cap};
  constexpr int BM = 128, BN = 128, WM = 2, WN = 2;
  const int64_t blocks = span_blocks(r_cap, E, !counts, BM, (N + BN - 1) / BN);
  if (blocks >= kSizeLimit) return EP_ERR_RANGE;
  const size_t lds = Product<BM, BN, WM, WN, false, QT>::kLds;
  hipLaunchKernelGGL((k_bf16_grouped_gemm<BM, BN, WM, WN, QT>), dim3((unsigned)blocks), dim3(64 * WM * WN), lds, s, rows, K,
                     weight, N, gr, out);
  return launch_status();
}

}  // namespace

MTB_EXPORT int32_t ep_bf16_grouped_gemm(const uint16_t* rows, int64_t r_cap, int64_t hidden, const uint16_t* weight,
                                        int64_t num_experts, int64_t width, const int32_t* counts,
                                        const int32_t* offsets, int64_t entries, uint16_t* out, void* stream) {
  const int32_t st = check_sizes(r_cap, hidden, width, num_experts, counts, offsets);
  if (st != EP_OK) return st;
  if (entries < 0) return EP_ERR_SHAPE;
  return product<false>(rows, r_cap, hidden, weight, num_experts, width, counts, offsets, out, (hipStream_t)stream);
}

MTB_EXPORT int32_t ep_bf16_grouped_dgrad(const uint16_t* dout, int64_t r_cap, int64_t width, const uint16_t* weight,
                                         int64_t num_experts, int64_t hidden, const int32_t* counts,
                                         const int32_t* offsets, int64_t entries, uint16_t* drows, void* stream) {
  const int32_t st = check_sizes(r_cap, hidden, width, num_experts, counts, offsets);
  if (st != EP_OK) return st;
  if (entries < 0) return EP_ERR_SHAPE;
  return product<true>(dout, r_cap, width, weight, num_experts, hidden, counts, offsets, drows, (hipStream_t)stream);
}

MTB_EXPORT size_t ep_bf16_grouped_wgrad_workspace_bytes(int64_t width, int64_t hidden, int64_t num_experts,
                                                        int64_t entries) {
  return 0;
}

MTB_EXPORT int32_t ep_bf16_grouped_wgrad(const uint16_t* dout, const uint16_t* rows, int64_t r_cap, int64_t width,
                                         int64_t hidden, int64_t num_experts, const int32_t* counts,
                                         const int32_t* offsets, int64_t entries, void* dweight, int32_t f32, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  const int32_t st = check_sizes(r_cap, hidden, width, num_experts, counts, offsets);
  if (st != EP_OK) return st;
  if (entries < 0) return EP_ERR_SHAPE;
  if (!dweight || (r_cap > 0 && (!dout || !rows))) return EP_ERR_NULL;
  constexpr int BM = 128, BN = 128, WM = 2, WN = 2;
  const Groups gr{counts, offsets, (int)num_experts, (int)r_cap};
  const dim3 grid((unsigned)((hidden + BN - 1) / BN), (unsigned)((width + BM - 1) / BM), (unsigned)num_experts);
  const size_t lds = Product<BM, BN, WM, WN, true, true>::kLds;
  if (f32)
    hipLaunchKernelGGL((k_bf16_grouped_wgrad<BM, BN, WM, WN, true>), grid, dim3(64 * WM * WN), lds, (hipStream_t)stream, dout,
                       width, rows, hidden, gr, dweight);
  else
    hipLaunchKernelGGL((k_bf16_grouped_wgrad<BM, BN, WM, WN, false>), grid, dim3(64 * WM * WN), lds, (hipStream_t)stream,
                       dout, width, rows, hidden, gr, dweight);
  return launch_status();
}
