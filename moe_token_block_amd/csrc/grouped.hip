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
// transposing read turns into the instruction's operand.  For few rows the weights'
// bytes are the time, and kernels of their own stream them.
//
// Measured (large library products of the same kinds reach 1620, 1410 and 1220
// TFLOP/s): 131072 rows of 32 experts, 7168 x 4096, 6.6 to 6.9 ms, 1120 to 1170
// TFLOP/s; the rows' gradient of 8192 uneven rows, 8 experts of 4096 x 4096, 312 us,
// 880; the weights' of 65536 rows, 16 experts of 4096 x 4096, 1.79 to 1.88 ms, 1170 to
// 1230.  The matrix units are busy in 0.57 to 0.64 of the CUs' busy cycles, at clocks
// below 1.8 GHz (the large product); the rest are the steps' barriers with the first LDS
// reads behind them, and the first loads and the stores of a tile, which nothing else on
// the CU overlaps (128 KB of LDS, 240 registers a lane).
// Measured without gain: a second barrier a step that lets the next step's operands be
// read ahead (8% slower), tiles of 256 x 128, raised wave priority, every load of a step
// before its products (20% slower), four waves of 128 x 128 (they spill).
#include <algorithm>

#include "common.h"
#include "grouped.h"
#include "launch.h"

namespace mtb {

constexpr int kBK = 64;  // terms of the sum in one step

// An operand's tile: C output rows (or columns) by 64 terms, C * 128 bytes of LDS,
// staged through registers by THREADS threads.
template <int C, int THREADS, bool T, int SETS>
struct Tile {
  static constexpr int kPieces = C * 8 / THREADS;  // 16-byte pieces a thread
  int tid, ld;                                     // of the THREADS that share the tile; values from row to row
  uint32_t off[kPieces];                           // bytes from the step's base
  u32x4 v[SETS][kPieces];                          // of the steps whose loads are under way

  // row: values from one row of the matrix to the next; c_n: rows (R) or columns (T)
  // that exist from the tile's first on, at least 1.
  __device__ __forceinline__ void init(int thread, int64_t row, int c_n) {
    tid = thread;
    ld = (int)row;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * THREADS;
      if (T) off[i] = (uint32_t)((p / (C / 8)) * (uint32_t)ld + 8 * min(p % (C / 8), (c_n - 1) >> 3)) * 2u;
      else off[i] = (uint32_t)(min(p >> 3, c_n - 1) * (uint32_t)ld + 8 * (p & 7)) * 2u;
    }
  }
  // base: the step's first value; terms: how many of the step's 64 exist.  Rows (R) that
  // do not exist repeat the last, and pieces of columns (T) the last piece: what comes of
  // them is not stored.  EDGE: terms that do not exist are zeros, and nothing past a
  // row's end is read (without it up to 7 values of the next row are).
  template <bool EDGE>
  __device__ __forceinline__ void load_piece(int set, int i, const uint16_t* base, int terms, int c_n) {
    const uint16_t* src = reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(base) + off[i]);
    const int p = tid + i * THREADS;
    if (!EDGE) {
      v[set][i] = ld_any<u32x4>(src);
    } else if (T) {
      const int k = p / (C / 8), past = max(k - (terms - 1), 0);
      v[set][i] = load_end(src - (int64_t)past * ld, c_n - 8 * min(p % (C / 8), (c_n - 1) >> 3), ld >= 8);
      if (past) v[set][i] = u32x4{0u, 0u, 0u, 0u};
    } else {
      v[set][i] = load_end(src, terms - 8 * (p & 7), ld >= 8);
    }
  }
  template <bool EDGE>
  __device__ __forceinline__ void load(int set, const uint16_t* base, int terms, int c_n) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) load_piece<EDGE>(set, i, base, terms, c_n);
  }
  // T: the 32 lanes of half a transposing read take 32 bytes of each of eight rows
  // (four terms of two lane groups): the rows' 32-byte pieces are permuted so that
  // they meet every bank once.
  static __device__ __forceinline__ int key(int k) { return (k & 3) + (C >= 128 ? 4 * ((k >> 3) & 1) : 0); }
  __device__ __forceinline__ void store_piece(int set, int i, char* lds) const {
    const int p = tid + i * THREADS;
    uint32_t at;
    if (T) {
      const int k = p / (C / 8), c = p % (C / 8);
      at = k * (2 * C) + 16 * (c ^ (2 * key(k)));
    } else {
      const int row = p >> 3, c = p & 7;
      at = row * 128 + 16 * (c ^ (row & 7));
    }
    *reinterpret_cast<u32x4*>(lds + at) = v[set][i];
  }
  __device__ __forceinline__ void store(int set, char* lds) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) store_piece(set, i, lds);
  }
  // The instruction's operand of the 16 output rows (columns) from c0 on and the 32
  // terms from 32 ks on: lane (r, g) holds terms 8 g .. 8 g + 7 of c0 + r.
  static __device__ __forceinline__ bf16x8 frag(const char* lds, int c0, int ks) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    if (T) {
      typedef short i16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
      const int k = 32 * ks + 8 * g + (r >> 2);  // this lane's row of the four that are transposed
      const uint32_t at = k * (2 * C) + ((2 * c0 + 8 * (r & 3)) ^ (32 * key(k)));
      i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(lds + at));
      i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(lds + at + 8 * C));
      typedef short i16x8 __attribute__((ext_vector_type(8)));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    const int row = c0 + r;
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(lds + row * 128 + 16 * ((4 * ks + g) ^ (row & 7))));
  }
};

// acc = P Q^T over `terms` terms: P (BM output rows) and Q (BN output columns) with
// first values p and q, and rows p_ld and q_ld values apart.  SETS steps' loads are
// under way beside the step that LDS holds next.  SHARES groups of WM x WN waves take
// the steps in turn, each through buffers of its own; the first ends with the sum.
template <int BM, int BN, int WM, int WN, bool PT, bool QT, int SETS, int SHARES>
struct Product {
  static constexpr int kThreads = 64 * WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
  typedef Tile<BM, kThreads, PT, SETS> TileP;
  typedef Tile<BN, kThreads, QT, SETS> TileQ;
  static_assert(TileP::kPieces + TileQ::kPieces == 8, "a piece for each of a step's eight parts");
  static constexpr int kBuf = (BM + BN) * 128, kLds = 2 * SHARES * kBuf;
  f32x4 acc[MT][NT];

  // A step's products in eight parts, `between(part)` called in each.  The next part's
  // operands are read before it: no LDS read moves ahead of the stores in `between`.
  template <typename F>
  __device__ __forceinline__ void compute(const char* buf, int wm, int wn, F&& between) {
    constexpr int J = MT / 4;
    bf16x8 b[2][NT], a[2][J];
    auto read = [&](auto part) {
      constexpr int c = decltype(part)::value, ks = c / 4, jg = c % 4;
      if constexpr (jg == 0) {
#pragma unroll
        for (int i = 0; i < NT; ++i) b[ks][i] = TileQ::frag(buf + BM * 128, 16 * (wn * NT + i), ks);
      }
#pragma unroll
      for (int j = 0; j < J; ++j) a[c & 1][j] = TileP::frag(buf, 16 * (wm * MT + jg * J + j), ks);
    };
    read(std::integral_constant<int, 0>{});
    static_for<0, 8>([&](auto part) {
      constexpr int c = decltype(part)::value, ks = c / 4, jg = c % 4;
      if constexpr (c < 7) read(std::integral_constant<int, c + 1>{});
      between(part);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < NT; ++i)
          acc[jg * J + j][i] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[ks][i], a[c & 1][j], acc[jg * J + j][i], 0, 0, 0);
    });
  }

  __device__ __forceinline__ void run(char* all_lds, const uint16_t* p, int64_t p_ld, int p_n, const uint16_t* q,
                                      int64_t q_ld, int q_n, int terms) {
    const int share = SHARES == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    const int tid = threadIdx.x - share * kThreads;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    char* lds = all_lds + share * 2 * kBuf;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (terms <= 0) return;
    TileP tp;
    TileQ tq;
    tp.init(tid, p_ld, p_n);
    tq.init(tid, q_ld, q_n);
    const int64_t p_step = PT ? kBK * p_ld : kBK, q_step = QT ? kBK * q_ld : kBK;
    const bool p_cut = PT && p_n < BM && p_n % 8, q_cut = QT && q_n < BN && q_n % 8;
    p += share * p_step;
    q += share * q_step;
    int left = terms - share * kBK;  // from this group's next step on: terms that are not loaded yet
    const int all = (terms + kBK - 1) / kBK, steps = (all + SHARES - 1) / SHARES;
    const int mine = (all - share + SHARES - 1) / SHARES;  // steps of this group; the first has `steps`
    auto advance = [&]() {
      p += SHARES * p_step;
      q += SHARES * q_step;
      left -= SHARES * kBK;
    };
    auto load = [&](int set) {
      if (left <= 0) return;
      if (left >= kBK && !p_cut) tp.template load<false>(set, p, left, p_n);
      else tp.template load<true>(set, p, left, p_n);
      if (left >= kBK && !q_cut) tq.template load<false>(set, q, left, q_n);
      else tq.template load<true>(set, q, left, q_n);
      advance();
    };
    load(0);
    if (mine > 0) {
      tp.store(0, lds);
      tq.store(0, lds + BM * 128);
    }
    static_for<0, SETS>([&](auto set) { load(set); });  // set i: the step 1 + i
    __syncthreads();
    // The steps whose loads (1 + SETS steps ahead) are whole: one run of instructions,
    // the next step's values on their way to LDS and a later one's to the registers
    // they leave, a piece at a time between the products.
    int t = 0;
    // the same for both groups; without the last where a row's end is read past
    const int whole = terms / kBK / SHARES - 1 - SETS - (p_cut || q_cut ? 1 : 0);
    for (; t + SETS <= whole; t += SETS) {
      static_for<0, SETS>([&](auto sub) {
        constexpr int set = decltype(sub)::value;
        const char* cur = lds + (((t + set) & 1) ? kBuf : 0);
        char* next = lds + (((t + set) & 1) ? 0 : kBuf);
        compute(cur, wm, wn, [&](auto part) {
          constexpr int c = decltype(part)::value;
          if constexpr (c < TileP::kPieces) {
            tp.store_piece(set, c, next);
            tp.template load_piece<false>(set, c, p, kBK, p_n);
          } else {
            tq.store_piece(set, c - TileP::kPieces, next + BM * 128);
            tq.template load_piece<false>(set, c - TileP::kPieces, q, kBK, q_n);
          }
        });
        advance();
        __syncthreads();
      });
    }
    for (; t < steps; t += SETS) {
      static_for<0, SETS>([&](auto sub) {
        constexpr int set = decltype(sub)::value;
        if (t + set >= steps) return;
        const char* cur = lds + (((t + set) & 1) ? kBuf : 0);
        char* next = lds + (((t + set) & 1) ? 0 : kBuf);
        if (t + set + 1 < mine) {
          tp.store(set, next);
          tq.store(set, next + BM * 128);
          load(set);
        }
        if (t + set < mine) compute(cur, wm, wn, [](auto) {});
        __syncthreads();
      });
    }
    if constexpr (SHARES == 2) {  // the buffers are free: the second group's sums to the first
      static_assert(kLds >= BM * BN * 4, "the sums fit the buffers");
      join_shares(acc, all_lds, tid, share);
    }
  }
};

// out[m, n] for grouped rows m: P the rows, Q the weights (QT: their transposes).  A tile
// whose rows hold no entry, and those behind an expert's last, are cleared.
template <int BM, int BN, int WM, int WN, int SETS, int SHARES, bool QT>
__global__ __launch_bounds__(64 * WM * WN * SHARES) void k_bf16_grouped_gemm(const uint16_t* __restrict__ rows, int64_t K,
                                                                    const uint16_t* __restrict__ weight, int64_t N,
                                                                    Groups gr, uint16_t* __restrict__ out) {
  typedef Product<BM, BN, WM, WN, false, QT, SETS, SHARES> P;
  extern __shared__ char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  Span s;
  int tn;
  if (!find_span<BM>(gr, (int)((N + BN - 1) / BN), s, tn)) return;
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
  if (s.extent > BM)
    clear_rows(out + (int64_t)s.row0 * N + n0, N, BM, s.extent, (int)min((int64_t)BN, N - n0));
  if (wave >= WM * WN) return;
  const int m = wm * P::MT * 16, n = n0 + wn * 64;
  store_block64<P::MT>(prod.acc, lds + wave * P::MT * 2048, out + (int64_t)(s.row0 + m) * N + n, N, s.used - m,
                       s.extent - m, (int)min((int64_t)64, N - n));
}

// out[m, n] for experts with few rows, where the time is that of reading the weights.
// A workgroup takes 16 RT weight rows of one expert and 16 NT of its rows at a time (the
// z-th of gridDim.z first, then every gridDim.z-th); its waves take the sum's steps of
// 128 terms in turn and join their sums through LDS.  Weights and rows go from memory to
// registers, four lanes on 64 contiguous bytes (a lane a row costs the L1 four times the
// accesses), and are brought into the instruction's order within lane quads; a step's
// loads are in flight while the step before is multiplied.  One token, 2 of 8 experts of
// 4096 x 4096: 14 us for 68 MB (4.8 TB/s; the first loads' latency and the join are a
// third); 128 rows of 32 experts of 4096 x 7168: 307 us for 1.88 GB (6.1 TB/s).
template <int RT, int NT>
__global__ __launch_bounds__(NT == 1 ? 512 : 256) void k_bf16_grouped_few(const uint16_t* __restrict__ rows, int64_t K,
                                                          const uint16_t* __restrict__ weight, int64_t N, Groups gr,
                                                          uint16_t* __restrict__ out) {
  extern __shared__ char lds[];
  float* red = reinterpret_cast<float*>(lds);  // [waves][RT * NT][16 rows][16 columns]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), W = blockDim.x >> 6;
  const int n0 = (int)blockIdx.x * 16 * RT, cols = (int)min((int64_t)16 * RT, N - n0);
  const int e = blockIdx.y;
  int lo, hi, cnt, clear;
  if (!few_rows(gr, lo, hi, cnt, clear)) return;
  clear_rows(out + (int64_t)lo * N + n0, N, clear, hi - lo, cols);

  // lane 16 g + 4 b + c loads, for j = 0..3, chunk 4 g + c (8 terms) of row 4 b + j; the
  // quad's exchange leaves chunk 4 g + j of row 4 b + c in register j
  const int g = lane >> 4, b4 = lane & 12, k0 = 8 * (4 * g + (lane & 3));
  const uint16_t* w = weight + ((int64_t)e * N + n0) * K + k0;
  uint32_t woff[RT][4];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) woff[i][j] = (uint32_t)min(16 * i + b4 + j, cols - 1) * (uint32_t)K;
  const int steps = (int)((K + 127) / 128);
  struct Step {
    u32x4 w[RT][4], x[NT][4];
  };
  for (int c0 = 16 * NT * (int)blockIdx.z; c0 < cnt; c0 += 16 * NT * (int)gridDim.z) {
    const int used = min(cnt - c0, 16 * NT);
    const uint16_t* x = rows + (int64_t)(lo + c0) * K + k0;
    uint32_t xoff[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) xoff[i][j] = (uint32_t)min(16 * i + b4 + j, used - 1) * (uint32_t)K;
    f32x4 acc[NT][RT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < RT; ++i) acc[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto load = [&](int s, Step& d) {
      const int at = s * 128, left = (int)min((int64_t)K - at - k0, (int64_t)8);
      if ((int64_t)at + 128 <= K) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int i = 0; i < RT; ++i) d.w[i][j] = ld_any<u32x4>(w + woff[i][j] + at);
#pragma unroll
          for (int i = 0; i < NT; ++i) d.x[i][j] = ld_any<u32x4>(x + xoff[i][j] + at);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int i = 0; i < RT; ++i) d.w[i][j] = load_end(w + woff[i][j] + at, left, K >= 8);
#pragma unroll
          for (int i = 0; i < NT; ++i) d.x[i][j] = load_end(x + xoff[i][j] + at, left, K >= 8);
        }
      }
    };
    auto multiply = [&](Step& d) {
#pragma unroll
      for (int i = 0; i < RT; ++i) quad_transpose(d.w[i]);
#pragma unroll
      for (int i = 0; i < NT; ++i) quad_transpose(d.x[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < RT; ++i)
            acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, d.w[i][j]),
                                                                __builtin_bit_cast(bf16x8, d.x[t][j]), acc[t][i], 0, 0, 0);
    };
    Step s0, s1;
    int s = wave;
    if (s < steps) load(s, s0);
    for (; s < steps; s += 2 * W) {
      if (s + W < steps) load(s + W, s1);
      multiply(s0);
      if (s + 2 * W < steps) load(s + 2 * W, s0);
      if (s + W < steps) multiply(s1);
    }
    join_few<RT, NT>(acc, red, out + (int64_t)(lo + c0) * N + n0, N, used, cols);
  }
}

// drows for experts with few rows: as k_bf16_grouped_few, but the weights' rows are the
// sum's terms: a wave's 64 of them by 64 columns go through LDS of its own, whose
// transposing read makes the instruction's operand.  One token, 2 of 8 experts of 4096 x
// 2048 (width first): 14.2 us for 34 MB, 64 blocks with work and 8 steps a wave; of 2048 x
// 4096, 128 blocks and 4 steps, 10.5 us; 128 rows, 8 experts of 4096 x 4096: 61 us for 270 MB.
__global__ __launch_bounds__(512) void k_bf16_grouped_few_across(const uint16_t* __restrict__ dout, int64_t N,
                                                                 const uint16_t* __restrict__ weight, int64_t K,
                                                                 Groups gr, uint16_t* __restrict__ drows) {
  extern __shared__ char lds[];  // 8 KB a wave; at the end [waves][4 * NT][16 rows][16 columns] floats
  typedef Tile<64, 64, true, 1> TileQ;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), W = blockDim.x >> 6;
  const int k0 = (int)blockIdx.x * 64, cols = (int)min((int64_t)64, K - k0), e = blockIdx.y;
  int lo, hi, cnt, clear;
  if (!few_rows(gr, lo, hi, cnt, clear)) return;
  clear_rows(drows + (int64_t)lo * K + k0, K, clear, hi - lo, cols);
  const int r = lane & 15, g = lane >> 4;
  char* own = lds + wave * 8192;
  constexpr int NT = 2;  // 32 rows at a time
  const int steps = (int)((N + 63) / 64);
  for (int c0 = 16 * NT * (int)blockIdx.z; c0 < cnt; c0 += 16 * NT * (int)gridDim.z) {
    const int used = min(cnt - c0, 16 * NT);
    const uint16_t* x = dout + (int64_t)(lo + c0) * N + 8 * g;
    uint32_t xoff[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xoff[t] = (uint32_t)min(16 * t + r, used - 1) * (uint32_t)N;
    const uint16_t* w = weight + ((int64_t)e * N + 64 * wave) * K + k0;
    f32x4 acc[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    struct Step {
      TileQ q;
      u32x4 x[NT][2];
    };
    Step s0, s1;
    s0.q.init(lane, K, cols);
    s1.q.init(lane, K, cols);
    auto load = [&](int s, Step& d) {
      const int left = (int)min(N - 64 * (int64_t)s, (int64_t)64);
      if (left == 64 && cols == 64) d.q.template load<false>(0, w, 64, 64);
      else d.q.template load<true>(0, w, left, cols);
      w += 64 * (int64_t)W * K;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          d.x[t][ks] = left == 64 ? ld_any<u32x4>(x + xoff[t] + 64 * s + 32 * ks)
                                  : load_end(x + xoff[t] + 64 * s + 32 * ks, left - 32 * ks - 8 * g, N >= 8);
    };
    auto multiply = [&](Step& d) {
      d.q.store(0, own);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 b = TileQ::frag(own, 16 * i, ks);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, __builtin_bit_cast(bf16x8, d.x[t][ks]), acc[t][i], 0, 0, 0);
        }
    };
    int s = wave;
    if (s < steps) load(s, s0);
    for (; s < steps; s += 2 * W) {
      if (s + W < steps) load(s + W, s1);
      multiply(s0);
      if (s + 2 * W < steps) load(s + 2 * W, s0);
      if (s + W < steps) multiply(s1);
    }
    __syncthreads();  // the waves' own LDS is free
    join_few<4, NT>(acc, reinterpret_cast<float*>(lds), drows + (int64_t)(lo + c0) * K + k0, K, used, cols);
  }
}

// Tiles of one expert's share that one XCD takes: as many as run there at once.
template <int BM>
constexpr int kWholeOnXcd = BM == 256 ? 32 : 64;

// dW of one expert, or one of `parts` shares of it (the rows' steps of 64 taken in
// equal runs; FP32, share i at out + i * E * N * K): P dout's columns, Q the rows'.  Short
// sums are bound by a tile's fixed costs: 222 rows an expert, 32 of 2040 x 2440, 200 us
// for 380 MB.
template <int BM, int BN, int WM, int WN, typename OUT>
__global__ __launch_bounds__(64 * WM * WN) void k_bf16_grouped_wgrad(const uint16_t* __restrict__ dout, int64_t N,
                                                                     const uint16_t* __restrict__ rows, int64_t K,
                                                                     Groups gr, int parts, OUT* __restrict__ out) {
  typedef Product<BM, BN, WM, WN, true, true, 1, 1> P;
  extern __shared__ char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  const int tm = (int)((N + BM - 1) / BM), tn = (int)((K + BN - 1) / BN);
  const int per = tm * tn, x = (int)(blockIdx.x & 7), at = (int)(blockIdx.x >> 3);  // x: the XCD
  int group, id;  // which share of which expert, and which of its tiles
  if (per <= kWholeOnXcd<BM>) {
    // all on one XCD, whose L2 then reads the share's rows once (32 experts of 512 x 512,
    // 4096 rows: 97 us, spread 130); an expert's shares on one after the other
    group = at / per * 8 + x;
    id = at % per;
  } else {
    // a run on each: experts differ in their rows, and whole ones would leave most XCDs
    // idle (16 of 1592 x 3304, loads by 1 / rank^1.2: 585 -> 199 us)
    const int run = (per + 7) >> 3;
    group = at / run;
    id = x * run + at % run;
  }
  if (group >= parts * gr.experts || id >= per) return;
  const int e = group / parts, part = group - e * parts;
  int i, j;
  banded(id, tm, tn, i, j);
  const int m0 = i * BM, n0 = j * BN;
  int lo, hi, cnt, tiles;
  group_rows(gr, e, BM, lo, hi, cnt, tiles);
  if (parts > 1) {
    const int run = ((cnt + parts - 1) / parts + kBK - 1) / kBK * kBK, first = min(part * run, cnt);
    lo += first;
    cnt = min(cnt - first, run);
  }
  P prod;
  prod.run(lds, dout + (int64_t)lo * N + m0, N, (int)min((int64_t)BM, N - m0), rows + (int64_t)lo * K + n0, K,
           (int)min((int64_t)BN, K - n0), cnt);
  const int m = m0 + wm * P::MT * 16, n = n0 + wn * 64;
  OUT* o = out + (((int64_t)part * gr.experts + e) * N + m) * K + n;
  const int rest = (int)(N - m), cols = (int)min((int64_t)64, K - n);
  if constexpr (sizeof(OUT) == 2) store_block64<P::MT>(prod.acc, lds + wave * P::MT * 2048, o, K, rest, rest, cols);
  else store_block64<P::MT>(prod.acc, lds + wave * P::MT * 2048, o, K, rest, cols);
}

// The shares' sums, in their order: 4 values a lane.
template <typename OUT>
__global__ __launch_bounds__(256) void k_wgrad_join(const float* __restrict__ part, int parts, int64_t n,
                                                    OUT* __restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const int left = (int)min(n - i, (int64_t)4);
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int p = 0; p < parts; ++p) {
    const float* at = part + p * n + i;
    if (left == 4) {
      const f32x4 w = ld_any<f32x4>(at);
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] += w[q];
    } else {
      for (int q = 0; q < left; ++q) v[q] += at[q];
    }
  }
  for (int q = 0; q < left; ++q) {
    if constexpr (sizeof(OUT) == 2) out[i + q] = __builtin_bit_cast(uint16_t, (__bf16)v[q]);
    else out[i + q] = v[q];
  }
}

}  // namespace mtb

using namespace mtb;

namespace {

// Sizes of the three products: r_cap grouped rows, [width, depth] weights.
int32_t check_sizes(int64_t r_cap, int64_t depth, int64_t width, int64_t experts, const int32_t* counts,
                    const int32_t* offsets, bool plan = true) {
  if (r_cap < 0 || depth < 1 || width < 1 || experts < 1 || experts > 1024) return EP_ERR_SHAPE;
  if (plan && (!counts != !offsets || (!counts && experts != 1))) return EP_ERR_SHAPE;
  // a tile's rows are addressed by 32 bits of bytes
  if (r_cap >= ((int64_t)1 << 25) || depth > (1 << 20) || width > (1 << 20)) return EP_ERR_RANGE;
  return EP_OK;
}

template <int BM, int BN, int WM, int WN, int SETS, int SHARES, bool QT>
int32_t product_tiles(const uint16_t* rows, int64_t r_cap, int64_t K, const uint16_t* weight, int64_t E, int64_t N,
                const int32_t* counts, const int32_t* offsets, int64_t entries, uint16_t* out, hipStream_t s) {
  const Groups gr{counts, offsets, (int)E, (int)r_cap};
  const int64_t blocks = span_blocks(r_cap, E, !counts, entries, BM, (N + BN - 1) / BN);
  if (!grid_fits(blocks, 64 * WM * WN * SHARES)) return EP_ERR_RANGE;
  const size_t lds = Product<BM, BN, WM, WN, false, QT, SETS, SHARES>::kLds;
  hipLaunchKernelGGL((k_bf16_grouped_gemm<BM, BN, WM, WN, SETS, SHARES, QT>), dim3((unsigned)blocks), dim3(64 * WM * WN * SHARES), lds, s, rows, K,
                     weight, N, gr, out);
  return launch_status();
}

template <int RT, int NT>
int32_t product_few(const uint16_t* rows, int64_t r_cap, int64_t K, const uint16_t* weight, int64_t E, int64_t N,
                    const int32_t* counts, const int32_t* offsets, dim3 grid, uint16_t* out, int waves, hipStream_t s) {
  const Groups gr{counts, offsets, (int)E, (int)r_cap};
  const int W = K > 128 * (waves - 1) ? waves : (int)((K + 127) / 128);  // no wave without a step
  grid.x = (unsigned)((N + 16 * RT - 1) / (16 * RT));
  hipLaunchKernelGGL((k_bf16_grouped_few<RT, NT>), grid, dim3(64 * W), (size_t)W * RT * NT * 1024, s, rows, K, weight, N, gr,
                     out);
  return launch_status();
}

int32_t product_few_across(const uint16_t* dout, int64_t r_cap, int64_t N, const uint16_t* weight, int64_t E, int64_t K,
                           const int32_t* counts, const int32_t* offsets, dim3 grid, uint16_t* drows, hipStream_t s) {
  const Groups gr{counts, offsets, (int)E, (int)r_cap};
  const int W = N > 64 * 7 ? 8 : (int)((N + 63) / 64);  // no wave without a step
  grid.x = (unsigned)((K + 63) / 64);
  hipLaunchKernelGGL(k_bf16_grouped_few_across, grid, dim3(64 * W), (size_t)W * 8192, s, dout, N, weight, K, gr, drows);
  return launch_status();
}

template <bool QT>
int32_t product(const uint16_t* rows, int64_t r_cap, int64_t K, const uint16_t* weight, int64_t E, int64_t N,
                const int32_t* counts, const int32_t* offsets, int64_t entries, uint16_t* out, hipStream_t s) {
  if (r_cap == 0) return EP_OK;
  if (!rows || !weight || !out) return EP_ERR_NULL;
  const int64_t most = entries < r_cap ? entries : r_cap, mean = (most + E - 1) / E;
  // Few rows an expert (on average), or so few results that tiles would leave most CUs
  // idle: by blocks of 32 rows whose waves share out the sum.  8 experts of 4096 x 4096,
  // 4 rows each, 47 us (tiles 77); 32 of 4096 x 7168, 8 rows 312 (384), 16 rows 318 (390),
  // 32 rows 460 (396).  With more rows, up to 512 blocks: 4 experts of 512 x 1024, 256 rows
  // each (512 blocks), 10.7 (13.0), 512 rows each (1024) 16.5 (13.3); 8 of 512 x 4096, 96 rows
  // (384) 26 (34), 128 rows (512) 34.5 (33.8), 256 rows (1024) 67 (34); 4 of 2048 x 2048, 64
  // rows (512) 18.2 (19.8), 128 rows (1024) 27 (20).
  const int64_t chunks = (mean + 31) / 32;
  // Where the weights are read across, blocks are 64 columns wide, and many of them that
  // read each weight once are better off as tiles: 8 experts of 4096 x 4096, 16 rows, 63
  // (82); 32 of 4096 x 7168, 8 rows, 417 (386).  With more rows, up to 256 blocks: 4 experts
  // of 1024 x 1024 (drows' columns first), 128 rows each, 13.2 (13.8); 2 of 1024 x 4096, 128
  // rows (128 blocks), 18 (36); 8 of 2048 x 2048, 32 rows (256), 25 (21).
  const int64_t used = E < most ? E : most;  // experts with rows, at most
  const bool few = QT ? (mean <= 24 && used * ((N + 127) / 128) <= 1024) || E * ((N + 63) / 64) * chunks <= 256
                      : mean <= 24 || E * ((N + 31) / 32) * chunks <= 512;
  // workgroups beside each other for one expert's rows: as many as the mean asks for,
  // more (the loads may be uneven) where that leaves few
  const int64_t spare = 1024 / (E * ((N + 63) / 64)), all = (most + 31) / 32;
  const int64_t beside = std::clamp<int64_t>(std::max(chunks, std::min(spare, all)), 1, 32767);
  const int64_t groups = few_groups(r_cap, E, !counts, beside);
  if (few && groups <= 65535) {
    const dim3 grid(1, (unsigned)groups, (unsigned)beside);
    if constexpr (QT) return product_few_across(rows, r_cap, K, weight, E, N, counts, offsets, grid, out, s);
    // up to 12 rows 16 at a time by eight waves: 4 rows 47 us and 64, 8 rows 320 and 312,
    // 16 rows 430 and 318
    // (or where that leaves few workgroups: 48 rows times 86 x 4737, 2 experts, 11.1 us and
    // 18.1; 156 times 27 x 5888, 8 experts, 12.6 and 15.7)
    else if (mean <= 12 || E * ((N + 15) / 16) * ((mean + 15) / 16) <= 512)
      return product_few<1, 1>(rows, r_cap, K, weight, E, N, counts, offsets, dim3(1, grid.y, mean <= 12 ? grid.z : 2 * grid.z),
                               out, 8, s);
    else return product_few<2, 2>(rows, r_cap, K, weight, E, N, counts, offsets, grid, out, 4, s);
  }
  // Large tiles from 192 rows an expert on where they reach about half of the CUs: 8
  // experts of 4096 x 4096, 256 rows each (128 tiles) 112 us, by small ones 162; 128 rows
  // each 101 and 95; 4 experts of 1024 x 2048, 512 rows each (32 tiles) 48 and 33.
  if (mean >= 192 && E * ((mean + 255) / 256) * ((N + 255) / 256) >= 112)
    return product_tiles<256, 256, 2, 4, 1, 1, QT>(rows, r_cap, K, weight, E, N, counts, offsets, entries, out, s);
  // Small ones: where they are fewer than the CUs (or as many, and the sum long) two
  // groups of waves share the sum (4
  // experts of 1024 x 2048, 512 rows: 21.5 us, by one group 28; of 4096 x 4096, 8 rows,
  // 95 and 77), and else two steps' loads are under way (32 of 4096 x 7168, 32 rows: 406
  // us, with one 445; where the weights are read across 492 and 402).
  const int64_t tiles = E * ((mean + 127) / 128) * ((N + 127) / 128);
  if (tiles <= 192 || (tiles <= 256 && K >= 1536) || (QT && mean <= 24))
    return product_tiles<128, 128, 2, 2, 1, 2, QT>(rows, r_cap, K, weight, E, N, counts, offsets, entries, out, s);
  return product_tiles<128, 128, 2, 2, QT ? 1 : 2, 1, QT>(rows, r_cap, K, weight, E, N, counts, offsets, entries, out, s);
}

template <int BM, int BN, int WM, int WN, typename OUT>
int32_t wgrad_tiles(const uint16_t* dout, const uint16_t* rows, int64_t width, int64_t hidden, const Groups& gr, int parts,
                    OUT* out, hipStream_t s) {
  const int64_t per = ((width + BM - 1) / BM) * ((hidden + BN - 1) / BN), groups = (int64_t)parts * gr.experts;
  const int64_t blocks = per <= kWholeOnXcd<BM> ? (groups + 7) / 8 * 8 * per : groups * ((per + 7) / 8 * 8);
  if (!grid_fits(blocks, 64 * WM * WN)) return EP_ERR_RANGE;
  const size_t lds = Product<BM, BN, WM, WN, true, true, 1, 1>::kLds;
  hipLaunchKernelGGL((k_bf16_grouped_wgrad<BM, BN, WM, WN, OUT>), dim3((unsigned)blocks), dim3(64 * WM * WN), lds, s, dout,
                     width, rows, hidden, gr, parts, out);
  return launch_status();
}

// Into how many shares an expert's rows are cut (by the mean): where 128 x 128 tiles are
// fewer than two a CU (four where the shares are small to store), as many as make up for
// it, each of 256 (128) rows at least.  2 experts of 512 x 512, 8192 rows each: 107 us
// whole, 25 in 16 shares.
int wgrad_parts(int64_t width, int64_t hidden, int64_t E, int64_t entries) {
  const int64_t tiles = E * ((width + 127) / 128) * ((hidden + 127) / 128);
  const int64_t more = E * width * hidden <= (1 << 20) ? 2 : 1;
  int64_t parts = more * 512 / tiles, most = more * (entries / E) / 256;
  parts = parts < most ? parts : most;
  return (int)(parts < 2 ? 1 : parts > 16 ? 16 : parts);
}

template <typename OUT>
int32_t wgrad(const uint16_t* dout, const uint16_t* rows, int64_t width, int64_t hidden, const Groups& gr, int64_t entries,
              OUT* out, float* workspace, hipStream_t s) {
  const int parts = wgrad_parts(width, hidden, gr.experts, entries);
  if (parts > 1) {
    const int32_t st = wgrad_tiles<128, 128, 2, 2>(dout, rows, width, hidden, gr, parts, workspace, s);
    if (st != EP_OK) return st;
    const int64_t n = gr.experts * width * hidden;
    hipLaunchKernelGGL(k_wgrad_join<OUT>, dim3((unsigned)((n + 1023) / 1024)), dim3(256), 0, s, workspace, parts, n, out);
    return launch_status();
  }
  // Large tiles where they are as many as the CUs: 8 experts of 4096 x 4096 (2048 tiles),
  // 512 rows each, 175 us, by small ones 234; 32 of 512 x 512 (128), 4096 rows, 105 and 97;
  // 4 of 1024 x 2048 (128), 2048 rows, 55 (57 in two shares) and 45.
  if (gr.experts * ((width + 255) / 256) * ((hidden + 255) / 256) >= 256)
    return wgrad_tiles<256, 256, 2, 4>(dout, rows, width, hidden, gr, 1, out, s);
  return wgrad_tiles<128, 128, 2, 2>(dout, rows, width, hidden, gr, 1, out, s);
}

}  // namespace

MTB_EXPORT int32_t ep_bf16_grouped_gemm(const uint16_t* rows, int64_t r_cap, int64_t hidden, const uint16_t* weight,
                                        int64_t num_experts, int64_t width, const int32_t* counts,
                                        const int32_t* offsets, int64_t entries, uint16_t* out, void* stream) {
  const int32_t st = check_sizes(r_cap, hidden, width, num_experts, counts, offsets);
  if (st != EP_OK) return st;
  if (entries < 0) return EP_ERR_SHAPE;
  if (entries >= kSizeLimit) return EP_ERR_RANGE;
  return product<false>(rows, r_cap, hidden, weight, num_experts, width, counts, offsets, entries, out, (hipStream_t)stream);
}

MTB_EXPORT int32_t ep_bf16_grouped_dgrad(const uint16_t* dout, int64_t r_cap, int64_t width, const uint16_t* weight,
                                         int64_t num_experts, int64_t hidden, const int32_t* counts,
                                         const int32_t* offsets, int64_t entries, uint16_t* drows, void* stream) {
  const int32_t st = check_sizes(r_cap, hidden, width, num_experts, counts, offsets);
  if (st != EP_OK) return st;
  if (entries < 0) return EP_ERR_SHAPE;
  if (entries >= kSizeLimit) return EP_ERR_RANGE;
  return product<true>(dout, r_cap, width, weight, num_experts, hidden, counts, offsets, entries, drows, (hipStream_t)stream);
}

MTB_EXPORT size_t ep_bf16_grouped_wgrad_workspace_bytes(int64_t width, int64_t hidden, int64_t num_experts,
                                                        int64_t entries) {
  if (check_sizes(0, hidden, width, num_experts, nullptr, nullptr, false) != EP_OK || entries < 0 || entries >= kSizeLimit)
    return 0;
  const int parts = wgrad_parts(width, hidden, num_experts, entries);
  return parts > 1 ? (size_t)(parts * num_experts * width * hidden) * 4 : 0;
}

MTB_EXPORT int32_t ep_bf16_grouped_wgrad(const uint16_t* dout, const uint16_t* rows, int64_t r_cap, int64_t width,
                                         int64_t hidden, int64_t num_experts, const int32_t* counts,
                                         const int32_t* offsets, int64_t entries, void* dweight, int32_t f32, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  const int32_t st = check_sizes(r_cap, hidden, width, num_experts, counts, offsets);
  if (st != EP_OK) return st;
  if (entries < 0) return EP_ERR_SHAPE;
  if (entries >= kSizeLimit) return EP_ERR_RANGE;
  if (!dweight || (r_cap > 0 && (!dout || !rows))) return EP_ERR_NULL;
  const size_t need = ep_bf16_grouped_wgrad_workspace_bytes(width, hidden, num_experts, entries);
  if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 15))) return EP_ERR_WORKSPACE;
  const Groups gr{counts, offsets, (int)num_experts, (int)r_cap};
  if (f32)
    return wgrad(dout, rows, width, hidden, gr, entries, (float*)dweight, (float*)workspace, (hipStream_t)stream);
  return wgrad(dout, rows, width, hidden, gr, entries, (uint16_t*)dweight, (float*)workspace, (hipStream_t)stream);
}
