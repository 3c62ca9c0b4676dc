// Products of grouped MXFP4 or MXFP8 rows with MXFP4 weights:
//   out[g, n] = sum over blocks b of 32 of 2^(sa[g, b] - 127) 2^(sw[n, b] - 127)
//               sum_i a[g, 32 b + i] w[n, 32 b + i]
// on v_mfma_scale_f32_16x16x128_f8f6f4, which takes the codes and the blocks'
// scale bytes as they are stored.  Sums are FP32 and every product is exact in them.
// The instruction adds eight neighbouring products at a time, each cut 13 bits below the
// largest one's exponent (of the factors' own: mantissas do not count).  E2M1 products
// span 2^7 and lose nothing; E4M3 times E2M1 span 2^21, so MXFP8 rows are multiplied as
// the sum of two parts of eight exponents each (split_e4m3), which lose nothing either: at
// twice the instructions, the BF16 rate, and as exact as decoding to BF16, without the
// decoded operands' LDS and registers.
//
// Measured: 131072 MXFP4 rows of 32 experts, 7168 x 4096, 2.24 to 2.41 ms, 3190 to 3430
// TFLOP/s (the unit's own rate is 10 PFLOP/s, 2.5 for MXFP8 rows); 32768 MXFP8 rows of 8
// experts, 4096 x 4096, 0.88 ms, 1250 TFLOP/s.  A step has the bytes of a BF16 step of a
// quarter of its terms, and the same parts bound it: barriers, LDS reads behind them, a
// tile's first loads and its stores, 28 steps in 7168 values instead of 112.  A second
// set of loads under way did not help (the small tiles then spill).
#include "common.h"
#include "grouped.h"
#include "launch.h"

namespace mtb {

constexpr int kE2M1 = 4, kE4M3 = 0;  // the instruction's operand formats

__device__ __forceinline__ i32x8 wide(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// E4M3 bytes as the sum of those of magnitude 2 and more (exponents 1 to 8; the NaN) and
// the others (-6 to 0, the subnormals among them): bit 6 of a byte tells.  Zeros are in
// the places of values of the other part.
__device__ __forceinline__ void split_e4m3(u32x4 v, u32x4& high, u32x4& low) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // selectors 8 to 11 repeat bits 15 and 31 of the second and of the first source over a byte
    const uint32_t m = __builtin_amdgcn_perm(v[i] << 1, v[i] << 9, 0x0B090A08u);
    high[i] = v[i] & m;
    low[i] = v[i] & ~m;
  }
}

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
  int tid;  // of the THREADS that share the tile
  static constexpr int kRowPieces = RB / 16, kPieces = C * kRowPieces / THREADS;
  static constexpr int kWords = C * SB / 4, kSc = (kWords + THREADS - 1) / THREADS;
  static constexpr int kBytes = C * (RB + SB);
  uint32_t off[kPieces], soff[kSc];
  u32x4 v[kPieces];
  uint32_t sv[kSc];

  __device__ __forceinline__ void init(int thread, int64_t row_bytes, int64_t row_blocks, int c_n) {
    tid = thread;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int p = tid + i * THREADS;
      off[i] = (uint32_t)(min(p / kRowPieces, c_n - 1) * (uint32_t)row_bytes + 16 * (p % kRowPieces));
    }
#pragma unroll
    for (int i = 0; i < kSc; ++i) {
      const int p = min(tid + i * THREADS, kWords - 1);
      soff[i] = (uint32_t)(min(p / (SB / 4), c_n - 1) * (uint32_t)row_blocks + 4 * (p % (SB / 4)));
    }
  }
  // bytes and blocks: what is left of a row from the step's first value on; values
  // past it are zeros.
  template <bool EDGE>
  __device__ __forceinline__ void load_piece(int i, const uint8_t* codes, int bytes) {
    const int p = tid + i * THREADS;
    if (!EDGE || 16 * (p % kRowPieces) < bytes) v[i] = ld_any<u32x4>(codes + off[i]);
    else v[i] = u32x4{0u, 0u, 0u, 0u};
  }
  template <bool EDGE>
  __device__ __forceinline__ void load_scales(const uint8_t* scales, int blocks) {
#pragma unroll
    for (int i = 0; i < kSc; ++i) {
      if (!EDGE) {
        sv[i] = ld_any<uint32_t>(scales + soff[i]);
        continue;
      }
      const int p = min(tid + i * THREADS, kWords - 1), n = blocks - 4 * (p % (SB / 4));
      sv[i] = 0;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (b < n) sv[i] |= (uint32_t)scales[soff[i] + b] << (8 * b);
    }
  }
  template <bool EDGE>
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* scales, int bytes, int blocks) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) load_piece<EDGE>(i, codes, bytes);
    load_scales<EDGE>(scales, blocks);
  }
  __device__ __forceinline__ void store_piece(int i, char* lds) const {
    const int p = tid + i * THREADS;
    *reinterpret_cast<u32x4*>(lds + chunk_at<RB>(p / kRowPieces, p % kRowPieces)) = v[i];
  }
  // Eight scale bytes of a row (two lanes' words) are stored as 0, 4, 1, 5, 2, 6, 3, 7,
  // so that one 16-bit read has a lane group's blocks of both halves of a step.
  __device__ __forceinline__ void store_scales(char* lds) const {
#pragma unroll
    for (int i = 0; i < kSc; ++i) {
      const int p = tid + i * THREADS;
      uint32_t w = sv[i];
      if (SB == 8) {
        const uint32_t o = lane_xor1(w), lo = p & 1 ? o : w, hi = p & 1 ? w : o;
        w = __builtin_amdgcn_perm(hi, lo, p & 1 ? 0x07030602u : 0x05010400u);
      }
      if (kWords % THREADS == 0 || p < kWords) *reinterpret_cast<uint32_t*>(lds + C * RB + 4 * p) = w;
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) store_piece(i, lds);
    store_scales(lds);
  }
};

// One output tile of BM x BN per workgroup, 256 values (MXFP8 rows: 128) a step
// through two LDS buffers.  SHARES groups of WM x WN waves take the steps in turn, each
// through buffers of its own; the first ends with the sum.
template <int BM, int BN, int WM, int WN, int SHARES, bool A8>
struct MxProduct {
  static constexpr int kThreads = 64 * WM * WN, MT = BM / WM / 16, NT = BN / WN / 16;
  static constexpr int kStep = A8 ? 128 : 256, SB = kStep / 32, kRowW = kStep / 2;
  typedef MxTile<BM, kThreads, 128, SB> TileA;
  typedef MxTile<BN, kThreads, kRowW, SB> TileW;
  static constexpr int kBuf = TileA::kBytes + TileW::kBytes;
  static constexpr int kOut = WM * WN * MT * 2048, kAll = 2 * SHARES * kBuf, kLds = kAll > kOut ? kAll : kOut;
  f32x4 acc[MT][NT];

  // A step's products in kParts parts, `between(part)` called before each.
  static constexpr int kParts = A8 ? MT : 8;
  template <typename F>
  __device__ __forceinline__ void compute(const char* a_lds, const char* w_lds, int wm, int wn, F&& between) {
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
    if constexpr (A8) {
      // lane group g: weights 32 g .. + 31, row values 16 g .. + 15 and 64 + 16 g .. + 15,
      // the scale of values 32 g .. + 31, as the instruction has them
      u32x4 w[NT], a[2][2];
#pragma unroll
      for (int i = 0; i < NT; ++i)
        w[i] = *reinterpret_cast<const u32x4*>(w_lds + chunk_at<kRowW>(16 * (wn * NT + i) + r, g));
      auto read = [&](auto part) {
        constexpr int c = decltype(part)::value;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          a[c & 1][h] = *reinterpret_cast<const u32x4*>(a_lds + chunk_at<128>(16 * (wm * MT + c) + r, 4 * h + g));
      };
      read(std::integral_constant<int, 0>{});
      static_for<0, kParts>([&](auto part) {
        constexpr int c = decltype(part)::value;
        // ahead of the stores in `between`, which no LDS read passes
        if constexpr (c + 1 < kParts) read(std::integral_constant<int, c + 1>{});
        between(part);
        u32x4 high[2], low[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) split_e4m3(a[c & 1][h], high[h], low[h]);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          acc[c][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(w[i], none), wide(low[0], low[1]), acc[c][i],
                                                                       kE2M1, kE4M3, 0, sw[i], 0, sa[c]);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          acc[c][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(w[i], none), wide(high[0], high[1]), acc[c][i],
                                                                       kE2M1, kE4M3, 0, sw[i], 0, sa[c]);
      });
    } else {
      // lane group g: values 32 g .. + 31 of the step's first half, then of its second
      // (neighbouring chunks: groups that took every other one would meet in LDS's banks).
      // Rows' operands are read as needed: a part ahead took 41 us instead of 30 (1024 rows
      // of 8 experts, 4096 x 4096, small tiles) and 2340 instead of 2310 (large ones).
      u32x4 w[NT];
      static_for<0, kParts>([&](auto part) {
        constexpr int c = decltype(part)::value, S = c / 4, J = MT / 4;
        if constexpr (c % 4 == 0) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
            w[i] = *reinterpret_cast<const u32x4*>(w_lds + chunk_at<kRowW>(16 * (wn * NT + i) + r, 4 * S + g));
        }
        between(part);
#pragma unroll
        for (int j = c % 4 * J; j < (c % 4 + 1) * J; ++j) {
          const u32x4 a = *reinterpret_cast<const u32x4*>(a_lds + chunk_at<128>(16 * (wm * MT + j) + r, 4 * S + g));
#pragma unroll
          for (int i = 0; i < NT; ++i)
            acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(w[i], none), wide(a, none), acc[j][i], kE2M1,
                                                                         kE2M1, S, sw[i], S, sa[j]);
        }
      });
    }
  }

  __device__ __forceinline__ void run(char* all_lds, const uint8_t* a, const uint8_t* as, int a_n, const uint8_t* w,
                                      const uint8_t* ws, int w_n, int K) {
    const int share = SHARES == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    const int tid = threadIdx.x - share * kThreads;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave / WN, wn = wave % WN;
    char* lds = all_lds + share * 2 * kBuf;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (K <= 0) return;
    TileA ta;
    TileW tw;
    ta.init(tid, A8 ? K : K / 2, K / 32, a_n);
    tw.init(tid, K / 2, K / 32, w_n);
    const int all = (K + kStep - 1) / kStep, steps = (all + SHARES - 1) / SHARES;
    const int mine = (all - share + SHARES - 1) / SHARES;  // steps of this group; the first has `steps`
    int left = K - share * kStep;  // from this group's next step on: values that are not loaded yet
    a += share * 128;
    as += share * SB;
    w += share * kRowW;
    ws += share * SB;
    auto advance = [&]() {
      a += SHARES * 128;
      as += SHARES * SB;
      w += SHARES * kRowW;
      ws += SHARES * SB;
      left -= SHARES * kStep;
    };
    auto load = [&]() {
      if (left <= 0) return;
      if (left >= kStep) {
        ta.template load<false>(a, as, 0, 0);
        tw.template load<false>(w, ws, 0, 0);
      } else {
        ta.template load<true>(a, as, A8 ? left : left / 2, left / 32);
        tw.template load<true>(w, ws, left / 2, left / 32);
      }
      advance();
    };
    load();
    if (mine > 0) {
      ta.store(lds);
      tw.store(lds + TileA::kBytes);
    }
    load();
    __syncthreads();
    // The steps whose loads (two steps ahead) are whole: the next step's values on their
    // way to LDS and the one after's to the registers they leave, between the products.
    int t = 0;
    for (; t < K / kStep / SHARES - 2; ++t) {  // as many for each group
      const char* cur = lds + ((t & 1) ? kBuf : 0);
      char* next = lds + ((t & 1) ? 0 : kBuf);
      compute(cur, cur + TileA::kBytes, wm, wn, [&](auto part) {
        constexpr int c = decltype(part)::value, P = TileA::kPieces + TileW::kPieces;
        if constexpr (c == 0) {
          ta.store_scales(next);
          tw.store_scales(next + TileA::kBytes);
          ta.template load_scales<false>(as, 0);
          tw.template load_scales<false>(ws, 0);
        }
        static_for<c * P / kParts, (c + 1) * P / kParts>([&](auto piece) {
          constexpr int i = decltype(piece)::value;
          if constexpr (i < TileA::kPieces) {
            ta.store_piece(i, next);
            ta.template load_piece<false>(i, a, 0);
          } else {
            tw.store_piece(i - TileA::kPieces, next + TileA::kBytes);
            tw.template load_piece<false>(i - TileA::kPieces, w, 0);
          }
        });
      });
      advance();
      __syncthreads();
    }
    for (; t < steps; ++t) {
      const char* cur = lds + ((t & 1) ? kBuf : 0);
      char* next = lds + ((t & 1) ? 0 : kBuf);
      if (t + 1 < mine) {
        ta.store(next);
        tw.store(next + TileA::kBytes);
        load();
      }
      if (t < mine) compute(cur, cur + TileA::kBytes, wm, wn, [](auto) {});
      __syncthreads();
    }
    if constexpr (SHARES == 2) {  // the buffers are free
      static_assert(kLds >= BM * BN * 4, "the sums fit the buffers");
      join_shares(acc, all_lds, tid, share);
    }
  }
};

template <int BM, int BN, int WM, int WN, int SHARES, bool A8>
__global__ __launch_bounds__(64 * WM * WN * SHARES) void k_mxfp4_grouped_gemm(const uint8_t* __restrict__ data,
                                                                     const uint8_t* __restrict__ scales, int K,
                                                                     const uint8_t* __restrict__ wcodes,
                                                                     const uint8_t* __restrict__ wscales, int64_t N,
                                                                     Groups gr, uint16_t* __restrict__ out) {
  typedef MxProduct<BM, BN, WM, WN, SHARES, A8> P;
  extern __shared__ char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wm = wave / WN, wn = wave % WN;
  Span s;
  int tn;
  if (!find_span<BM>(gr, (int)((N + BN - 1) / BN), s, tn)) return;
  P prod;
  const int n0 = tn * BN;
  const int64_t row = s.row0, col = (int64_t)s.expert * N + n0;
  if (s.used > 0)
    prod.run(lds, data + row * (A8 ? K : K / 2), scales + row * (K / 32), s.used, wcodes + col * (K / 2),
             wscales + col * (K / 32), (int)min((int64_t)BN, N - n0), K);
  else
    prod.run(lds, data, scales, 1, wcodes, wscales, 1, 0);
  static_assert(P::NT % 4 == 0, "a wave stores 64 columns at a time");
  if (s.extent > BM)
    clear_rows(out + row * N + n0, N, BM, s.extent, (int)min((int64_t)BN, N - n0));
  if (wave >= WM * WN) return;
  const int m = wm * P::MT * 16;
  static_for<0, P::NT / 4>([&](auto block) {
    constexpr int b = decltype(block)::value;
    f32x4 acc[P::MT][4];
#pragma unroll
    for (int j = 0; j < P::MT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = prod.acc[j][4 * b + i];
    const int n = n0 + (wn * P::NT / 4 + b) * 64;
    store_block64<P::MT>(acc, lds + wave * P::MT * 2048, out + (row + m) * N + n, N, s.used - m, s.extent - m,
                         (int)min((int64_t)64, N - n));
  });
}

// For experts with few rows, where the time is that of reading the weights.  A
// workgroup takes 16 RT weight rows of one expert and 16 of its rows at a time (the
// z-th of gridDim.z first, then every gridDim.z-th); its waves take the sum's steps of
// 512 values in turn and join their sums through LDS.  Codes go from memory to
// registers, four lanes on 64 contiguous bytes, and are brought into the instruction's
// order within lane quads; a step's loads are in flight while the step before is
// multiplied.  One token, 2 of 8 experts of 4096 x 2048: 4.5 us for 9.9 MB; 128 rows of 32
// experts of 4096 x 7168: 94 us for 500 MB (5.3 TB/s), MXFP8 rows 143.
template <int RT, bool A8>
__global__ __launch_bounds__(256, 2) void k_mxfp4_grouped_few(
    const uint8_t* __restrict__ data, const uint8_t* __restrict__ scales, int K, const uint8_t* __restrict__ wcodes,
    const uint8_t* __restrict__ wscales, int64_t N, Groups gr, uint16_t* __restrict__ out) {
  extern __shared__ char lds[];
  float* red = reinterpret_cast<float*>(lds);  // [waves][RT][16 rows][16 columns]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), W = blockDim.x >> 6;
  const int n0 = (int)blockIdx.x * 16 * RT, cols = (int)min((int64_t)16 * RT, N - n0), e = blockIdx.y;
  int lo, hi, cnt, clear;
  if (!few_rows(gr, lo, hi, cnt, clear)) return;
  clear_rows(out + (int64_t)lo * N + n0, N, clear, hi - lo, cols);

  // lane 16 g + 4 b + c loads, for j = 0..3, chunk 4 g + c (32 values) of row 4 b + j; the
  // quad's exchange leaves chunk 4 g + j of row 4 b + c in register j, lane group g's block
  // of the j-th product.  Of MXFP8 rows the instruction wants, beside a group's block
  // scales, 16 values of block g / 2 and 16 of block 2 + g / 2: chunks of 16 values.
  const int g = lane >> 4, r = lane & 15, b4 = lane & 12, c = lane & 3;
  const int wchunk = 4 * g + c, xchunk = A8 ? 8 * (g >> 1) + 2 * c + (g & 1) : wchunk;
  const uint32_t wrow = K / 2, xrow = A8 ? K : K / 2, srow = K / 32;
  const int64_t col = (int64_t)e * N + n0;
  const uint8_t* w = wcodes + col * wrow + 16 * wchunk;
  const uint8_t* ws = wscales + col * srow + 4 * g;
  uint32_t woff[RT][4], wsoff[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) woff[i][j] = (uint32_t)min(16 * i + b4 + j, cols - 1) * wrow;
    wsoff[i] = (uint32_t)min(16 * i + r, cols - 1) * srow;
  }
  const int steps = (K + 511) / 512;
  constexpr int H = A8 ? 2 : 1;
  struct Step {
    u32x4 w[RT][4], x[H][4];
    uint32_t sw[RT], sx;
  };
  auto scale4 = [](const uint8_t* p, int n) {
    if (n >= 4) return ld_any<uint32_t>(p);
    uint32_t v = 0;
#pragma unroll
    for (int b = 0; b < 3; ++b)
      if (b < n) v |= (uint32_t)p[b] << (8 * b);
    return v;
  };
  for (int c0 = 16 * (int)blockIdx.z; c0 < cnt; c0 += 16 * (int)gridDim.z) {
    const int used = min(cnt - c0, 16);
    const uint8_t* x = data + (int64_t)(lo + c0) * xrow + 16 * xchunk;
    const uint8_t* xs = scales + (int64_t)(lo + c0) * srow + 4 * g;
    uint32_t xoff[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) xoff[j] = (uint32_t)min(b4 + j, used - 1) * xrow;
    const uint32_t xsoff = (uint32_t)min(r, used - 1) * srow;
    f32x4 acc[1][RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[0][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto load = [&](int s, Step& d) {
      const u32x4 none = {0u, 0u, 0u, 0u};
      const int left = K - 512 * s;  // values from the step's first on
      const bool whole = left >= 512;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
          d.w[i][j] = whole || 32 * wchunk < left ? ld_any<u32x4>(w + woff[i][j] + 256 * s) : none;
#pragma unroll
        for (int h = 0; h < H; ++h)
          d.x[h][j] = whole || (A8 ? 16 * (xchunk + 16 * h) : 32 * xchunk) < left
                          ? ld_any<u32x4>(x + xoff[j] + (A8 ? 512 : 256) * s + 256 * h)
                          : none;
      }
      const int blocks = whole ? 4 : left / 32 - 4 * g;
#pragma unroll
      for (int i = 0; i < RT; ++i) d.sw[i] = scale4(ws + wsoff[i] + 16 * s, blocks);
      d.sx = scale4(xs + xsoff + 16 * s, blocks);
    };
    auto multiply = [&](Step& d) {
      const u32x4 none = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int i = 0; i < RT; ++i) quad_transpose(d.w[i]);
#pragma unroll
      for (int h = 0; h < H; ++h) quad_transpose(d.x[h]);
      static_for<0, 4>([&](auto block) {
        constexpr int j = decltype(block)::value;
        i32x8 x = wide(d.x[0][j], none);
        if constexpr (A8) {
          u32x4 high[2], low[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) split_e4m3(d.x[h][j], high[h], low[h]);
          x = wide(high[0], high[1]);
#pragma unroll
          for (int i = 0; i < RT; ++i)
            acc[0][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(d.w[i][j], none), wide(low[0], low[1]), acc[0][i],
                                                                         kE2M1, kE4M3, j, (int)d.sw[i], j, (int)d.sx);
        }
#pragma unroll
        for (int i = 0; i < RT; ++i)
          acc[0][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide(d.w[i][j], none), x, acc[0][i], kE2M1,
                                                                       A8 ? kE4M3 : kE2M1, j, (int)d.sw[i], j, (int)d.sx);
      });
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
    join_few<RT, 1>(acc, red, out + (int64_t)(lo + c0) * N + n0, N, used, cols);
  }
}

}  // namespace mtb

using namespace mtb;

namespace {
template <int BM, int BN, int WM, int WN, int SHARES, bool A8>
int32_t mx_tiles(const uint8_t* data, const uint8_t* scales, int64_t r_cap, int64_t K, const uint8_t* wcodes,
                   const uint8_t* wscales, int64_t E, int64_t N, const int32_t* counts, const int32_t* offsets,
                   int64_t entries, uint16_t* out, hipStream_t s) {
  const Groups gr{counts, offsets, (int)E, (int)r_cap};
  const int64_t blocks = span_blocks(r_cap, E, !counts, entries, BM, (N + BN - 1) / BN);
  if (!grid_fits(blocks, 64 * WM * WN * SHARES)) return EP_ERR_RANGE;
  const size_t lds = MxProduct<BM, BN, WM, WN, SHARES, A8>::kLds;
  hipLaunchKernelGGL((k_mxfp4_grouped_gemm<BM, BN, WM, WN, SHARES, A8>), dim3((unsigned)blocks), dim3(64 * WM * WN * SHARES), lds, s, data,
                     scales, (int)K, wcodes, wscales, N, gr, out);
  return launch_status();
}

template <int RT, bool A8>
int32_t mx_few(const uint8_t* data, const uint8_t* scales, int64_t r_cap, int64_t K, const uint8_t* wcodes,
               const uint8_t* wscales, int64_t E, int64_t N, const int32_t* counts, const int32_t* offsets, dim3 grid,
               uint16_t* out, hipStream_t s) {
  const Groups gr{counts, offsets, (int)E, (int)r_cap};
  const int W = K > 512 * 3 ? 4 : (int)((K + 511) / 512);  // no wave without a step
  grid.x = (unsigned)((N + 16 * RT - 1) / (16 * RT));
  hipLaunchKernelGGL((k_mxfp4_grouped_few<RT, A8>), grid, dim3(64 * W), (size_t)W * RT * 1024, s, data, scales, (int)K,
                     wcodes, wscales, N, gr, out);
  return launch_status();
}

template <bool A8>
int32_t mx_product(const uint8_t* data, const uint8_t* scales, int64_t r_cap, int64_t K, const uint8_t* wcodes,
                   const uint8_t* wscales, int64_t E, int64_t N, const int32_t* counts, const int32_t* offsets,
                   int64_t entries, uint16_t* out, hipStream_t s) {
  const int64_t most = entries < r_cap ? entries : r_cap, mean = (most + E - 1) / E;
  // Up to 16 rows an expert (on average) by the kernel that streams the weights, MXFP4
  // rows 32 weight rows at a time, MXFP8 rows, which take twice the registers, 16: 32
  // experts of 4096 x 7168, 8 rows each, 99 us (tiles 137) and 153 (231); 16 rows 132
  // (140) and 223 (234); 32 rows of MXFP4 199 (148).
  // With more rows, too, where a long sum would be left to few tiles: a workgroup for
  // each 16 rows, up to 1024 of them (MXFP8 rows 2048).  4096 values, MXFP4 rows: 8 experts
  // of width 512, 128 rows each (1024 workgroups), 14.8 us (tiles 17.7); one of 1024, 1024
  // rows (2048), 22.9 (18.2); 4 of 4096, 60 rows (2048), 26 (17).  MXFP8 rows: the first of
  // these (2048) 24.7 (31.6), the others (4096) 42 (32) and 44 (30).  8 of width 512, 64 rows
  // each, of 2048 values 9.5 (MXFP8 rows; tiles 16.6) and 9.3 (10.5), of 1024 9.3 (11.2); 4
  // of 256, 128 rows each, of 512 values alike.
  constexpr int RT = A8 ? 1 : 2;
  const int64_t chunks = mean > 16 ? (mean + 15) / 16 : 1;  // without entries, too: the rows are cleared
  const bool thin = K >= 1024 && E * ((N + 16 * RT - 1) / (16 * RT)) * chunks <= (A8 ? 2048 : 1024);
  const int64_t groups = few_groups(r_cap, E, !counts, chunks);
  if ((mean <= 16 || thin) && groups <= 65535)
    return mx_few<RT, A8>(data, scales, r_cap, K, wcodes, wscales, E, N, counts, offsets,
                          dim3(1, (unsigned)groups, (unsigned)chunks), out, s);
  // Large tiles from 192 rows an expert on.  MXFP4 rows: where they reach about half of the
  // CUs: 8 experts of 4096 x 4096, 259 rows each (256 tiles), 40 us, by small ones 52; 128
  // rows each 35 and 31; 4 experts of 1024 x 2048, 512 rows each (32 tiles), 22 and 13.
  // MXFP8 rows, whose waves split their rows' operands once in a small tile and four times
  // over in a large one: from six tiles a CU on: 8 experts of 4096 x 4096, 259 rows each 96
  // and 88, 2048 rows each (1024 tiles) 477 and 455, 4096 (2048 tiles) 880 and 887; 32 of
  // 4096 x 7168, 1024 rows each (2048 tiles), 1573 and 1638.
  if (mean >= 192 && E * ((mean + 255) / 256) * ((N + 255) / 256) >= (A8 ? 1536 : 112))
    return mx_tiles<256, 256, 2, 4, 1, A8>(data, scales, r_cap, K, wcodes, wscales, E, N, counts, offsets, entries, out, s);
  // Small ones: where they are fewer than the CUs two groups of waves share the sum (MXFP8
  // rows, 4 experts of 1024 x 2048, 512 rows each: 18.0 us, by one group 22.1; 8 of 4096 x
  // 4096, 128 rows each (256 tiles): 61.7 and 54.2).  MXFP8 rows' waves lie one below the
  // other, each with all of the tile's columns, so that no two split the same rows (8 of 4096
  // x 4096, 128 rows each: 54 us, two by two 61).
  constexpr int WM = A8 ? 4 : 2, WN = A8 ? 1 : 2;
  if (E * ((mean + 127) / 128) * ((N + 127) / 128) <= 192)
    return mx_tiles<128, 128, WM, WN, 2, A8>(data, scales, r_cap, K, wcodes, wscales, E, N, counts, offsets, entries, out, s);
  return mx_tiles<128, 128, WM, WN, 1, A8>(data, scales, r_cap, K, wcodes, wscales, E, N, counts, offsets, entries, out, s);
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
  if (entries >= kSizeLimit || r_cap >= ((int64_t)1 << 25) || hidden > (1 << 20) || width > (1 << 20)) return EP_ERR_RANGE;
  if (r_cap == 0) return EP_OK;
  if (!data || !scales || !weight_codes || !weight_scales || !out) return EP_ERR_NULL;
  if (row_format == EP_ROWS_MXFP8)
    return mx_product<true>(data, scales, r_cap, hidden, weight_codes, weight_scales, num_experts, width, counts, offsets,
                            entries, out, (hipStream_t)stream);
  return mx_product<false>(data, scales, r_cap, hidden, weight_codes, weight_scales, num_experts, width, counts, offsets,
                           entries, out, (hipStream_t)stream);
}
