// Few token rows times the NVFP4 weights of their experts: the products of an
// expert layer that serves single tokens, where each weight byte is used once
// or a few times and the time is that of reading it.
//
// A weight is e2m1 * s_b * t with at most 2 + 4 significant bits (t is a power
// of two), so it is exact in BF16 and its product with a BF16 activation is
// exact in FP32: the weights are decoded in registers and the sums made by
// v_mfma_f32_16x16x32_bf16, 16 weight rows by 16 entries, whose other columns
// are idle when fewer entries share the expert (the matrix unit is far from its
// rate; decoding, two instructions a weight, is the larger share).
#include "common.h"
#include "launch.h"

namespace mtb {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kStep = 512;  // K values of one wave step: 16 chunks of 32 per row
constexpr int kMaxEntries = 4096;
constexpr int kRsrcRaw = 0x00020000;  // word 3 of a raw (unstrided, untyped) buffer resource

// A step of a tile: 16 rows by 512 K values, 256 code bytes and 32 scale bytes a
// row.  Lane l = 16 g + 4 b + c loads, for j = 0..3, the 16 bytes of chunk 4 g + c
// of row 4 b + j: four neighbouring lanes read 64 contiguous bytes and an
// instruction four rows' 256 (a lane per row, the matrix operand's own order,
// costs the L1 four times the accesses).  A 4 x 4 transpose within each lane
// quad, registers against lanes, then leaves chunk 4 g + j of row 4 b + c in
// register j: row l % 16 and K group l / 16, as the matrix instruction wants it.
// Which 8 K values a lane group holds is free as long as both operands agree.
struct WTile {
  u32x4 c[4];
  uint2 s;  // the scale bytes of chunks 4 g .. 4 g + 3 of row 4 b + c
};

// The neighbour's value (lane ^ 1 or lane ^ 2) where `take`, else own.
template <int CTRL>
__device__ __forceinline__ uint32_t quad_mix(bool take, uint32_t other, uint32_t own) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)other, CTRL, 0xF, 0xF, true);
  return take ? o : own;
}

__device__ __forceinline__ void quad_transpose(u32x4* c) {
  const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
#pragma unroll
  for (int p = 0; p < 4; p += 2)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = c[p][w], y = c[p + 1][w];
      c[p][w] = quad_mix<0xB1>(odd, y, x);
      c[p + 1][w] = quad_mix<0xB1>(!odd, x, y);
    }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t x = c[p][w], y = c[p + 2][w];
      c[p][w] = quad_mix<0x4E>(high, y, x);
      c[p + 2][w] = quad_mix<0x4E>(!high, x, y);
    }
}

__device__ __forceinline__ bf16x8 decode8(uint32_t w, float s, float t) {
  const f32x2 p0 = fp4_unpack2<0>(w, t), p1 = fp4_unpack2<1>(w, t), p2 = fp4_unpack2<2>(w, t), p3 = fp4_unpack2<3>(w, t);
  u32x4 o = {bf16pair(p0[0] * s, p0[1] * s), bf16pair(p1[0] * s, p1[1] * s), bf16pair(p2[0] * s, p2[1] * s),
             bf16pair(p3[0] * s, p3[1] * s)};
  return __builtin_bit_cast(bf16x8, o);
}

// The b-th of four E4M3 scale bytes.
__device__ __forceinline__ float block_scale(uint32_t s, int b) {
  return b == 0   ? __builtin_amdgcn_cvt_f32_fp8((int)s, 0)
         : b == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)s, 1)
         : b == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)s, 2)
                  : __builtin_amdgcn_cvt_f32_fp8((int)s, 3);
}

// What a weight row is decoded with in place of its t, and what its sums are
// multiplied by.  Below t = 2^-32 every row is taken at 2^-32 instead: its weights
// are normal BF16 numbers then (the least is 2^-10 t, which small rows would lose),
// and no sum of up to 2^20 products with the largest activations leaves FP32's
// range (2^20 * 2688 * 2^-32 * 2^128 < 2^128).  Both steps are exact.
__device__ __forceinline__ float lift_row(float& t) {
  const bool small = t < 0x1p-32f;
  const float post = small ? t * 0x1p32f : 1.0f;
  t = small ? 0x1p-32f : t;
  return post;
}

// A tile's rows as a buffer: 16 from row `row` of expert e on, or fewer where the
// rows end; what lies past them reads as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rows(const uint8_t* weight, size_t first, int rows, uint32_t rb) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(weight) + first * rb, 0,
                                           (int)((uint32_t)min(16, rows) * rb), kRsrcRaw);
}

// This lane's share of a step of a tile at kb.
__device__ __forceinline__ void load_tile(__amdgpu_buffer_rsrc_t rows, uint32_t code, uint32_t scale, uint32_t rb,
                                          int kb, WTile& w) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w.c[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, (int)(code + j * rb + (kb >> 1)), 0, 0));
  w.s = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(rows, (int)(scale + (kb >> 4)), 0, 0));
}

// The codes in the matrix operand's order; scales of zero for K values past the row.
__device__ __forceinline__ void arrange(WTile& w, int kb, int K, int g) {
  quad_transpose(w.c);
  w.s.x = kb + 128 * g < K ? w.s.x : 0u;
  w.s.y = kb + 128 * g + 64 < K ? w.s.y : 0u;
}

// Four entries a lane, from `base` on (past the last: none).
template <typename IDX>
__device__ __forceinline__ void load_ids(const IDX* __restrict__ ids, int M, int base, IDX* id) {
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int i = base + u * (int)blockDim.x + (int)threadIdx.x;
    id[u] = i < M ? ids[i] : (IDX)-1;
  }
}

// The entries of expert e in order, and the rows of x they take; returns how
// many.  id: the first four of each lane, read before the first weights (loads
// come back in order: behind the weights they would wait for them).
template <typename IDX>
__device__ __forceinline__ int expert_entries(const IDX* __restrict__ ids, int M, int e, int x_div, IDX* id,
                                              uint16_t* list, uint16_t* xrows, int* wcount /* [4 * waves] */) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, B = blockDim.x, W = B >> 6;
  int n = 0;
  for (int base = 0; base < M; base += 4 * B) {
    bool hit[4];
    uint64_t m[4];
    if (base) load_ids(ids, M, base, id);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      hit[u] = id[u] == (IDX)e;
      m[u] = __builtin_amdgcn_ballot_w64(hit[u]);
      if (lane == 0) wcount[u * W + wave] = __popcll(m[u]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      int at = n;
      for (int w = 0; w < W; ++w) {
        if (w < wave) at += wcount[u * W + w];
        n += wcount[u * W + w];
      }
      if (!hit[u]) continue;
      const int i = base + u * B + tid;
      at += __popcll(m[u] & ((1ull << lane) - 1));
      list[at] = (uint16_t)i;
      xrows[at] = (uint16_t)(i / x_div);
    }
    __syncthreads();
  }
  return n;
}

// Zero rows, in the output columns [col0, col1), for the entries i0, i0 + step,
// ... that name no expert.
template <typename IDX>
__device__ __forceinline__ void clear_unnamed(const IDX* __restrict__ ids, int i0, int step, int M, int E, int col0,
                                              int col1, int NO, uint16_t* __restrict__ out, int32_t* d_error) {
  for (int i = i0; i < M; i += step) {
    const IDX id = ids[i];
    if (id >= 0 && id < E) continue;
    for (int c = col0; c < min(col1, NO); ++c) out[(size_t)i * NO + c] = 0;
    if (id != -1 && d_error && col0 == 0) atomicOr(d_error, EP_DEVERR_EXPERT_ID);
  }
}

// Few entries per expert, or few blocks.  One block per expert (by_entry: per
// entry, and the first with an expert takes all of that expert's; or several that
// take the expert's entries 16 at a time in turn) and WN * RT tiles of 16 weight
// rows.  WN waves side by side have RT tiles each; WK waves deep take the K steps
// in turn, and their sums are joined through LDS.  16 entries are taken in one
// pass over the weights; their activations come through LDS, kc columns at a time
// (a power of two, whole rounds of the WK waves), rows padded by 16 bytes so that
// the 16 entries of a read lie in different banks.
//
// 8 tokens, top-8 of 32 experts, 7168 x 2048: 61 us for 232 MB (3.8 TB/s); one
// token, top-8 of 32, 4096 x 7168 with SwiGLU: 30 us for 132 MB (4.4 TB/s); the
// same weights by a wave per output and entry: 133 us for the first.  What is left
// above the copy rate is a block's first loads, which the few blocks of such a
// call do not hide, and lines fetched twice: rows of 9 K / 16 + 4 bytes end
// inside 128-byte lines, and a line that two steps share has often left the L2
// in between (331 MB come past the L2 in the first call, 43% more than its bytes,
// at 5.5 TB/s; 718 for 530 MB at 32 tokens, top-8 of 32, 4096 x 7168; reading
// further ahead makes it more).
template <int RT, int WN, bool SWIGLU, typename IDX>
__global__ __launch_bounds__(512) void k_nvfp4_matvec(const uint16_t* __restrict__ x, int K, int x_div,
                                                      const uint8_t* __restrict__ weight, int E, int N,
                                                      const IDX* __restrict__ ids, int M, int by_entry, int lds_x,
                                                      uint16_t* __restrict__ out, int32_t* __restrict__ d_error) {
  extern __shared__ char smem[];
  __shared__ int wcount[4 * 8];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int WK = (blockDim.x >> 6) / WN, wn = wave % WN, wk = wave / WN;
  uint16_t* xs = reinterpret_cast<uint16_t*>(smem);            // [16][kc + 8]
  float* red = reinterpret_cast<float*>(smem);                 // [WK][WN][RT][16 entries][16 rows], after xs is done with
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + lds_x);  // the entries of this block's expert
  uint16_t* xrows = list + M;                                  // and their rows of x
  constexpr int GT = SWIGLU ? RT / 2 : RT;                     // tiles of output columns per wave
  const int NO = SWIGLU ? N / 2 : N, col0 = (int)blockIdx.x * (16 * GT * WN);
  const int r = lane & 15, g = lane >> 4;
  const uint32_t rb = 9 * ((uint32_t)K / 16) + 4;
  const uint32_t code = (uint32_t)(r & ~3) * rb + 16u * (4 * g + (r & 3)), scale = (uint32_t)r * rb + (K >> 1) + 8 * g;
  const int stride = WK * kStep, rounds = (K + stride - 1) / stride;  // K values of one round of the block

  int e = 0, n = M;
  IDX id4[4];
  if (ids) {
    load_ids(ids, M, 0, id4);
    e = blockIdx.y;
    if (by_entry)
      clear_unnamed(ids, tid == 0 ? e : M, M, M, E, col0, col0 + 16 * GT * WN, NO, out, d_error);
    else if (e == 0)
      clear_unnamed(ids, tid, blockDim.x, M, E, col0, col0 + 16 * GT * WN, NO, out, d_error);
    if (by_entry) {
      const IDX id = ids[e];
      if (id < 0 || id >= E) return;
      e = (int)id;
    }
  }
  // the first weights are on their way while the entries are found
  __amdgpu_buffer_rsrc_t rows[RT];
  WTile w[RT];
  float t[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row0 = min(col0 + 16 * (wn * GT + i % GT), NO);
    rows[i] = tile_rows(weight, (size_t)e * N + row0 + (SWIGLU && i >= GT ? NO : 0), NO - row0, rb);
    load_tile(rows[i], code, scale, rb, wk * kStep, w[i]);
    t[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rows[i], (int)((uint32_t)r * rb + (K >> 1) + (K >> 4)), 0, 0));
  }
  if (ids) {
    n = expert_entries(ids, M, e, x_div, id4, list, xrows, wcount);
    if (n == 0 || (by_entry && list[0] != blockIdx.y)) return;  // an earlier block has this expert
  } else {
    for (int i = tid; i < M; i += blockDim.x) list[i] = xrows[i] = (uint16_t)i;
    __syncthreads();
  }
  float post[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) post[i] = lift_row(t[i]);

  const int first = 16 * (int)blockIdx.z;
  for (int c0 = first; c0 < n; c0 += 16 * (int)gridDim.z) {
    const int cols = min(n - c0, 16);
    if (c0 != first) {
#pragma unroll
      for (int i = 0; i < RT; ++i) load_tile(rows[i], code, scale, rb, wk * kStep, w[i]);
    }
    // kc: as many columns of the entries as the LDS holds, in whole rounds
    int kc = stride;
    while (kc < K && cols * (2 * kc + 8) * 2 <= lds_x) kc *= 2;
    const int xrow = kc + 8;
    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    auto stage = [&](int k0) {  // activations [cols][k0, k0 + kc), zeros past K
      const int sh = 31 - __builtin_clz(kc >> 3), pieces = cols << sh;
      for (int p0 = tid; p0 < pieces; p0 += 8 * blockDim.x) {
        u32x4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int p = p0 + u * blockDim.x, k = k0 + 8 * (p & ((1 << sh) - 1));
          v[u] = u32x4{0u, 0u, 0u, 0u};
          if (p < pieces && k < K) v[u] = ld_any<u32x4>(x + (size_t)xrows[c0 + (p >> sh)] * K + k);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int p = p0 + u * blockDim.x;
          if (p < pieces) *reinterpret_cast<u32x4*>(xs + (p >> sh) * xrow + 8 * (p & ((1 << sh) - 1))) = v[u];
        }
      }
    };
    for (int round = 0; round < rounds; ++round) {
      const int kb = round * stride + wk * kStep;
      if ((round * stride & (kc - 1)) == 0) {
        if (round) __syncthreads();
        stage(round * stride);
        __syncthreads();
      }
      const uint16_t* xl = xs + min(r, cols - 1) * xrow + (kb & (kc - 1)) + 128 * g;
#pragma unroll
      for (int i = 0; i < RT; ++i) arrange(w[i], kb, K, g);
      // a wave that has its weights goes first, so that those of a CU fall out of
      // step and one's loads meet another's products (64 entries of 7168 x 7168:
      // 33 -> 28 us; 4096 x 7168 of 32 experts, 16 tokens: 120 -> 116; where each SIMD
      // has the waves of one deep block, which wait for each other anyway: -1%)
      if (WN == 2) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int j = 0; j < 16; ++j) {  // word j % 4 of chunk j / 4
        const bf16x8 b = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(xl + 8 * j));
#pragma unroll
        for (int i = 0; i < RT; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              decode8(w[i].c[j >> 2][j & 3], block_scale(j < 8 ? w[i].s.x : w[i].s.y, (j >> 1) & 3), t[i]), b, acc[i], 0, 0, 0);
      }
      if (WN == 2) __builtin_amdgcn_s_setprio(0);
      if (kb + stride < K) {
#pragma unroll
        for (int i = 0; i < RT; ++i) load_tile(rows[i], code, scale, rb, kb + stride, w[i]);
      }
    }
    __syncthreads();  // xs is done with
#pragma unroll
    for (int i = 0; i < RT; ++i)
      *reinterpret_cast<f32x4*>(red + (((wk * WN + wn) * RT + i) * 16 + r) * 16 + 4 * g) = acc[i];
    float* posts = red + WK * WN * RT * 256;  // [WN][RT][16]
    if (wk == 0 && g == 0) {
#pragma unroll
      for (int i = 0; i < RT; ++i) posts[(wn * RT + i) * 16 + r] = post[i];
    }
    __syncthreads();
    for (int o = tid; o < WN * GT * 16 * cols; o += blockDim.x) {  // output column col0 + o % (16 GT WN) of entry m
      const int c = o & 15, v = (o >> 4) % (GT * WN), m = (o >> 4) / (GT * WN);
      const int col = col0 + 16 * v + c, i = v % GT, h = v / GT;
      if (col >= NO) continue;
      float ys[8], us[8];  // up to eight waves' sums, read together
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int at = ((((k < WK ? k : 0) * WN + h) * RT + i) * 16 + m) * 16 + c;
        ys[k] = red[at];
        us[k] = SWIGLU ? red[at + GT * 256] : 0.0f;
      }
      float y = 0.0f, u = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        y += k < WK ? ys[k] : 0.0f;
        u += k < WK ? us[k] : 0.0f;
      }
      y *= posts[(h * RT + i) * 16 + c];
      if (SWIGLU) y = y * __builtin_amdgcn_rcpf(1.0f + __expf(-y)) * (u * posts[(h * RT + i + GT) * 16 + c]);
      out[(size_t)list[c0 + m] * NO + col] = __builtin_bit_cast(uint16_t, (__bf16)y);
    }
    __syncthreads();
  }
}

// Many entries per expert: four waves side by side, RT tiles of 16
// weight rows each over all of K, and up to 16 NT entries whose activations every
// wave reads from LDS.  A step of 512 K values is taken in two halves (words 0-7
// and 8-15 of each lane's codes, that is 64 K values of each lane group), whose
// activations lie in two LDS buffers: while one is used, the next half is on its
// way in registers, and so are the next step's weights, issued after it, so that
// neither wait includes the other.
//
// 128 tokens, top-8 of 32, 4096 x 7168 with SwiGLU: 169 to 183 us from process to
// process, 3.2 to 2.9 TB/s of its 535 MB (849 come past the L2, up to 5.0 TB/s) and
// 355 to 328 TFLOP/s; VALU instructions issue 46% of the time, the matrix unit is
// busy 18%; passes of 16 entries, which read the weights again for every
// 16, take 309.  Alone, the reads take 89 us and the decoding and products 104:
// the two waves of a SIMD, in step with their blocks' barriers, overlap them only
// in part.  Measured without gain: weights two and three steps ahead (they share
// more lines with a neighbour that has left the L2), eight waves a block, half the
// blocks, a grid that fills the GPU once, and FP16 weights and activations, which
// halve the decoding (164 us, for one more launch and a rounding).
template <int RT, int NT, bool SWIGLU, typename IDX>
__global__ __launch_bounds__(256, 2) void k_nvfp4_matvec_wide(const uint16_t* __restrict__ x, int K, int x_div,
                                                              const uint8_t* __restrict__ weight, int E, int N,
                                                              const IDX* __restrict__ ids, int M,
                                                              uint16_t* __restrict__ out,
                                                              int32_t* __restrict__ d_error) {
  constexpr int GT = SWIGLU ? RT / 2 : RT, kRow = 256 + 8, kBuf = 16 * NT * kRow;
  extern __shared__ char smem[];
  uint16_t* xs = reinterpret_cast<uint16_t*>(smem);  // [2][16 NT][264]
  uint16_t* list = xs + 2 * kBuf;
  uint16_t* xrows = list + M;
  __shared__ int wcount[4 * 4];
  __shared__ float posts[4][RT][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int NO = SWIGLU ? N / 2 : N, col0 = (int)blockIdx.x * (64 * GT);
  int e = 0, n = M;
  if (!ids) {
    for (int i = tid; i < M; i += 256) list[i] = xrows[i] = (uint16_t)i;
    __syncthreads();
  } else {
    e = blockIdx.y;
    if (e == 0) clear_unnamed(ids, tid, 256, M, E, col0, col0 + 64 * GT, NO, out, d_error);
    IDX id4[4];
    load_ids(ids, M, 0, id4);
    n = expert_entries(ids, M, e, x_div, id4, list, xrows, wcount);
    if (n == 0) return;
  }

  const uint32_t rb = 9 * ((uint32_t)K / 16) + 4;
  __amdgpu_buffer_rsrc_t rows[RT];
  float t[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row0 = min(col0 + 16 * (wave * GT + i % GT), NO);
    rows[i] = tile_rows(weight, (size_t)e * N + row0 + (SWIGLU && i >= GT ? NO : 0), NO - row0, rb);
    t[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rows[i], (int)((uint32_t)r * rb + (K >> 1) + (K >> 4)), 0, 0));
    posts[wave][i][r] = lift_row(t[i]);
  }
  const uint32_t code = (uint32_t)(r & ~3) * rb + 16u * (4 * g + (r & 3)), scale = (uint32_t)r * rb + (K >> 1) + 8 * g;
  auto load_w = [&](int kb, WTile* w) {
#pragma unroll
    for (int i = 0; i < RT; ++i) load_tile(rows[i], code, scale, rb, kb, w[i]);
  };

  // One pass: NA tiles of 16 entries from c0 on (their number a constant, so that
  // a step is one straight run of instructions the scheduler can interleave).
  auto pass = [&](auto na, int c0, int cols) {
    constexpr int NA = decltype(na)::value;
    f32x4 acc[RT][NA];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int c = 0; c < NA; ++c) acc[i][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // this lane's share of a half: piece tid % 32 of entries tid / 32 + 8 u (past
    // the last: its own again, for columns that are not stored)
    const int kx = 128 * ((tid >> 3) & 3) + 8 * (tid & 7);
    uint32_t xo[2 * NA];  // the entries' rows, in units of 64 values
#pragma unroll
    for (int u = 0; u < 2 * NA; ++u) xo[u] = (uint32_t)xrows[c0 + min((tid >> 5) + 8 * u, cols - 1)] * (uint32_t)(K >> 6);
    u32x4 xv[2 * NA];
    auto load_x = [&](int k0) {
      const bool in = k0 + kx < K;
#pragma unroll
      for (int u = 0; u < 2 * NA; ++u) xv[u] = ld_any<u32x4>(x + ((size_t)xo[u] << 6) + (in ? k0 + kx : 0));
    };
    auto store_x = [&](int buf, int k0) {
      const bool in = k0 + kx < K;
#pragma unroll
      for (int u = 0; u < 2 * NA; ++u) {
        const u32x4 z = {in ? xv[u][0] : 0u, in ? xv[u][1] : 0u, in ? xv[u][2] : 0u, in ? xv[u][3] : 0u};
        *reinterpret_cast<u32x4*>(xs + buf * kBuf + ((tid >> 5) + 8 * u) * kRow + 8 * (tid & 31)) = z;
      }
    };
    auto half = [&](int h, const WTile* w) {
      const uint16_t* xl = xs + h * kBuf + r * kRow + 64 * g;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        bf16x8 b[NA];
#pragma unroll
        for (int c = 0; c < NA; ++c)
          b[c] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(xl + 16 * c * kRow + 8 * j));
#pragma unroll
        for (int i = 0; i < RT; ++i) {
          const bf16x8 a = decode8(w[i].c[2 * h + (j >> 2)][j & 3], block_scale(h == 0 ? w[i].s.x : w[i].s.y, j >> 1), t[i]);
#pragma unroll
          for (int c = 0; c < NA; ++c) acc[i][c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[c], acc[i][c], 0, 0, 0);
        }
      }
    };
    // With three tiles or four the products take longest, and a wave that has its
    // operands goes first (7168 x 2048, 128 tokens, top-8 of 32: 102 -> 97 us; with one
    // or two, which wait for weights most: 144 -> 153 us at 64 tokens of 4096 x 7168).
    auto step = [&](int kb, WTile* w, WTile* next) {
      load_x(kb + 64);
      if (kb + kStep < K) load_w(kb + kStep, next);
#pragma unroll
      for (int i = 0; i < RT; ++i) arrange(w[i], kb, K, g);
      if (NA >= 3) __builtin_amdgcn_s_setprio(1);
      half(0, w);
      if (NA >= 3) __builtin_amdgcn_s_setprio(0);
      store_x(1, kb + 64);
      __syncthreads();
      load_x(kb + kStep);
      if (NA >= 3) __builtin_amdgcn_s_setprio(1);
      half(1, w);
      if (NA >= 3) __builtin_amdgcn_s_setprio(0);
      store_x(0, kb + kStep);
      __syncthreads();
    };
    WTile wa[RT], wb[RT];
    load_x(0);
    load_w(0, wa);
    store_x(0, 0);
    __syncthreads();
    for (int kb = 0; kb < K; kb += 2 * kStep) {
      step(kb, wa, wb);
      if (kb + kStep < K) step(kb + kStep, wb, wa);
    }
    // lane (r, g): rows 4 g .. 4 g + 3 of a tile, entry r of a column tile
#pragma unroll
    for (int c = 0; c < NA; ++c) {
      const int m = 16 * c + r;
      if (m >= cols) continue;
      uint16_t* o = out + (size_t)list[c0 + m] * NO;
#pragma unroll
      for (int i = 0; i < GT; ++i) {
        const int col = col0 + 16 * (wave * GT + i) + 4 * g;
        uint16_t v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y = acc[i][c][q] * posts[wave][i][4 * g + q];
          if (SWIGLU) y = y * __builtin_amdgcn_rcpf(1.0f + __expf(-y)) * (acc[i + GT][c][q] * posts[wave][i + GT][4 * g + q]);
          v[q] = __builtin_bit_cast(uint16_t, (__bf16)y);
        }
        if (col + 4 <= NO) {
          st_any(o + col, make_uint2((uint32_t)v[0] | (uint32_t)v[1] << 16, (uint32_t)v[2] | (uint32_t)v[3] << 16));
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (col + q < NO) o[col + q] = v[q];
        }
      }
    }
  };
  for (int c0 = 0; c0 < n; c0 += 16 * NT) {
    const int cols = min(n - c0, 16 * NT);
    if (cols <= 16) pass(std::integral_constant<int, 1>{}, c0, cols);
    else if (NT < 3 || cols <= 32) pass(std::integral_constant<int, NT < 2 ? NT : 2>{}, c0, cols);
    else if (NT < 4 || cols <= 48) pass(std::integral_constant<int, NT < 3 ? NT : 3>{}, c0, cols);
    else pass(std::integral_constant<int, NT>{}, c0, cols);
  }
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
  if (idx_dtype != EP_IDX_INT32 && idx_dtype != EP_IDX_INT64) return EP_ERR_DTYPE;
  if (tokens >= kSizeLimit || top_k > 1024 || hidden > (1 << 20) || width > (1 << 24) || tokens * top_k > kMaxEntries)
    return EP_ERR_RANGE;
  if (tokens == 0) return EP_OK;  // before topk_idx is looked at: an empty tensor's address may be NULL
  if (!topk_idx && (num_experts != 1 || top_k != 1)) return EP_ERR_SHAPE;
  if (!x || !weight || !out) return EP_ERR_NULL;
  const int M = (int)(tokens * top_k), E = (int)num_experts, N = (int)width, K = (int)hidden;
  const int by_entry = topk_idx && M < E, x_div = x_per_entry ? 1 : (int)top_k;  // entry -> row of x
  hipStream_t s = (hipStream_t)stream;
  const int NO = swiglu ? N / 2 : N;
  constexpr int RT = 2;
  // From 16 entries an expert on (on average), the wide kernel, if its blocks reach
  // every CU: the narrow one reads an expert's weights again for every 16 entries.
  // Wide and narrow, 32 experts, top-8, by the mean of uniform routing: 4096 x 7168
  // with SwiGLU, 16: 152, 185 us; 15: 150, 179; 14: 151, 172; 13: 148, 162; 12: 146,
  // 145; 8: 142, 127; 7168 x 2048, 16: 88, 99; 14: 86, 91; 13: 86, 87; 12: 85, 81;
  // 8: 83, 74.  So the two cross between 12 and 13, and means of 13 to 16 are
  // served up to a fifth slower than they could be.  Skewed ids (exponent 1.2) at 12:
  // 146, 157 and 84, 88.  128 entries of one 7168 x 7168 matrix would be 56 of the
  // wide kernel's blocks and 119 us, against 47.
  const int wide_cols = (swiglu ? 32 : 64) * RT, wide_blocks = (NO + wide_cols - 1) / wide_cols * E;
  if (M >= 16 * E && wide_blocks >= 256) {
    constexpr int NT = 4;
    const dim3 grid((unsigned)(wide_blocks / E), (unsigned)E);
    const size_t lds = (size_t)NT * 16 * 264 * 2 * 2 + 4 * (size_t)M;
#define MTB_WIDE(SW, IDX)                                                                                      \
  hipLaunchKernelGGL((k_nvfp4_matvec_wide<RT, NT, SW, IDX>), grid, dim3(256), lds, s, x, K, x_div, weight, E, N, \
                     (const IDX*)topk_idx, M, out, d_error)
    if (idx_dtype == EP_IDX_INT64) {
      if (swiglu) MTB_WIDE(true, int64_t);
      else MTB_WIDE(false, int64_t);
    } else {
      if (swiglu) MTB_WIDE(true, int32_t);
      else MTB_WIDE(false, int32_t);
    }
#undef MTB_WIDE
    return launch_status();
  }
  const int slots = topk_idx ? (by_entry ? M : E) : 1, mc = min(M, 16);  // mc: entries of one pass
  // Blocks of 2 x 2 waves.  Where those would not reach every CU, an expert's
  // entries are shared out too, 16 a block (up to twice the mean; a block takes the
  // rest in turn).  Where that is not enough either, a block has half the rows,
  // and up to eight waves share out its K steps, as its share of the CU's LDS
  // allows.  7168 x 7168 times 64 entries: 28 us, with half rows 53, by few wide
  // blocks 61; 16 entries: 15 with half rows, 38 by few wide blocks; one
  // token, 2 of 8 experts, 4096 x 4096: 9.8 against 13.2 by whole rows; 8 tokens,
  // top-8 of 32, 7168 x 2048: 70 and 60.
  const int cols2 = (swiglu ? 16 : 32) * RT;
  const int64_t blocks2 = (int64_t)((NO + cols2 - 1) / cols2) * slots;
  const int parts = by_entry || blocks2 >= 256 ? 1 : min((M + 15) / 16, (2 * M + 16 * E - 1) / (16 * E));
  const bool few = blocks2 * parts < 256;
  const int WN = few ? 1 : 2, most = few ? 8 : 2, cols = (swiglu ? 8 : 16) * RT * WN;
  const dim3 grid((unsigned)((NO + cols - 1) / cols), (unsigned)slots, (unsigned)parts);
  // one block a CU, or two (32 entries of 7168 x 7168: 22 us, 28 by one at a time)
  const size_t room = (few && grid.x * grid.y * grid.z <= 256 ? 140 : 70) << 10;
  int WK = 1;
  while (2 * WK <= most && WK * kStep < K && (size_t)mc * (2 * WK * kStep + 8) * 2 <= room) WK *= 2;
  size_t lds_x = max((size_t)mc * (WK * kStep + 8) * 2, (size_t)WK * WN * RT * 1024 + WN * RT * 64);
  lds_x = max(lds_x, min((size_t)mc * (4 * (size_t)K + 16), (size_t)32 << 10));
  lds_x = (lds_x + 15) & ~(size_t)15;
  const dim3 block(64 * WK * WN);
  const size_t lds = lds_x + 4 * (size_t)M;
#define MTB_MATVEC(WN, SW, IDX)                                                                                 \
  hipLaunchKernelGGL((k_nvfp4_matvec<RT, WN, SW, IDX>), grid, block, lds, s, x, K, x_div, weight, E, N,         \
                     (const IDX*)topk_idx, M, by_entry, (int)lds_x, out, d_error)
#define MTB_MATVEC_I(SW, IDX)                 \
  do {                                        \
    if (few) MTB_MATVEC(1, SW, IDX);          \
    else MTB_MATVEC(2, SW, IDX);              \
  } while (0)
  if (idx_dtype == EP_IDX_INT64) {
    if (swiglu) MTB_MATVEC_I(true, int64_t);
    else MTB_MATVEC_I(false, int64_t);
  } else {
    if (swiglu) MTB_MATVEC_I(true, int32_t);
    else MTB_MATVEC_I(false, int32_t);
  }
#undef MTB_MATVEC_I
#undef MTB_MATVEC
  return launch_status();
}
