// BF16 token rows to their experts and back (P2, review comments: one routing
// serves the dispatch and the combine): the copy into grouped rows, the
// weighted sum of a token's expert rows, and the gradients of both.
#include "common.h"
#include "launch.h"

namespace mtb {

// Rows are cut into pieces of 8 values, one 16-byte access per lane; an odd
// width only moves the addresses (any 2-byte boundary will do).  The last piece
// of a width that is no multiple of 8 starts at hidden - 8: its first values are
// those of the piece before it, computed twice and stored twice alike.
constexpr int kPiece = 8;
constexpr int kWaveCols = 64 * kPiece;    // columns of one access of a wave
constexpr int kBlockCols = 4 * kWaveCols;  // and of a block of four waves

typedef u32x4 u32x4_row __attribute__((aligned(2)));

// STREAM: a read past the caches, for rows that are read once and exceed the
// 256 MB MALL (combine at 16384 x 7168, top-8: 370 -> 357 us).  Rows that fit it
// were often just written by the product before and are found there (4096 x
// 4096, top-2: 16.0 us against 18.2 streamed).
template <bool STREAM>
__device__ __forceinline__ u32x4 ld8(const uint16_t* p) {
  if (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_row*>(p));
  return *reinterpret_cast<const u32x4_row*>(p);
}

// Results are streamed out: whole lines that no kernel here reads again (398 ->
// 370 us at the same combine, 375 -> 340 us at its dispatch).
__device__ __forceinline__ void st8(uint16_t* p, u32x4 v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4_row*>(p));
}

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f32_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Grouped rows that belong to no token, kPadRows of them per block, are cleared
// by the first blocks of the dispatch and of the combine's gradient; one ballot
// finds them.
constexpr int kPadRows = 8;

__device__ __forceinline__ void clear_padding(int g0, const int32_t* __restrict__ src_row, int T, int r_cap, int H,
                                              uint16_t* __restrict__ out) {
  const int lane = threadIdx.x & 63, n = min(kPadRows, r_cap - g0);
  const int s = lane < n ? src_row[g0 + lane] : 0;
  uint64_t pad = __builtin_amdgcn_ballot_w64(lane < n && (s < 0 || s >= T));
  while (pad) {
    uint16_t* o = out + (size_t)(g0 + __builtin_ctzll(pad)) * H;
    pad &= pad - 1;
    const int nch = H / kPiece;
    for (int c = threadIdx.x; c < nch; c += 256) st8(o + kPiece * c, u32x4{0u, 0u, 0u, 0u});
    const int i = kPiece * nch + (int)threadIdx.x;
    if (i < H) o[i] = 0;
  }
}

// The wave of a token and 512 of its columns: t, and this lane's piece c (false
// for lanes past the row).
__device__ __forceinline__ bool wave_piece(int wave, int segs, int H, int& t, int& c) {
  t = wave / segs;
  const int c0 = (wave - t * segs) * kWaveCols + (int)(threadIdx.x & 63) * kPiece;
  c = min(c0, H - kPiece);
  return c0 < H;
}

// out[dst_row[t, j]] = x[t] for every used slot: a wave per token and 512
// columns, whose slots are scalars.  A token's row is read once and written
// top_k times; the other way round, a wave per grouped row that reads its token,
// rows are read top_k times at scattered times (16384 x 7168, top-8: 575 us
// against 373; 4096 x 4096, top-2: 20.8 against 15.0).  A block per token, which
// lasts longer than a wave, gave 405 us and, at 32768 x 4096, top-2, 144 us
// against 109.
__global__ __launch_bounds__(256) void k_bf16_dispatch(const uint16_t* __restrict__ x, int T, int H, int k, int r_cap,
                                                       int pad_blocks, int segs, int waves,
                                                       const int32_t* __restrict__ dst_row,
                                                       const int32_t* __restrict__ src_row,
                                                       uint16_t* __restrict__ out) {
  if ((int)blockIdx.x < pad_blocks) {
    clear_padding((int)blockIdx.x * kPadRows, src_row, T, r_cap, H, out);
    return;
  }
  const int wv = __builtin_amdgcn_readfirstlane(((int)blockIdx.x - pad_blocks) * 4 + (int)(threadIdx.x >> 6));
  int t, c;
  if (wv >= waves || !wave_piece(wv, segs, H, t, c)) return;
  const u32x4 v = ld8<false>(x + (size_t)t * H + c);
  for (int j = 0; j < k; ++j) {
    const int g = dst_row[(size_t)t * k + j];
    if ((uint32_t)g < (uint32_t)r_cap) st8(out + (size_t)g * H + c, v);
  }
}

// The grouped row of a slot; none (-1) where the routing's id of the slot names no
// expert (IDX void: no ids, the map alone says which slots are used).
template <typename IDX>
__device__ __forceinline__ int slot_row(const int32_t* __restrict__ dst_row, const IDX* __restrict__ ids, int E,
                                        size_t slot) {
  const int g = dst_row[slot];
  if constexpr (std::is_void_v<IDX>) {
    return g;
  } else {
    const IDX id = ids[slot];
    return id >= 0 && id < E ? g : -1;
  }
}

// out[t] = sum over slots j, in order, of w[t, j] * rows[dst_row[t, j]], in
// FP32, rounded once.  One wave per token and 512 columns; the token is the
// same in every lane, so its slots are scalars, and the loads of KU slots go
// out before the first is used (one slot at a time, with a wave per block and
// 2-byte loads, took 1072 us at 16384 x 7168, top-8).  Bound by memory: 2115 MB
// in 357 us are 5.9 TB/s; a copy of 1 GiB by the same 16-byte streamed accesses
// reaches 6.5, a read alone 7.1.
template <int KU, bool STREAM, typename IDX>
__global__ __launch_bounds__(256) void k_bf16_combine(const uint16_t* __restrict__ rows, int r_cap, int H, int k,
                                                      int segs, int waves, const int32_t* __restrict__ dst_row,
                                                      const IDX* __restrict__ ids, int E,
                                                      const float* __restrict__ weights, uint16_t* __restrict__ out) {
  const int wv = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4u + (threadIdx.x >> 6)));
  int t, c;
  if (wv >= waves || !wave_piece(wv, segs, H, t, c)) return;
  const size_t slot0 = (size_t)t * k;
  float acc[8] = {};
  for (int j0 = 0; j0 < k; j0 += KU) {
    u32x4 v[KU];
    bool used[KU];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const int g = j0 + u < k ? slot_row(dst_row, ids, E, slot0 + j0 + u) : -1;
      used[u] = (uint32_t)g < (uint32_t)r_cap;
      if (used[u]) v[u] = ld8<STREAM>(rows + (size_t)g * H + c);
    }
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      if (!used[u]) continue;
      const float w = weights ? weights[slot0 + j0 + u] : 1.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] = __builtin_fmaf(w, bf16lo(v[u][i]), acc[2 * i]);
        acc[2 * i + 1] = __builtin_fmaf(w, bf16hi(v[u][i]), acc[2 * i + 1]);
      }
    }
  }
  st8(out + (size_t)t * H + c, u32x4{bf16pair(acc[0], acc[1]), bf16pair(acc[2], acc[3]), bf16pair(acc[4], acc[5]),
                                     bf16pair(acc[6], acc[7])});
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
  return v;
}

// Gradients of the combine: drows[dst] = w * dout, dw = <dout, rows[dst]>.  A
// block per token (a wave per token: 314 against 253 us at 32768 x 4096, top-2;
// its slots then follow one another).  A lane keeps NP pieces of dout for all
// the token's slots, so dout is read once; the loads of KU slots go out
// together.  Each lane sums its own products, then the lanes and the four waves
// in a fixed order.  Bound by memory: 1345 MB in 244 us, 5.5 TB/s.
template <int NP, int KU, bool STREAM>
__global__ __launch_bounds__(256) void k_bf16_combine_bwd(const uint16_t* __restrict__ dout,
                                                          const uint16_t* __restrict__ rows, int T, int H, int k,
                                                          int r_cap, int pad_blocks,
                                                          const int32_t* __restrict__ dst_row,
                                                          const int32_t* __restrict__ src_row,
                                                          const float* __restrict__ weights,
                                                          uint16_t* __restrict__ drows, float* __restrict__ dweights) {
  if ((int)blockIdx.x < pad_blocks) {
    clear_padding((int)blockIdx.x * kPadRows, src_row, T, r_cap, H, drows);
    return;
  }
  __shared__ float part[4][KU];
  const int t = (int)blockIdx.x - pad_blocks;
  const size_t slot0 = (size_t)t * k;
  for (int j0 = 0; j0 < k; j0 += KU) {
    float dot[KU] = {};
    for (int cb = (int)threadIdx.x * kPiece; cb < H; cb += NP * kBlockCols) {
      u32x4 q[NP], v[KU][NP];
      bool used[KU];
      int c[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        c[p] = min(cb + p * kBlockCols, H - kPiece);  // past the row: its last piece, read and not used
        q[p] = ld8<STREAM>(dout + (size_t)t * H + c[p]);
      }
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        const int g = j0 + u < k ? dst_row[slot0 + j0 + u] : -1;
        used[u] = (uint32_t)g < (uint32_t)r_cap;
        if (!used[u]) continue;
#pragma unroll
        for (int p = 0; p < NP; ++p) v[u][p] = ld8<STREAM>(rows + (size_t)g * H + c[p]);
      }
#pragma unroll
      for (int u = 0; u < KU; ++u) {
        if (!used[u]) continue;
        const float w = weights[slot0 + j0 + u];
        uint16_t* o = drows + (size_t)dst_row[slot0 + j0 + u] * H;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int skip = cb + p * kBlockCols - c[p];  // values of the last piece that the one before it holds
          if (skip >= kPiece) continue;
          u32x4 r;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = bf16lo(q[p][i]), b = bf16hi(q[p][i]);
            const float fa = __builtin_fmaf(a, bf16lo(v[u][p][i]), dot[u]);
            dot[u] = 2 * i >= skip ? fa : dot[u];
            const float fb = __builtin_fmaf(b, bf16hi(v[u][p][i]), dot[u]);
            dot[u] = 2 * i + 1 >= skip ? fb : dot[u];
            r[i] = bf16pair(w * a, w * b);
          }
          st8(o + c[p], r);
        }
      }
    }
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      const float s = wave_sum(dot[u]);
      if (lane == u) part[wave][u] = s;
    }
    __syncthreads();
    if ((int)threadIdx.x < KU && j0 + (int)threadIdx.x < k)
      dweights[slot0 + j0 + threadIdx.x] =
          (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
    __syncthreads();
  }
}

// Widths below one piece: a lane per token, value by value.
enum Narrow { kNarrowDispatch, kNarrowCombine, kNarrowCombineBwd };
template <Narrow OP, typename IDX>
__global__ __launch_bounds__(256) void k_bf16_narrow(const uint16_t* __restrict__ x, const uint16_t* __restrict__ rows,
                                                     int T, int H, int k, int r_cap, int pad_blocks,
                                                     const int32_t* __restrict__ dst_row,
                                                     const int32_t* __restrict__ src_row,
                                                     const IDX* __restrict__ ids, int E,
                                                     const float* __restrict__ weights, uint16_t* __restrict__ out,
                                                     float* __restrict__ dweights) {
  if ((int)blockIdx.x < pad_blocks) {
    clear_padding((int)blockIdx.x * kPadRows, src_row, T, r_cap, H, out);
    return;
  }
  const int t = ((int)blockIdx.x - pad_blocks) * 256 + (int)threadIdx.x;
  if (t >= T) return;
  const uint16_t* xt = x + (size_t)t * H;
  float acc[kPiece] = {};
  for (int j = 0; j < k; ++j) {
    const size_t slot = (size_t)t * k + j;
    const int g = slot_row(dst_row, ids, E, slot);
    const bool used = (uint32_t)g < (uint32_t)r_cap;
    const size_t at = (size_t)(used ? g : 0) * H;
    const float w = OP != kNarrowDispatch && weights && used ? weights[slot] : 1.0f;
    float dot = 0.0f;
    for (int c = 0; c < H && used; ++c) {
      if (OP == kNarrowDispatch) out[at + c] = xt[c];
      if (OP == kNarrowCombine) acc[c] = __builtin_fmaf(w, bf16_f32(rows[at + c]), acc[c]);
      if (OP == kNarrowCombineBwd) {
        dot = __builtin_fmaf(bf16_f32(xt[c]), bf16_f32(rows[at + c]), dot);
        out[at + c] = f32_bf16(w * bf16_f32(xt[c]));
      }
    }
    if (OP == kNarrowCombineBwd) dweights[slot] = dot;
  }
  if (OP == kNarrowCombine)
    for (int c = 0; c < H; ++c) out[(size_t)t * H + c] = f32_bf16(acc[c]);
}

}  // namespace mtb

using namespace mtb;

namespace {
// Sizes every call here checks first.  hidden from 1 to 2^20; a grid of one
// lane per piece of every token, and one of a block per token and per kPadRows
// grouped rows, both below 2^32 lanes.
int32_t check_sizes(int64_t tokens, int64_t hidden, int64_t top_k, int64_t r_cap) {
  if (tokens < 0 || hidden <= 0 || top_k < 1 || r_cap < 0) return EP_ERR_SHAPE;
  if (tokens >= (1 << 23) || r_cap >= (1 << 25) || hidden > (1 << 20) || top_k > 1024 || tokens * top_k > INT32_MAX / 4)
    return EP_ERR_RANGE;
  if (tokens * ((hidden + kWaveCols - 1) / kWaveCols) >= (1 << 25)) return EP_ERR_RANGE;
  return EP_OK;
}

// Reads of more than the MALL holds are streamed.
bool streamed(int64_t entries, int64_t hidden) { return entries * hidden * 2 > ((int64_t)256 << 20); }

struct Combine {
  const uint16_t* rows;
  const int32_t* dst_row;
  const float* weights;
  uint16_t* out;
  int R, H, T, k;
  hipStream_t s;
};

template <bool STREAM, typename IDX>
int32_t launch_combine(const Combine& c, const IDX* ids, int E) {
  if (c.H < kPiece) {
    hipLaunchKernelGGL((k_bf16_narrow<kNarrowCombine, IDX>), dim3((unsigned)((c.T + 255) / 256)), dim3(256), 0, c.s,
                       nullptr, c.rows, c.T, c.H, c.k, c.R, 0, c.dst_row, nullptr, ids, E, c.weights, c.out, nullptr);
    return launch_status();
  }
  const int segs = (c.H + kWaveCols - 1) / kWaveCols, waves = c.T * segs;
  const dim3 grid((unsigned)((waves + 3) / 4)), block(256);
  if (c.k <= 2)
    hipLaunchKernelGGL((k_bf16_combine<2, STREAM, IDX>), grid, block, 0, c.s, c.rows, c.R, c.H, c.k, segs, waves,
                       c.dst_row, ids, E, c.weights, c.out);
  else
    hipLaunchKernelGGL((k_bf16_combine<8, STREAM, IDX>), grid, block, 0, c.s, c.rows, c.R, c.H, c.k, segs, waves,
                       c.dst_row, ids, E, c.weights, c.out);
  return launch_status();
}
}  // namespace

MTB_EXPORT int32_t ep_bf16_dispatch(const uint16_t* x, int64_t tokens, int64_t hidden, int64_t top_k, int64_t r_cap,
                                    const int32_t* dst_row, const int32_t* src_row, uint16_t* out, void* stream) {
  const int32_t st = check_sizes(tokens, hidden, top_k, r_cap);
  if (st != EP_OK) return st;
  if (r_cap == 0) return EP_OK;
  if (!src_row || !out || (tokens > 0 && (!x || !dst_row))) return EP_ERR_NULL;
  hipStream_t s = (hipStream_t)stream;
  const int T = (int)tokens, H = (int)hidden, R = (int)r_cap;
  const int pad_blocks = (R + kPadRows - 1) / kPadRows;
  if (H < kPiece) {
    hipLaunchKernelGGL((k_bf16_narrow<kNarrowDispatch, void>), dim3((unsigned)(pad_blocks + (T + 255) / 256)),
                       dim3(256), 0, s, x, nullptr, T, H, (int)top_k, R, pad_blocks, dst_row, src_row, nullptr, 0,
                       nullptr, out, nullptr);
    return launch_status();
  }
  const int segs = (H + kWaveCols - 1) / kWaveCols, waves = T * segs;
  hipLaunchKernelGGL(k_bf16_dispatch, dim3((unsigned)(pad_blocks + (waves + 3) / 4)), dim3(256), 0, s, x, T, H,
                     (int)top_k, R, pad_blocks, segs, waves, dst_row, src_row, out);
  return launch_status();
}

MTB_EXPORT int32_t ep_bf16_combine(const uint16_t* rows, int64_t r_cap, int64_t hidden, int64_t tokens,
                                   int64_t top_k, const int32_t* dst_row, const float* weights, uint16_t* out,
                                   void* stream) {
  const int32_t st = check_sizes(tokens, hidden, top_k, r_cap);
  if (st != EP_OK) return st;
  if (tokens == 0) return EP_OK;
  if (!dst_row || !out || (r_cap > 0 && !rows)) return EP_ERR_NULL;
  const Combine c{rows, dst_row, weights, out, (int)r_cap, (int)hidden, (int)tokens, (int)top_k, (hipStream_t)stream};
  return streamed(tokens * top_k, hidden) ? launch_combine<true, void>(c, nullptr, 0)
                                          : launch_combine<false, void>(c, nullptr, 0);
}

MTB_EXPORT int32_t ep_bf16_combine_topk(const uint16_t* rows, int64_t r_cap, int64_t hidden, int64_t tokens,
                                        int64_t top_k, const int32_t* dst_row, const void* topk_idx,
                                        int32_t idx_dtype, int64_t num_experts, const float* weights, uint16_t* out,
                                        void* stream) {
  const int32_t st = check_sizes(tokens, hidden, top_k, r_cap);
  if (st != EP_OK) return st;
  if (num_experts < 1 || num_experts > 1024) return EP_ERR_SHAPE;
  if (idx_dtype != EP_IDX_INT32 && idx_dtype != EP_IDX_INT64) return EP_ERR_DTYPE;
  if (tokens == 0) return EP_OK;
  if (!dst_row || !topk_idx || !out || (r_cap > 0 && !rows)) return EP_ERR_NULL;
  const Combine c{rows, dst_row, weights, out, (int)r_cap, (int)hidden, (int)tokens, (int)top_k, (hipStream_t)stream};
  // not streamed: its rows are a few tokens' expert products, which the caches still hold
  return idx_dtype == EP_IDX_INT64 ? launch_combine<false>(c, (const int64_t*)topk_idx, (int)num_experts)
                                   : launch_combine<false>(c, (const int32_t*)topk_idx, (int)num_experts);
}

MTB_EXPORT int32_t ep_bf16_combine_bwd(const uint16_t* dout, const uint16_t* rows, int64_t tokens, int64_t hidden,
                                       int64_t top_k, int64_t r_cap, const int32_t* dst_row, const int32_t* src_row,
                                       const float* weights, uint16_t* drows, float* dweights, void* stream) {
  const int32_t st = check_sizes(tokens, hidden, top_k, r_cap);
  if (st != EP_OK) return st;
  if (tokens == 0 && r_cap == 0) return EP_OK;
  if (r_cap > 0 && (!rows || !drows || !src_row)) return EP_ERR_NULL;
  if (tokens > 0 && (!dout || !dst_row || !weights || !dweights)) return EP_ERR_NULL;
  hipStream_t s = (hipStream_t)stream;
  const int T = (int)tokens, H = (int)hidden, k = (int)top_k, R = (int)r_cap;
  const int pad_blocks = (R + kPadRows - 1) / kPadRows;
  if (H < kPiece) {
    hipLaunchKernelGGL((k_bf16_narrow<kNarrowCombineBwd, void>), dim3((unsigned)(pad_blocks + (T + 255) / 256)),
                       dim3(256), 0, s, dout, rows, T, H, k, R, pad_blocks, dst_row, src_row, nullptr, 0, weights,
                       drows, dweights);
    return launch_status();
  }
#define MTB_BWD(NP, KU, ST)                                                                                          \
  hipLaunchKernelGGL((k_bf16_combine_bwd<NP, KU, ST>), dim3((unsigned)(pad_blocks + T)), dim3(256), 0, s, dout, rows, \
                     T, H, k, R, pad_blocks, dst_row, src_row, weights, drows, dweights)
  if (streamed(tokens * top_k, hidden)) {
    if (k <= 2) MTB_BWD(2, 2, true);
    else MTB_BWD(1, 8, true);
  } else {
    if (k <= 2) MTB_BWD(2, 2, false);
    else MTB_BWD(1, 8, false);
  }
#undef MTB_BWD
  return launch_status();
}
