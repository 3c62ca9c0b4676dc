// What the products of grouped rows share: the matrix instruction's types, the
// tile a workgroup takes, and how a wave's results reach memory.
#pragma once

#include "common.h"

namespace mtb {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// The grouped rows as a routing plan has them: expert e's are [offsets[e],
// offsets[e + 1]), of which the first counts[e] hold entries.  counts NULL: one
// matrix, every row of it an entry.  Whatever the arrays hold, the spans taken
// from them lie within [0, r_cap).
struct Groups {
  const int32_t* counts;
  const int32_t* offsets;
  int experts, r_cap;
};

// A stretch of at most `rows` grouped rows from row0 on, all of one expert: the
// first `used` of its `extent` rows hold entries, the others get zeros.
struct Span {
  int expert, row0, used, extent;
};

// The t-th of the tiles of BM rows that cover every expert's rows and then those
// behind the last expert's; `total` of them.  All lanes of a wave call it
// together; the scan over the experts costs about the latency of two loads.
template <int BM>
__device__ __forceinline__ bool find_span(const Groups& gr, int tiles_n, Span& s, int& tile_n, int GM) {
  const int lane = threadIdx.x & 63;
  const int nb = gr.counts ? gr.experts + 1 : 1;
  int total = 0;
  // how many tiles there are
  for (int base = 0; base < nb; base += 64) {
    const int e = base + lane;
    int tiles = 0;
    if (e < nb) {
      const int lo = gr.counts ? min(max(gr.offsets[e], 0), gr.r_cap) : 0;
      const int hi = gr.counts && e < gr.experts ? min(max(gr.offsets[e + 1], lo), gr.r_cap) : gr.r_cap;
      tiles = (hi - lo + BM - 1) / BM;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) tiles += __shfl_xor(tiles, o, 64);
    total += tiles;
  }
  total = __builtin_amdgcn_readfirstlane(total);
  // Neighbouring workgroups lie on different XCDs: each of the eight takes a run of
  // tiles of its own, GM rows of tiles by all columns at a time, so that what runs
  // at once on one XCD shares its operands in that XCD's L2.
  const int all = total * tiles_n, chunk = (all + 7) >> 3;
  const int at = (int)(blockIdx.x >> 3), id = (int)(blockIdx.x & 7) * chunk + at;
  if (at >= chunk || id >= all) return false;
  const int band = id / (GM * tiles_n), in = id - band * (GM * tiles_n), gm = min(GM, total - band * GM);
  int t = band * GM + in % gm;
  tile_n = in / gm;
  // which expert the t-th belongs to
  for (int base = 0;; base += 64) {
    const int e = base + lane;
    int tiles = 0, lo = 0, hi = 0, cnt = 0;
    if (e < nb) {
      lo = gr.counts ? min(max(gr.offsets[e], 0), gr.r_cap) : 0;
      hi = gr.counts && e < gr.experts ? min(max(gr.offsets[e + 1], lo), gr.r_cap) : gr.r_cap;
      cnt = gr.counts ? (e < gr.experts ? min(max(gr.counts[e], 0), hi - lo) : 0) : hi;
      tiles = (hi - lo + BM - 1) / BM;
    }
    int upto = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    const uint64_t past = __builtin_amdgcn_ballot_w64(upto > t);
    if (past) {
      const int who = __builtin_ctzll(past);
      const int first = (t - (__builtin_amdgcn_readlane(upto, who) - __builtin_amdgcn_readlane(tiles, who))) * BM;
      s.expert = base + who;
      s.row0 = __builtin_amdgcn_readlane(lo, who) + first;
      s.extent = min(__builtin_amdgcn_readlane(hi, who) - s.row0, BM);
      s.used = min(max(__builtin_amdgcn_readlane(cnt, who) - first, 0), s.extent);
      return true;
    }
    t -= __builtin_amdgcn_readlane(upto, 63);
  }
}

// Upper bound of find_span's workgroups for any plan (0 where it passes 2^31).
inline int64_t span_blocks(int64_t r_cap, int64_t experts, bool dense, int bm, int64_t tiles_n) {
  const int64_t tiles_m = dense ? (r_cap + bm - 1) / bm : r_cap / bm + experts + 1;
  return (tiles_m * tiles_n + 7) / 8 * 8;
}

// Eight 16-bit values of which the first n exist.
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n) {
  if (n >= 8) return ld_any<u32x4>(p);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return u32x4{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ void store8(uint16_t* p, u32x4 v, int n) {
  if (n >= 8) {
    st_any<u32x4>(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
}

// A wave's 16 MT x 64 block of results to memory as BF16.  Lane (r, g) holds
// columns 16 i + 4 g .. + 3 of row 16 j + r in acc[j][i]; through `lds` (MT * 2048
// bytes of this wave's own) eight neighbouring lanes get a row's 128 bytes, so that
// whole lines are written.  `rows`: rows of the block that exist, of which the
// first `used` are results and the others zeros; cols: columns that exist.
template <int MT>
__device__ __forceinline__ void store_block64(const f32x4 (&acc)[MT][4], char* lds, uint16_t* out, int64_t ld, int used,
                                              int rows, int cols) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < MT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint2 v = make_uint2(bf16pair(acc[j][i][0], acc[j][i][1]), bf16pair(acc[j][i][2], acc[j][i][3]));
      const int chunk = (2 * i + (g >> 1)) ^ (r & 7);
      *reinterpret_cast<uint2*>(lds + (16 * j + r) * 128 + 16 * chunk + 8 * (g & 1)) = v;
    }
  const int c = lane & 7;
#pragma unroll
  for (int p = 0; p < 2 * MT; ++p) {
    const int row = 8 * p + (lane >> 3);
    u32x4 v = *reinterpret_cast<const u32x4*>(lds + row * 128 + 16 * (c ^ (row & 7)));
    if (row >= used) v = u32x4{0u, 0u, 0u, 0u};
    if (row < rows && 8 * c < cols) store8(out + row * ld + 8 * c, v, cols - 8 * c);
  }
}

}  // namespace mtb
