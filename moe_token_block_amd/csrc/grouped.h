// What the products of grouped rows share: the matrix instruction's types, the
// tile a workgroup takes, and how a wave's results reach memory.
#pragma once

#include "common.h"
#include "quad.h"

namespace mtb {

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

// A stretch of an expert's rows from row0 on, of which the first `used` (at most a
// tile's) hold entries: the rest of its `extent`, which may be more than a tile's,
// gets zeros.
struct Span {
  int expert, row0, used, extent;
};

constexpr int kTailRows = 256;  // rows behind the last expert that one workgroup clears

// Expert e's rows (e == experts: those behind the last expert's) and its tiles of BM.
__device__ __forceinline__ void group_rows(const Groups& gr, int e, int BM, int& lo, int& hi, int& cnt, int& tiles) {
  lo = hi = cnt = tiles = 0;
  if (!gr.counts) {
    if (e == 0) {
      hi = cnt = gr.r_cap;
      tiles = (cnt + BM - 1) / BM;
    }
  } else if (e < gr.experts) {
    lo = min(max(gr.offsets[e], 0), gr.r_cap);
    hi = min(max(gr.offsets[e + 1], lo), gr.r_cap);
    cnt = min(max(gr.counts[e], 0), hi - lo);
    tiles = hi > lo ? max((cnt + BM - 1) / BM, 1) : 0;
  } else if (e == gr.experts) {
    lo = min(max(gr.offsets[e], 0), gr.r_cap);
    hi = gr.r_cap;
    tiles = (hi - lo + kTailRows - 1) / kTailRows;
  }
}

// The id-th of tiles_m x tiles_n tiles in bands of eight rows by all columns.
__device__ __forceinline__ void banded(int id, int tiles_m, int tiles_n, int& m, int& n) {
  constexpr int kBand = 8;
  const int band = id / (kBand * tiles_n), in = id - band * (kBand * tiles_n), rows = min(kBand, tiles_m - band * kBand);
  m = band * kBand + in % rows;
  n = in / rows;
}

// Workgroup `block`'s tile of tiles_m x tiles_n; false: none.  Neighbouring workgroups
// lie on different XCDs: each of the eight takes a run of tiles of its own, so that
// the tiles that run at once on one XCD share their operands in that XCD's L2.
__device__ __forceinline__ bool tile_of(uint32_t block, int tiles_m, int tiles_n, int& m, int& n) {
  const int all = tiles_m * tiles_n, chunk = (all + 7) >> 3;
  const int at = (int)(block >> 3), id = (int)(block & 7) * chunk + at;
  if (at >= chunk || id >= all) return false;
  banded(id, tiles_m, tiles_n, m, n);
  return true;
}

// The workgroup's tile of BM rows by one of tiles_n stretches of columns; false: none.
// All lanes of a wave call it together; the scan over the experts costs about the
// latency of two loads.
template <int BM>
__device__ __forceinline__ bool find_span(const Groups& gr, int tiles_n, Span& s, int& tile_n) {
  const int lane = threadIdx.x & 63;
  int lo, hi, cnt, tiles, upto, total = 0;
  auto take = [&](int base) {  // 64 groups from base on, and the running sum of their tiles
    group_rows(gr, base + lane, BM, lo, hi, cnt, tiles);
    upto = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    return __builtin_amdgcn_readlane(upto, 63);
  };
  for (int base = 0; base <= gr.experts; base += 64) total += take(base);
  int t;
  if (!tile_of(blockIdx.x, total, tiles_n, t, tile_n)) return false;
  // which group the t-th belongs to
  for (int base = 0; base <= gr.experts; base += 64) {
    const int sum = gr.experts < 64 ? total : take(base);  // one stretch of 64: it is there already
    const uint64_t past = __builtin_amdgcn_ballot_w64(upto > t);
    if (past) {
      const int who = __builtin_ctzll(past), n = __builtin_amdgcn_readlane(tiles, who);
      const int i = t - (__builtin_amdgcn_readlane(upto, who) - n);
      const int first = i * (base + who < gr.experts ? BM : kTailRows);
      s.expert = base + who;
      s.row0 = __builtin_amdgcn_readlane(lo, who) + first;
      s.used = min(max(__builtin_amdgcn_readlane(cnt, who) - first, 0), BM);
      const int rest = __builtin_amdgcn_readlane(hi, who) - s.row0;
      s.extent = base + who == gr.experts ? min(rest, kTailRows) : i == n - 1 ? rest : BM;
      return true;
    }
    t -= sum;
  }
  return false;
}

// Upper bound of find_span's workgroups for any plan of so many entries.
inline int64_t span_blocks(int64_t r_cap, int64_t experts, bool dense, int64_t entries, int bm, int64_t tiles_n) {
  const int64_t most = entries < r_cap ? entries : r_cap;
  const int64_t tiles_m = dense ? (r_cap + bm - 1) / bm : most / bm + experts + r_cap / kTailRows + 1;
  return (tiles_m * tiles_n + 7) / 8 * 8;
}

// Whether `blocks` workgroups of `threads` make one grid (2^32 threads an axis do not).
inline bool grid_fits(int64_t blocks, int threads) { return blocks < ((int64_t)1 << 32) / threads; }

// Eight 16-bit values of which the first n exist.
__device__ __forceinline__ u32x4 load8(const uint16_t* p, int n) {
  if (n >= 8) return ld_any<u32x4>(p);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
  return u32x4{w[0], w[1], w[2], w[3]};
}

// The same where p + n is the end of a row (n may be negative): without a branch, from
// the row's last eight values shifted down.  wide: the row has eight.
__device__ __forceinline__ u32x4 load_end(const uint16_t* p, int n, bool wide) {
  // kept apart from a whole load on another path: merged with it, that one would be
  // shifted too, and waited for at once (256 rows of 1024 times 512 x 1024: 10.2 -> 15.2 us)
  asm volatile("" : "+v"(n));
  if (!wide) return load8(p, n);
  const u32x4 v = ld_any<u32x4>(p - (8 - min(n, 8)));
  const int past = 8 - max(min(n, 8), 0);  // values of p's eight that do not exist
  const uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
  const int s = 16 * (past & 3);
  uint64_t a = lo >> s | (s ? hi << (64 - s) : 0), b = hi >> s;
  if (past >= 4) {
    a = b;
    b = 0;
  }
  if (past >= 8) a = 0;
  return u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
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

// The same in FP32, 16 rows at a time through 4096 bytes of LDS: sixteen lanes write a
// row's 256 bytes.
template <int MT>
__device__ __forceinline__ void store_block64(const f32x4 (&acc)[MT][4], char* lds, float* out, int64_t ld, int rows,
                                              int cols) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4*>(lds + r * 256 + 16 * ((4 * i + g) ^ (r & 7))) = acc[j][i];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int row = 4 * p + g, n = cols - 4 * r;
      const f32x4 v = *reinterpret_cast<const f32x4*>(lds + row * 256 + 16 * (r ^ (row & 7)));
      float* o = out + (16 * j + row) * ld + 4 * r;
      if (16 * j + row >= rows) continue;
      if (n >= 4) {
        st_any<f32x4>(o, v);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < n) o[q] = v[q];
      }
    }
  }
}

// The sums of two groups of waves that shared a tile's terms: the second's (share 1)
// through LDS to the first's.  tid: within the group.
template <int MT, int NT>
__device__ __forceinline__ void join_shares(f32x4 (&acc)[MT][NT], char* lds, int tid, int share) {
  f32x4* at = reinterpret_cast<f32x4*>(lds) + tid * MT * NT;
  const int turn = tid & 7;  // a lane's pieces in another order for each of eight: no bank is met twice
  if (share) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) at[(j * NT + i) ^ turn] = acc[j][i];
  }
  __syncthreads();
  if (!share) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[j][i] += at[(j * NT + i) ^ turn];
  }
  __syncthreads();
}

// Rows [first, rows) and columns [0, cols) of a tile: zeros.
__device__ __forceinline__ void clear_rows(uint16_t* out, int64_t ld, int first, int rows, int cols) {
  const int pieces = (cols + 7) >> 3;
  for (int i = threadIdx.x; i < (rows - first) * pieces; i += blockDim.x)
    store8(out + (int64_t)(first + i / pieces) * ld + 8 * (i % pieces), u32x4{0u, 0u, 0u, 0u}, cols - 8 * (i % pieces));
}

// The kernels for few rows: blockIdx.y is an expert, whose rows gridDim.z workgroups
// share, or, past the last, gridDim.z stretches of the rows behind it.
inline int64_t few_groups(int64_t r_cap, int64_t experts, bool dense, int64_t z) {
  return dense ? 1 : experts + (r_cap / kTailRows + z) / z;
}
// Its rows [lo, hi), the first cnt of which hold entries, and the first row that this
// workgroup clears; false: none.
__device__ __forceinline__ bool few_rows(const Groups& gr, int& lo, int& hi, int& cnt, int& clear) {
  const int e = blockIdx.y;
  int tiles;
  group_rows(gr, min(e, gr.experts), 16, lo, hi, cnt, tiles);
  clear = blockIdx.z ? hi - lo : cnt;
  if (gr.counts && e >= gr.experts) {
    lo += ((e - gr.experts) * (int)gridDim.z + (int)blockIdx.z) * kTailRows;
    hi = min(hi, lo + kTailRows);
    clear = 0;
  }
  return hi > lo;
}

// The waves' sums of 16 RT columns by 16 NT rows, added in the waves' order and stored
// as BF16; lane (r, g) holds columns 16 i + 4 g .. + 3 of row 16 t + r in acc[t][i].
// red: 1024 RT NT bytes a wave.
template <int RT, int NT>
__device__ __forceinline__ void join_few(const f32x4 (&acc)[NT][RT], float* red, uint16_t* out, int64_t ld, int used,
                                         int cols) {
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6, W = blockDim.x >> 6;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < RT; ++i)
      *reinterpret_cast<f32x4*>(red + (((wave * NT + t) * RT + i) * 16 + r) * 16 + 4 * g) = acc[t][i];
  __syncthreads();
  for (int o = threadIdx.x; o < used * 16 * RT; o += blockDim.x) {
    const int n = o % (16 * RT), m = o / (16 * RT);
    const float* at = red + (((m >> 4) * RT + (n >> 4)) * 16 + (m & 15)) * 16 + (n & 15);
    float y = 0.0f;
    for (int v = 0; v < W; ++v) y += at[v * NT * RT * 256];
    if (n < cols) out[m * ld + n] = __builtin_bit_cast(uint16_t, (__bf16)y);
  }
  __syncthreads();
}

}  // namespace mtb
