// Which expert's group an output tile of the expert-grouped GEMMs belongs to:
// shared by the small-tile kernel (bsq_gemm_grouped.hip) and the grouped forms of
// the 256 x 256 kernels.
#pragma once

#include "bsq_gemm_common.hpp"
#include "bsq_internal.hpp"

namespace bsq {

namespace {

enum { kGroupNone = 0, kGroupRows = 1, kGroupWgrad = 2 };

struct GroupRef {
  const int32_t* offsets;   // [experts + 1]
  int experts;
  int ba_n;                 // per-tensor scales of B: 1 or experts
};

// A tile's group: rows [row0, row1) from the tile's first row to the group's end.
struct GroupTile {
  int e;                    // -1: the rows of no group
  int64_t row0, row1;
};

// Group bounds as stored, kept inside [0, rows] and ordered, so that no offset
// reaches outside the operands.
__device__ __forceinline__ void group_bounds(const int32_t* off, int e, int64_t rows, int64_t& b, int64_t& n) {
  b = off[e];
  n = off[e + 1];
  b = b < 0 ? 0 : b > rows ? rows : b;
  n = n < b ? b : n > rows ? rows : n;
}

// Inclusive prefix sum over the 64 lanes: within rows of 16 by shifts, then the
// rows' totals carried on (DPP: no LDS round trips on the way to the first load).
__device__ __forceinline__ int lanes_prefix(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row 0 -> 1, 2 -> 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row 1 -> 2, 3
  return v;
}

// Tile `pid` of the row-grouped product: row tiles of MT rows, groups in order,
// each starting a new tile, then the rows of no group (e = -1: past the last, before
// the first), in the XCD-aware order of tile_of_block over all of them.  Returns false past the
// last tile (the grid covers the most there can be).  Every wave computes it
// for itself, 64 experts at a time.
template <int MT>
__device__ __forceinline__ bool group_tile_rows(const GroupRef& g, int64_t rows, int pid, int tiles_n,
                                                GroupTile& t, int& tn) {
  const int lane = threadIdx.x & 63;
  int64_t b = 0, n = 0;
  int inc = 0, mine = 0, total = 0, e0 = 0;
  const auto block = [&](int first) {
    const int e = first + lane;
    b = n = 0;
    if (e < g.experts) group_bounds(g.offsets, e, rows, b, n);
    mine = (int)((n - b + MT - 1) / MT);
    inc = lanes_prefix(mine);
  };
  for (e0 = 0; e0 < g.experts; e0 += 64) {
    block(e0);
    total += __builtin_amdgcn_readlane(inc, 63);
  }
  int64_t last = g.offsets[g.experts];
  last = last < 0 ? 0 : last > rows ? rows : last;
  int64_t first = g.offsets[0];
  first = first < 0 ? 0 : first > rows ? rows : first;
  const int past = (int)((rows - last + MT - 1) / MT);
  const int all = total + past + (int)((first + MT - 1) / MT);
  if ((int64_t)pid >= (int64_t)all * tiles_n) return false;
  int tm;
  tile_of_block(pid, all, tiles_n, tm, tn);
  if (tm >= total) {
    const bool before = tm - total >= past;
    const int64_t from = before ? 0 : last;
    t.e = -1;
    t.row0 = from + (int64_t)(tm - total - (before ? past : 0)) * MT;
    t.row1 = before ? first : rows;
    return t.row0 >= from && t.row0 < t.row1;
  }
  int before = 0;
  for (e0 = 0; e0 < g.experts; e0 += 64) {
    if (g.experts > 64) block(e0);                 // else: still held from above
    const uint64_t hit = __ballot(before + inc > tm);
    if (hit) {
      const int w = __builtin_ctzll(hit);
      const int64_t gb = __builtin_amdgcn_readlane((int)b, w);
      t.e = e0 + w;
      t.row0 = gb + (int64_t)(tm - before - __builtin_amdgcn_readlane(inc - mine, w)) * MT;
      t.row1 = __builtin_amdgcn_readlane((int)n, w);
      // always so for ascending offsets (others could overflow the counts)
      return t.row0 >= gb && t.row0 < t.row1;
    }
    before += __builtin_amdgcn_readlane(inc, 63);
  }
  return false;
}

// Tile of workgroup `pid` of the reduction-grouped product, expert by expert;
// returns the expert.  Every XCD takes an eighth of each expert's tiles: with
// whole experts per XCD the longest group's XCD finished last (8 experts of
// 16,384 rows, 14336 x 4096: 2.65 ms against 1.52 ms).
__device__ __forceinline__ int wgrad_tile(int pid, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int e = pid / (tiles_m * tiles_n);
  tile_of_block(pid - e * tiles_m * tiles_n, tiles_m, tiles_n, tm, tn);
  return e;
}

// Reduction range of group e in whole blocks of BLK rows, from the multiple of
// UNIT at or below its first row (t.row0): rows lo <= k < hi of it count; hi = 0
// for an empty group.
template <int BLK, int UNIT>
__device__ __forceinline__ void group_range(const GroupRef& g, int e, int64_t rows, int& lo, int& hi, GroupTile& t) {
  int64_t b, n;
  group_bounds(g.offsets, e, rows, b, n);
  b = b / BLK * BLK;
  n = n / BLK * BLK;
  t.e = e;
  t.row0 = b / UNIT * UNIT;
  t.row1 = n;
  lo = (int)(b - t.row0);
  hi = n > b ? (int)(n - t.row0) : 0;
}

// Most row tiles of MT rows there can be: every group with rows (the rows of no
// group count as two) has at most one partly filled tile.
inline int64_t max_row_tiles(int64_t rows, int experts, int MT) {
  const int64_t g = rows < experts + 2 ? rows : experts + 2;
  return (rows - g) / MT + g;
}

// Zeros in the 256 x 256 tile at (m0, n0) of c [M, N] (256 threads): the rows of
// no group, and the product of an empty group.
__device__ __forceinline__ void zero_tile(uint16_t* c, int64_t ldc, int64_t M, int64_t N, int64_t m0, int64_t n0,
                                          int vec_store) {
  for (int i = threadIdx.x; i < 256 * 32; i += 256) {
    const int64_t m = m0 + (i >> 5), n = n0 + (i & 31) * 8;
    if (m >= M) return;
    uint16_t* dst = c + m * ldc + n;
    if (vec_store && n + 7 < N) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
    } else {
      for (int e = 0; e < 8; ++e)
        if (n + e < N) dst[e] = 0;
    }
  }
}

}  // namespace

}  // namespace bsq
