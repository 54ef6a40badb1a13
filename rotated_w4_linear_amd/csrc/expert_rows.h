// Which rows and weights a workgroup of the W4 kernels works on: consecutive
// tokens and one weight block (AllRows), or the rows of a mixture of experts, in
// expert order, and one block per expert (ExpertRows).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "paro_internal.h"

namespace paro {
namespace w4 {

struct AllRows {
  static constexpr bool kExperts = false, kGather = false;
};

// Inclusive sum over the wavefront's lanes (rows of 16 by shifts, then across them).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);  // row_shr 2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);  // row_shr 4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);  // row_shr 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast 31 into rows 2 and 3
  return v;
}

// Rows first .. end - 1 (in expert order) of one expert.
struct ExpertTile {
  int expert, first, end;
};

// GATHER: row r of the operand is its token, order[r] / k; else row r itself.
template <bool GATHER>
struct ExpertRows {
  static constexpr bool kExperts = true, kGather = GATHER;
  ExpertRouting t;

  // Rows of expert e0 + lane: first and last + 1, inside the rows whatever the
  // tables say.
  __device__ __forceinline__ void rows_of(int e0, int& a, int& z) const {
    const int e = e0 + (int)(threadIdx.x & 63);
    a = min(max(t.offsets[min(e, t.E)], 0), t.R);
    z = min(max(t.offsets[min(e + 1, t.E)], 0), t.R);
  }

  // Every wavefront looks for its workgroup's tile itself, 64 experts at a time: the
  // routing has no room for the tiles of each kernel's size.
  //
  // find: block `index` of all experts' rows cut into blocks of at most bm; false
  // past the last one.
  __device__ __forceinline__ bool find(int index, int bm, ExpertTile& out) const {
    for (int e0 = 0; e0 < t.E; e0 += 64) {
      int a, z;
      rows_of(e0, a, z);
      const int n = z > a ? (z - a + bm - 1) / bm : 0, s = wave_scan(n);
      const int total = __builtin_amdgcn_readlane(s, 63);
      if (index < total) {
        const int at = __builtin_ctzll(__ballot(s > index));
        const int mb = index - (__builtin_amdgcn_readlane(s, at) - __builtin_amdgcn_readlane(n, at));
        out.expert = e0 + at;
        out.first = __builtin_amdgcn_readlane(a, at) + bm * mb;
        out.end = min(__builtin_amdgcn_readlane(z, at), out.first + bm);
        return true;
      }
      index -= total;
    }
    return false;
  }

  // The tile of workgroup b, of all blocks of at most bm rows by nblk column
  // blocks; false where there is none. The tiles, walked expert by expert, eight
  // column blocks at a time, over the expert's rows, are cut into eight equal
  // runs, one for each XCD (workgroup b runs on XCD b % 8): an XCD's workgroups
  // then share few experts' weights and few rows, whatever the numbers of rows
  // and columns. (Column blocks dealt out to the XCDs instead, as for one weight
  // block, leave XCDs idle where there are few of them.)
  __device__ __forceinline__ bool find_tile(int b, int bm, int nblk, ExpertTile& out, int& nb) const {
    int a, z, blocks = 0;
    for (int e0 = 64; e0 < t.E; e0 += 64) {
      rows_of(e0, a, z);
      blocks += __builtin_amdgcn_readlane(wave_scan(z > a ? (z - a + bm - 1) / bm : 0), 63);
    }
    rows_of(0, a, z);
    int n = z > a ? (z - a + bm - 1) / bm : 0, s = wave_scan(n), total = __builtin_amdgcn_readlane(s, 63);
    const int all = (blocks + total) * nblk, per = (all + 7) >> 3;
    const int idx = b >> 3, tile = (b & 7) * per + idx;
    if (idx >= per || tile >= all) return false;
    int block = tile / nblk, e0 = 0;  // (its expert has the block of rows that it would be in, were they walked first)
    while (block >= total) {
      block -= total;
      e0 += 64;
      rows_of(e0, a, z);
      n = z > a ? (z - a + bm - 1) / bm : 0;
      s = wave_scan(n);
      total = __builtin_amdgcn_readlane(s, 63);
    }
    const int at = __builtin_ctzll(__ballot(s > block));
    const int rows = __builtin_amdgcn_readlane(n, at);
    // the expert's tiles: its blocks before it times nblk come first
    const int i = tile % nblk + (block - (__builtin_amdgcn_readlane(s, at) - rows)) * nblk;
    const int g = i / (8 * rows), rem = i - g * 8 * rows, cols = min(8, nblk - 8 * g);
    const int mb = rem / cols;
    nb = 8 * g + rem - mb * cols;
    out.expert = e0 + at;
    out.first = __builtin_amdgcn_readlane(a, at) + bm * mb;
    out.end = min(__builtin_amdgcn_readlane(z, at), out.first + bm);
    return true;
  }

  // Blocks that an expert's n rows make: those of more than bm / 2 rows, or (LAST) the
  // one of fewer that there may be.
  template <bool LAST>
  static __device__ __forceinline__ int blocks_of(int n, int bm) {
    if (n <= 0) return 0;
    const int full = n / bm, rest = n - full * bm;
    return LAST ? (rest > 0 && 2 * rest <= bm) : full + (2 * rest > bm);
  }
  template <bool LAST>
  __device__ __forceinline__ int count_blocks(int bm) const {
    int blocks = 0;
    for (int e0 = 0; e0 < t.E; e0 += 64) {
      int a, z;
      rows_of(e0, a, z);
      blocks += __builtin_amdgcn_readlane(wave_scan(blocks_of<LAST>(z - a, bm)), 63);
    }
    return blocks;
  }

  // Tile `tile` of these blocks by nblk column blocks, walked as above. There is one.
  template <bool LAST>
  __device__ __forceinline__ void tile_of(int tile, int bm, int nblk, ExpertTile& out, int& nb) const {
    int a, z, n, s, total, block = tile / nblk;  // (its expert has the block that it would be in, were they walked first)
    for (int e0 = 0;; e0 += 64) {
      rows_of(e0, a, z);
      n = blocks_of<LAST>(z - a, bm);
      s = wave_scan(n);
      total = __builtin_amdgcn_readlane(s, 63);
      if (block < total || e0 + 64 >= t.E) {
        out.expert = e0;
        break;
      }
      block -= total;
    }
    const int at = __builtin_ctzll(__ballot(s > block) | 1ull << 63);
    const int rows = __builtin_amdgcn_readlane(n, at);
    // the expert's tiles: its blocks before it times nblk come first
    const int i = tile % nblk + (block - (__builtin_amdgcn_readlane(s, at) - rows)) * nblk;
    const int g = i / (8 * rows), rem = i - g * 8 * rows, cols = min(8, nblk - 8 * g);
    const int mb = rem / cols;
    nb = 8 * g + rem - mb * cols;
    out.expert += at;
    const int first = __builtin_amdgcn_readlane(a, at);
    out.end = __builtin_amdgcn_readlane(z, at);
    out.first = first + bm * (LAST ? (out.end - first) / bm : mb);
    out.end = min(out.end, out.first + bm);
  }

  // The same where a block of at most bm / 2 rows takes half the time: those come
  // last, in eight runs of their own, so that the XCDs' work is even and ends with the
  // short tiles (calls in a row, find_tile's walk | this: 4096 tokens through 8 experts,
  // skewed, 4096 -> 14336 1932 | 1817 us; a whole gradient of 2048 tokens, 32 experts,
  // 2048 -> 1536, 360 | 324 by the first product's tiles and 336 | 324 by the second's).
  // At most 16 workgroups more than tiles.
  __device__ __forceinline__ bool find_tile_halves(int b, int bm, int nblk, ExpertTile& out, int& nb) const {
    int all = count_blocks<false>(bm) * nblk, per = (all + 7) >> 3, idx = b >> 3, tile = (b & 7) * per + idx;
    if (idx < per) {
      if (tile >= all) return false;
      tile_of<false>(tile, bm, nblk, out, nb);
      return true;
    }
    idx -= per;
    all = count_blocks<true>(bm) * nblk;
    per = (all + 7) >> 3;
    tile = (b & 7) * per + idx;
    if (idx >= per || tile >= all) return false;
    tile_of<true>(tile, bm, nblk, out, nb);
    return true;
  }

  // (pair of row r: inside the tables whatever they say)
  __device__ __forceinline__ int pair(int r) const { return min(max(t.order[r], 0), t.R - 1); }
  __device__ __forceinline__ int source(int r) const { return GATHER ? pair(r) / t.k : r; }
  __device__ __forceinline__ float weight(int r) const { return t.weights[pair(r)]; }
};

// Row `at` of the block from m0 on, as a row of the operand relative to the
// kernel's base (its first row for consecutive ones), and the operand's rows.
template <class ROWS>
__device__ __forceinline__ int source_row(const ROWS& rows, int m0, int at) {
  if constexpr (ROWS::kGather) return rows.source(m0 + at);
  else return at;
}
template <class ROWS>
__device__ __forceinline__ int rows_tokens(const ROWS& rows) {
  if constexpr (ROWS::kGather) return rows.t.M;
  else return 0;
}

}  // namespace w4
}  // namespace paro
