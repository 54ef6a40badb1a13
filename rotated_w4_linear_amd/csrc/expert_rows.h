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

// Rows first .. end - 1 (in expert order) of one expert.
struct ExpertTile {
  int expert, first, end;
};

// GATHER: row r of the operand is its token, order[r] / k; else row r itself.
template <bool GATHER>
struct ExpertRows {
  static constexpr bool kExperts = true, kGather = GATHER;
  ExpertRouting t;

  // Block `index` of all experts' rows cut into blocks of at most bm; false
  // past the last one. Every wavefront looks for itself, 64 experts at a time:
  // the tables have no room for the blocks of each kernel's size, and a scan of
  // offsets that sit in L2 is shorter than a tile's first loads. (Offsets are
  // held inside the rows whatever the tables say.)
  __device__ __forceinline__ bool find(int index, int bm, ExpertTile& out) const {
    const int lane = threadIdx.x & 63;
    for (int e0 = 0; e0 < t.E; e0 += 64) {
      const int e = e0 + lane;
      const int a = min(max(t.offsets[min(e, t.E)], 0), t.R), b = min(max(t.offsets[min(e + 1, t.E)], 0), t.R);
      const int n = b > a ? (b - a + bm - 1) / bm : 0;
      int s = n;
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) {
        const int o = __shfl_up(s, x);
        if (lane >= x) s += o;
      }
      const int total = __builtin_amdgcn_readlane(s, 63);
      if (index < total) {
        const int at = __builtin_ctzll(__ballot(s > index));
        out.expert = e0 + at;
        out.first = __builtin_amdgcn_readlane(a, at) +
                    bm * (index - (__builtin_amdgcn_readlane(s, at) - __builtin_amdgcn_readlane(n, at)));
        out.end = min(__builtin_amdgcn_readlane(b, at), out.first + bm);
        return true;
      }
      index -= total;
    }
    return false;
  }

  // Blocks of bm rows that the experts make.
  __device__ __forceinline__ int blocks(int bm) const {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int e0 = 0; e0 < t.E; e0 += 64) {
      const int e = e0 + lane;
      const int a = min(max(t.offsets[min(e, t.E)], 0), t.R), b = min(max(t.offsets[min(e + 1, t.E)], 0), t.R);
      n += b > a ? (b - a + bm - 1) / bm : 0;
    }
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) n += __shfl_xor(n, x);
    return __builtin_amdgcn_readfirstlane(n);
  }

  // The tile of workgroup b, of all blocks of at most bm rows by nblk column
  // blocks; false where there is none. The tiles, walked expert by expert, eight
  // column blocks at a time, over the expert's rows, are cut into eight equal
  // runs, one for each XCD (workgroup b runs on XCD b % 8): an XCD's workgroups
  // then share few experts' weights and few rows, whatever the numbers of rows
  // and columns. (Column blocks dealt out to the XCDs instead, as for one weight
  // block, leave XCDs idle where there are few of them.)
  __device__ __forceinline__ bool find_tile(int b, int bm, int nblk, ExpertTile& out, int& nb) const {
    const int lane = threadIdx.x & 63;
    const int all = blocks(bm) * nblk, per = (all + 7) >> 3;
    const int idx = b >> 3, tile = (b & 7) * per + idx;
    if (idx >= per || tile >= all) return false;
    int before = 0;  // tiles of the experts before e0
    for (int e0 = 0; e0 < t.E; e0 += 64) {
      const int e = e0 + lane;
      const int a = min(max(t.offsets[min(e, t.E)], 0), t.R), z = min(max(t.offsets[min(e + 1, t.E)], 0), t.R);
      const int n = (z > a ? (z - a + bm - 1) / bm : 0) * nblk;
      int s = n;
#pragma unroll
      for (int x = 1; x < 64; x <<= 1) {
        const int o = __shfl_up(s, x);
        if (lane >= x) s += o;
      }
      const int total = __builtin_amdgcn_readlane(s, 63);
      if (tile < before + total) {
        const int at = __builtin_ctzll(__ballot(before + s > tile));
        const int rows = __builtin_amdgcn_readlane(n, at) / nblk;
        const int i = tile - before - (__builtin_amdgcn_readlane(s, at) - __builtin_amdgcn_readlane(n, at));
        const int g = i / (8 * rows), rem = i - g * 8 * rows, cols = min(8, nblk - 8 * g);
        const int mb = rem / cols;
        nb = 8 * g + rem - mb * cols;
        out.expert = e0 + at;
        out.first = __builtin_amdgcn_readlane(a, at) + bm * mb;
        out.end = min(__builtin_amdgcn_readlane(z, at), out.first + bm);
        return true;
      }
      before += total;
    }
    return false;
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
