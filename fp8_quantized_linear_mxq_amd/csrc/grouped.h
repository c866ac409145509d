// Row tiles of a product grouped by expert: group g owns rows
// [off[g], off[g+1]) of the activations, the offsets live in device memory.
//
// The host only knows an upper bound of the number of row tiles (the groups'
// sizes are on the device and nothing waits for them), so every workgroup
// counts the tiles itself: a wave loads the offsets 64 groups at a time, scans
// the tile counts and picks the group that holds its tile.  That costs one
// load and some 60 instructions next to a product's main loop and spares a
// launch that builds a table.  Offsets are clamped to [0, M] and a group
// whose end lies before its start is empty, so offsets that are not sorted
// give unspecified results but no access outside the operands.  Such offsets can
// count a row in many groups: the sums are unsigned, which holds the tiles of 64
// groups (every other one with all of up to 2**30 rows, 16 to a tile) on top of
// the tiles before them, and a grid never works on more tiles than it was sized
// for.
#pragma once

#include "device_common.h"
#include "gemm_common.h"

namespace mxq {

// Rows [row0, row1) of group g, starting at the tile's first row.
struct GroupTile {
  int g, row0, row1;
};

__device__ __forceinline__ int group_rows(const int32_t* off, int groups, int M, int g, int& o0) {
  if (g >= groups) {
    o0 = 0;
    return 0;
  }
  const int a = off[g], b = off[g + 1];
  o0 = min(max(a, 0), M);
  const int o1 = min(max(b, 0), M);
  return max(o1 - o0, 0);
}

__device__ __forceinline__ uint32_t wave_scan(uint32_t v, int lane) {   // inclusive sum
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The row tiles of all groups.  Every lane of the wave takes part; up to 64
// groups are loaded and scanned once.
struct GroupScan {
  const int32_t* off;
  int groups, M, rows;
  int o0, n;         // of group `lane` of the first 64: first row, rows
  uint32_t upto;     // and tiles up to its end

  __device__ __forceinline__ GroupScan(const int32_t* off_, int groups_, int M_, int rows_)
      : off(off_), groups(groups_), M(M_), rows(rows_) {
    const int lane = threadIdx.x & 63;
    n = group_rows(off, groups, M, lane, o0);
    upto = wave_scan((n + rows - 1) / rows, lane);
  }

  // Tiles of all groups, at most `most` (the bound that the grid was sized for).
  __device__ __forceinline__ int tiles(int most) const {
    const int lane = threadIdx.x & 63;
    uint32_t total = min(last(upto), (uint32_t)most);
    for (int c = 64; c < groups; c += 64) {
      int o;
      const int m = group_rows(off, groups, M, c + lane, o);
      total = min(total + last(wave_scan((m + rows - 1) / rows, lane)), (uint32_t)most);
    }
    return (int)total;
  }

  // The group and rows of tile t (tiles of a group are consecutive); false
  // when there are fewer tiles.
  __device__ __forceinline__ bool find(int t, GroupTile& out) const {
    const int lane = threadIdx.x & 63;
    int o = o0, m = n;
    uint32_t up = upto;
    for (int c = 0;;) {
      const uint64_t past = __ballot(up > (uint32_t)t);
      if (past) {
        const int l = __builtin_ctzll(past);
        const int len = __builtin_amdgcn_readlane(m, l);
        // tiles before the group: at most t, as no group before reaches past t
        const int first = __builtin_amdgcn_readlane((int)up, l) - (len + rows - 1) / rows;
        out.g = c + l;
        out.row0 = __builtin_amdgcn_readlane(o, l) + (t - first) * rows;
        out.row1 = __builtin_amdgcn_readlane(o, l) + len;
        return true;
      }
      c += 64;
      if (c >= groups) return false;
      const uint32_t before = last(up);
      m = group_rows(off, groups, M, c + lane, o);
      up = before + wave_scan((m + rows - 1) / rows, lane);
    }
  }

 private:
  static __device__ __forceinline__ uint32_t last(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  }
};

// Turns the parameters of a grouped product into those of the one product
// that row tile t belongs to: rows up to the group's end, the group's weights
// and bias.  Returns the tile's first row, or -1 when there is no tile t.
__device__ __forceinline__ int enter_group(GemmP& p, const GroupScan& s, int t) {
  GroupTile gt;
  if (!s.find(t, gt)) return -1;
  p.M = gt.row1;
  const int64_t first = (int64_t)gt.g * p.N;
  p.w += first * p.ldw;
  p.ws += first * p.ldws;
  if (p.bias) p.bias += first;
  return gt.row0;
}

// Most row tiles that M rows in `groups` groups can make: a group that has
// rows adds at most one partial tile.
inline int64_t group_tiles_bound(int64_t M, int64_t groups, int64_t rows) {
  const int64_t used = groups < M ? groups : M;
  return (M + used * (rows - 1)) / rows;
}

}  // namespace mxq
