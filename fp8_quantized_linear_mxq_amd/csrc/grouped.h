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
// give unspecified results but no access outside the operands.
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

__device__ __forceinline__ int wave_scan(int v, int lane) {   // inclusive sum
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// All row tiles of `rows` rows.  Every lane of the wave takes part.
__device__ __forceinline__ int group_tiles(const int32_t* off, int groups, int M, int rows) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int c = 0; c < groups; c += 64) {
    int o0;
    const int n = group_rows(off, groups, M, c + lane, o0);
    total += __shfl(wave_scan((n + rows - 1) / rows, lane), 63);
  }
  return __builtin_amdgcn_readfirstlane(total);
}

// The group and rows of tile t (tiles of a group are consecutive); false when
// there are fewer tiles.
__device__ __forceinline__ bool group_tile(const int32_t* off, int groups, int M, int rows, int t,
                                           GroupTile& out) {
  const int lane = threadIdx.x & 63;
  int before = 0;
  for (int c = 0; c < groups; c += 64) {
    int o0;
    const int n = group_rows(off, groups, M, c + lane, o0);
    const int tiles = (n + rows - 1) / rows;
    const int upto = before + wave_scan(tiles, lane);
    const uint64_t past = __ballot(upto > t);
    if (past) {
      const int l = __builtin_ctzll(past);
      const int first = __builtin_amdgcn_readlane(upto - tiles, l);
      const int start = __builtin_amdgcn_readlane(o0, l), len = __builtin_amdgcn_readlane(n, l);
      out.g = c + l;
      out.row0 = start + (t - first) * rows;
      out.row1 = start + len;
      return true;
    }
    before = __builtin_amdgcn_readlane(upto, 63);
  }
  return false;
}

// Turns the parameters of a grouped product into those of the one product
// that row tile t belongs to: rows up to the group's end, the group's weights
// and bias.  Returns the tile's first row, or -1 when there is no tile t.
__device__ __forceinline__ int enter_group(GemmP& p, int rows, int t) {
  GroupTile gt;
  if (!group_tile(p.goff, p.groups, p.M, rows, t, gt)) return -1;
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
