// Products of a few rows (single tokens, small batches, few outputs): FP8 x FP8_TILE,
// plain or grouped by expert, and the gated projections on those or on bf16.
//
// Such a product is bound by reading the weights once, so nothing is staged: a lane
// loads 32 bytes of a weight row and of an activation row straight into the
// registers that the matrix instructions take, all loads of a round before its first
// product, and K is split over the waves of a workgroup, which meet in LDS.
//
// A step covers 128 bytes of 16 weight rows: lane (r = l % 16, q = l / 16) holds
// bytes 32 q + [0, 32) of row r.  That is K = 128 on one
// v_mfma_scale_f32_16x16x128_f8f6f4 from a zero accumulator, added with the block's
// scales, or K = 64 on two v_mfma_f32_16x16x32_bf16 (any order of K is right that
// both operands share).  Rows past the end of an operand re-read its last row and
// are never stored; pieces past the end of K count as zeros.
//
// One token, weights from HBM: FP8 4096 -> 8192 10.1 .. 10.8 us, 3.2 TB/s, and 4096 -> 11008 gated
// 20.2 .. 23, 4.2 TB/s, of 6.5 and 17.5 at a large copy's rate (the launch and one trip to
// memory are some 3 us of each); gated bf16 40 of 35; 256 rows of 32 experts, K 2048, N 4096,
// 77 of 53.
#include "block_gemm.h"

namespace mxq {
namespace {

// NT weight tiles of 16 rows (gated: of the gate and of the up projection each),
// K over W waves, S steps of a wave in flight.
template <int EL, bool GATED, bool GRP, int W, int S>
__global__ __launch_bounds__(64 * W) void block_few_kernel(BlockP p) {
  constexpr int NT = GATED ? 2 : 1;
  __shared__ v4f part[W][NT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const uint32_t bid = block_index();
  const int tn = bid % (uint32_t)p.tiles_n, tm = bid / (uint32_t)p.tiles_n;
  int m0 = tm * 16;
  if constexpr (GRP) {
    GroupTile gt;
    if (!GroupScan(p.goff, p.groups, p.M, 16).find(tm, gt)) return;
    m0 = gt.row0;
    p.M = gt.row1;
    const int64_t first = (int64_t)gt.g * p.N;
    p.w += first * p.ldw;
    p.ws += first / 128 * p.ldws;
    if (p.bias) p.bias += first;
  } else if (tm >= p.tiles_m) {
    return;
  }
  const int n0 = tn * 16;
  const int row_bytes = EL == EL_FP8 ? p.K : 2 * p.K, steps = (row_bytes + 127) / 128;
  const int64_t n = min(n0 + r16, p.N - 1), m = min(m0 + r16, p.M - 1);
  const uint8_t* const arow = p.a + m * p.lda + 32 * q;
  const uint8_t* wrow[NT];
  wrow[0] = p.w + n * p.ldw + 32 * q;
  if constexpr (GATED) wrow[1] = p.w2 + n * p.ldw2 + 32 * q;

  v4f acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = v4f{};
  for (int s0 = wave; s0 < steps; s0 += W * S) {
    v4i wf[S][NT][2], af[S][2];
    float sa[S], sw[S][NT];
#pragma unroll
    for (int t = 0; t < S; ++t) {
      const int s = s0 + t * W;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bool in = 128 * s + 32 * q + 16 * h < row_bytes;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          wf[t][j][h] = v4i{};
          if (in) wf[t][j][h] = *reinterpret_cast<const v4i*>(wrow[j] + (int64_t)128 * s + 16 * h);
        }
        af[t][h] = v4i{};
        if (in) af[t][h] = *reinterpret_cast<const v4i*>(arow + (int64_t)128 * s + 16 * h);
      }
      if constexpr (EL == EL_FP8) {
        const int b = min(s, steps - 1);
        sa[t] = p.as[b * p.ldas + m];
        sw[t][0] = p.ws[(int64_t)(n0 / 128) * p.ldws + b];
        if constexpr (GATED) sw[t][1] = p.ws2[(int64_t)(n0 / 128) * p.ldws2 + b];
      }
    }
#pragma unroll
    for (int t = 0; t < S; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (EL == EL_FP8) {
          const v8i wv = __builtin_shufflevector(wf[t][j][0], wf[t][j][1], 0, 1, 2, 3, 4, 5, 6, 7);
          const v8i av = __builtin_shufflevector(af[t][0], af[t][1], 0, 1, 2, 3, 4, 5, 6, 7);
          const v4f d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, v4f{}, 0, 0, 0, 127, 0, 127);
          const float sc = sa[t] * sw[t][j];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][e] = fmaf(d[e], sc, acc[j][e]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, wf[t][j][h]),
                                                             __builtin_bit_cast(v8bf, af[t][h]), acc[j], 0, 0, 0);
        }
      }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) part[wave][j][lane] = acc[j];
  __syncthreads();
  // lane l: activation row l % 16, outputs 4 (l / 16) + [0, 4)
  if (wave != 0 || m0 + r16 >= p.M) return;
  v4f sum[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    sum[j] = acc[j];
#pragma unroll
    for (int w = 1; w < W; ++w) sum[j] += part[w][j][lane];
  }
  uint16_t* const orow = p.out + m * p.ld_out;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = n0 + 4 * q + e;
    if (c >= p.N) continue;
    float v = sum[0][e];
    int to = c;
    if constexpr (GATED) {
      if (EL == EL_BF16 && p.gate) {
        p.gate[m * p.ld_saved + c] = v;
        p.up[m * p.ld_saved + c] = sum[1][e];
      }
      v = activation<false>(p.act, v) * sum[1][e];
    } else {
      if (p.col_map) to = p.col_map[c];
      if (to < 0 || to >= p.n_out) continue;
      if (p.bias) v += bf16_bits_to_f32(p.bias[to]);
    }
    orow[to] = (uint16_t)pack_bf16_rne(v, 0.f);
  }
}

template <int EL, bool GATED, bool GRP, int W, int S>
hipError_t go(const BlockP& p, hipStream_t s) {
  block_few_kernel<EL, GATED, GRP, W, S><<<grid_of((int64_t)p.tiles_m * p.tiles_n), 64 * W, 0, s>>>(p);
  return hipGetLastError();
}

template <int EL, bool GATED, bool GRP>
hipError_t by_waves(BlockP p, hipStream_t s) {
  p.tiles_m = GRP ? (int)group_tiles_bound(p.M, p.groups, 16) : (p.M + 15) / 16;
  p.tiles_n = (p.N + 15) / 16;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  constexpr int S = GATED ? 4 : 8;
  // K over 16 waves where the workgroups leave compute units idle
  if (tiles <= 256) return go<EL, GATED, GRP, 16, GATED ? 2 : 4>(p, s);
  return go<EL, GATED, GRP, 4, S>(p, s);
}

}  // namespace

// Where this kernel is the faster one, weights from HBM: up to 16 rows (gated: 32),
// by expert on average, and wherever its 16 x 16 tiles fit the GPU about once (FP8, K =
// 1152 / 4096: 32 x 4096 7.0 / 11.2 us against 7.1 / 15.8 on the tiled kernels, 128 x 1024
// 5.7 against 6.2, 64 x 4608 10.0 / 7.2; gated, 32 x 4096 x 4096 18.1 / 22, bf16 30 / 33, 64 rows
// 28.6 / 22.0, 51 / 34).
bool block_few(const BlockP& p, bool gated) {
  if (p.goff) return p.M <= 16 * (int64_t)p.groups;
  return p.M <= (gated ? 32 : 16) || (double)((p.M + 15) / 16) * ((p.N + 15) / 16) <= (gated ? 320 : 576);
}

hipError_t launch_block_few(const BlockP& p, int el, bool gated, hipStream_t s) {
  if (el == EL_BF16) return by_waves<EL_BF16, true, false>(p, s);
  if (gated) return by_waves<EL_FP8, true, false>(p, s);
  return p.goff ? by_waves<EL_FP8, false, true>(p, s) : by_waves<EL_FP8, false, false>(p, s);
}

}  // namespace mxq
