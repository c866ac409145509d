// Small products (single tokens, small batches, few outputs; in a product
// grouped by expert, few rows per group): INT8 x INT8, and grouped by expert also
// MXFP4 x MXFP4 and bf16 x MXFP4.
//
// Such a product is bound by reading W once, so nothing is staged: every lane
// loads its 16-byte pieces of the weight rows straight into the registers the
// matrix instruction takes, eight steps at a time, and the reduction is split
// over the four waves of a workgroup, which meet in LDS at the end.
//
// A step covers 64 bytes of a weight row: lane (r = l % 16, q = l / 16) holds
// bytes 16 q + [0, 16) of row r.  That is K = 64 (int8) on
// v_mfma_i32_16x16x64_i8; K = 128 (E2M1 codes, one 32-block per lane) on one
// v_mfma_scale_f32_16x16x128_f8f6f4, or, with bf16 activations, dequantized
// exactly to bf16 for four v_mfma_f32_16x16x32_bf16 (the lane's block split
// in four runs of 8; both operands permute K alike).  Waves take pairs of
// steps in turn, so each reads whole 128-byte lines.  Rows past the end of an
// operand re-read its last row and are never stored.
//
// One token, weights from HBM: int8 1152 -> 4608 in 4.6 us (5.3 MB, and 2.6 us
// of that is an empty launch), 2048 -> 1536 on 8 of 64 experts in 8.3 us (25 MB,
// 3.0 TB/s): every wave's loads are in flight at once, and what is left is
// starting the workgroups and one round trip to memory.
#include "device_common.h"
#include "gemm_common.h"
#include "gemm_pipe.h"
#include "grouped.h"
#include "kernels.h"

#include <type_traits>

namespace mxq {
namespace {

enum : int { P_I8 = 0, P_MX4 = 1, P_BF4 = 2 };

constexpr int kWaves = 4;
constexpr int kPairs = 4;    // step pairs in flight per wave

// NT weight tiles and one activation tile of 16 rows per workgroup.
template <int P, int NT, bool GRP>
__global__ __launch_bounds__(64 * kWaves) void gemm_few_kernel(GemmP p) {
  using Acc = std::conditional_t<P == P_I8, v4i, v4f>;
  constexpr int S = 2 * kPairs;                      // steps per round
  constexpr int AV = P == P_BF4 ? 4 : 1;             // 16-byte pieces of a per step
  static_assert(NT <= kWaves, "an output quad per thread");
  __shared__ Acc part[kWaves][NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const uint32_t bid = block_index();
  const int tn = bid % (uint32_t)p.tiles_n, tm = bid / (uint32_t)p.tiles_n;
  // in a plain product only the workgroups that fill the grid's last row are past
  // the end (then of at most 16 rows): they compute and store nothing, since a
  // test here would keep the arguments' loads behind it (5.0 -> 5.4 us for one token)
  int m0 = tm * 16;
  if constexpr (GRP) {
    m0 = enter_group(p, GroupScan(p.goff, p.groups, p.M, 16), tm);
    if (m0 < 0) return;
  }
  const int n0 = tn * 16 * NT;
  const int row_bytes = P == P_I8 ? p.K : p.K / 2;   // of a weight row
  const int steps = (row_bytes + 63) / 64;

  const uint8_t* wrow[NT];
  const uint8_t* wscl[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = min(n0 + j * 16 + r16, p.N - 1);
    wrow[j] = p.w + n * p.ldw + 16 * q;
    wscl[j] = p.ws + n * p.ldws;
  }
  const int64_t mr = min(m0 + r16, p.M - 1);
  const uint8_t* const arow = p.a + mr * p.lda + (P == P_BF4 ? 64 : 16) * q;
  const uint8_t* const ascl = p.as + mr * p.ldas;

  // The output quad this thread finishes: lane l of weight tile `wave` holds
  // activation row l % 16 and weight rows 4 (l / 16) + [0, 4).  Its scales, bias
  // and columns are on their way while the weights stream.
  const int m = m0 + r16, n = n0 + wave * 16 + 4 * q;
  const bool mine = wave < NT && m < p.M;
  float sa = 0.f, sw[4], bs[4];
  int col[4];
  if (mine) {
    if constexpr (P == P_I8) sa = *reinterpret_cast<const float*>(p.as + (int64_t)m * p.ldas);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int ne = min(n + e, p.N - 1);
      if constexpr (P == P_I8) sw[e] = *reinterpret_cast<const float*>(p.ws + (int64_t)ne * p.ldws);
      col[e] = p.col_map ? p.col_map[ne] : ne;
      if (n + e >= p.N || col[e] >= p.n_out) col[e] = -1;
      bs[e] = p.bias && col[e] >= 0 ? bf16_bits_to_f32(p.bias[col[e]]) : 0.f;
    }
  }

  // The fp32 pairs flush their sums into LDS once per round of the loop (K = 4096
  // over the four waves, a chain of 8 scaled or 32 bf16 instructions per wave): one
  // chain over a long K would lose what lies below the last place of its running
  // sum.  A sum of K values passes at most 32 + K / 4096 roundings.  A second
  // accumulator in registers would take the kernel from three (MXFP4) and two
  // (bf16) waves per SIMD to two and one: 2 tokens on 4 of 32 experts, bf16, K =
  // 4096, N = 2048 14.6 -> 17.3 us.
  Acc acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    acc[j] = Acc{};
    if constexpr (P != P_I8) part[wave][j][lane] = Acc{};
  }

  for (int s0 = 2 * wave; s0 < steps; s0 += 2 * kPairs * kWaves) {
    v4i wf[S][NT], af[S][AV];
    uint32_t wd[S][NT], ad[S];
#pragma unroll
    for (int t = 0; t < S; ++t) {
      const int s = s0 + (t >> 1) * 2 * kWaves + (t & 1);
      // pieces past the end of a row read nothing and count as zeros
      const bool in = 64 * s + 16 * q < row_bytes;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        wf[t][j] = v4i{};
        if (in) wf[t][j] = *reinterpret_cast<const v4i*>(wrow[j] + 64 * s);
        if constexpr (P != P_I8) {
          wd[t][j] = 0;
          if (in) wd[t][j] = *reinterpret_cast<const uint32_t*>(wscl[j] + 4 * s);
        }
      }
#pragma unroll
      for (int v = 0; v < AV; ++v) {
        af[t][v] = v4i{};
        if (in) af[t][v] = *reinterpret_cast<const v4i*>(arow + (P == P_BF4 ? 256 : 64) * s + 16 * v);
      }
      if constexpr (P == P_MX4) {
        ad[t] = 0;
        if (in) ad[t] = *reinterpret_cast<const uint32_t*>(ascl + 4 * s);
      }
    }
#pragma unroll
    for (int t = 0; t < S; ++t) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (P == P_I8) {
          acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[t][j], af[t][0], acc[j], 0, 0, 0);
        } else if constexpr (P == P_MX4) {
          const v4i &w4 = wf[t][j], &a4 = af[t][0];
          const v8i wv = __builtin_shufflevector(w4, w4, 0, 1, 2, 3, -1, -1, -1, -1);
          const v8i av = __builtin_shufflevector(a4, a4, 0, 1, 2, 3, -1, -1, -1, -1);
          acc[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              wv, av, acc[j], 4, 4, 0, (int)(wd[t][j] >> (8 * q)), 0, (int)(ad[t] >> (8 * q)));
        } else {
          // the block scale with its exponent raised by 2 (undone below), so
          // that code 0 is a normal fp32 scale for the converts
          const float sc = __uint_as_float((((wd[t][j] >> (8 * q)) & 0xFFu) + 2u) << 23);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const uint32_t d = (uint32_t)wf[t][j][v];
            const v8bf wv = __builtin_bit_cast(v8bf, make_uint4(
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, sc, 0)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, sc, 1)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, sc, 2)),
                __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, sc, 3))));
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, __builtin_bit_cast(v8bf, af[t][v]), acc[j], 0, 0, 0);
          }
        }
      }
    }
    if constexpr (P != P_I8) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        part[wave][j][lane] += acc[j];
        acc[j] = Acc{};
      }
      asm volatile("" ::: "memory");   // in LDS, not moved to registers for the loop
    }
  }
  if constexpr (P == P_I8) {   // exact in int32
#pragma unroll
    for (int j = 0; j < NT; ++j) part[wave][j][lane] = acc[j];
  }
  __syncthreads();
  if (!mine) return;

  Acc sum = part[0][wave][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) sum += part[w][wave][lane];
  uint16_t* const orow = p.out + (int64_t)m * p.ld_out;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (col[e] < 0) continue;
    float v;
    if constexpr (P == P_I8) {
      v = ((float)sum[e] * sa) * sw[e];
      if constexpr (!GRP) {
        const float* u = p.u + (int64_t)m * p.ld_u;
        const uint16_t* l2 = p.l2t + (int64_t)col[e] * p.rank;
        for (int r = 0; r < p.rank; ++r) v = fmaf(u[r], bf16_bits_to_f32(l2[r]), v);
      }
    } else {
      v = P == P_BF4 ? sum[e] * 0.25f : sum[e];
    }
    orow[col[e]] = (uint16_t)f32_to_bf16_bits(v + bs[e]);
  }
}

template <int P, int NT, bool GRP>
hipError_t go(GemmP p, hipStream_t s) {
  p.tiles_m = GRP ? (int)group_tiles_bound(p.M, p.groups, 16) : (p.M + 15) / 16;
  p.tiles_n = (p.N + 16 * NT - 1) / (16 * NT);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  gemm_few_kernel<P, NT, GRP><<<grid_of(tiles), 64 * kWaves, 0, s>>>(p);
  return hipGetLastError();
}

}  // namespace

// Where this kernel is the faster one, against the tiled kernels, operands
// from HBM: up to 16 rows (int8 16 x 4096 x 4096 7.3 us against 8.9), and wherever
// the workgroups fit the GPU about once (int8, K = 1152 / 4096: 64 x 1024 4.1 / 7.8
// us against 5.5 / 12.9, 128 x 1024 4.7 / 9.6 against 5.6 / 12.6 with two weight
// tiles, 256 x 1024 6.2 / 13.8 against 5.7 / 12.1; the low-rank branch is one
// output at a time here, so it stays with few rows).  By expert: int8 also up to
// four rows per group on average, where the weights' traffic decides (64 groups, N
// = 1536, K = 2048: 8 rows 8.1 / 10.7, 128 rows 35 / 42, 512 rows 52 / 45); 4-bit
// weights up to 768 tiles of 16 x 16 (K = 4096, N = 2048, one row each for 4 / 8 / 14
// experts: MXFP4 7.6 / 11.4 / 18.7 us against 10.2 / 12.3 / 15.5, bf16 x MXFP4 9.4 /
// 13.7 / 23.0 against 19.6 / 19.2 / 20.2; 264 rows, 4 experts, N = 387, K = 2176: bf16 x
// MXFP4 8.4 against 17.6).
bool few_rows(const GemmArgs& a) {
  const double tiles = gemm_tiles(a, 16, 16);
  if (a.goff && a.a_fmt != FMT_INT8) return tiles <= 768;
  if (a.goff ? a.M <= 4 * a.groups : a.M <= 16) return true;
  return a.rank == 0 && tiles <= 512;
}

hipError_t launch_gemm_few(const GemmArgs& a, hipStream_t s) {
  const GemmP p = gemm_params(a);
  if (a.a_fmt == FMT_MXFP4) return go<P_MX4, 2, true>(p, s);
  if (a.a_fmt != FMT_INT8) return go<P_BF4, 2, true>(p, s);
  // int8: one weight tile per workgroup where that fits the GPU once, or rows are few
  const bool two = !(a.goff ? a.M <= 4 * a.groups : a.M <= 16) && gemm_tiles(a, 16, 16) > 256;
  if (a.goff) return two ? go<P_I8, 2, true>(p, s) : go<P_I8, 1, true>(p, s);
  return two ? go<P_I8, 2, false>(p, s) : go<P_I8, 1, false>(p, s);
}

}  // namespace mxq
