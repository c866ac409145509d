// Products with few rows of activations (single tokens, small batches; in a
// product grouped by expert, few rows per group): INT8 x INT8, and grouped by
// expert also MXFP4 x MXFP4 and bf16 x MXFP4.
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

// NT weight tiles and RT activation tiles of 16 rows per workgroup.
template <int P, int NT, int RT, bool GRP>
__global__ __launch_bounds__(64 * kWaves) void gemm_few_kernel(GemmP p) {
  using Acc = std::conditional_t<P == P_I8, v4i, v4f>;
  constexpr int S = 2 * kPairs;                      // steps per round
  constexpr int AV = P == P_BF4 ? 4 : 1;             // 16-byte pieces of a per step
  __shared__ Acc part[kWaves][NT * RT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r16 = lane & 15, q = lane >> 4;
  const int tn = blockIdx.x % p.tiles_n, tm = blockIdx.x / p.tiles_n;
  int m0 = tm * 16 * RT;
  if constexpr (GRP) {
    m0 = enter_group(p, 16 * RT, tm);
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
  const uint8_t* arow[RT];
  const uint8_t* ascl[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t m = min(m0 + i * 16 + r16, p.M - 1);
    arow[i] = p.a + m * p.lda + (P == P_BF4 ? 64 : 16) * q;
    ascl[i] = p.as + m * p.ldas;
  }

  Acc acc[NT][RT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[j][i] = Acc{};

  for (int s0 = 2 * wave; s0 < steps; s0 += 2 * kPairs * kWaves) {
    v4i wf[S][NT], af[S][RT][AV];
    uint32_t wd[S][NT], ad[S][RT];
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
      for (int i = 0; i < RT; ++i) {
#pragma unroll
        for (int v = 0; v < AV; ++v) {
          af[t][i][v] = v4i{};
          if (in) af[t][i][v] = *reinterpret_cast<const v4i*>(arow[i] + (P == P_BF4 ? 256 : 64) * s + 16 * v);
        }
        if constexpr (P == P_MX4) {
          ad[t][i] = 0;
          if (in) ad[t][i] = *reinterpret_cast<const uint32_t*>(ascl[i] + 4 * s);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < S; ++t) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (P == P_I8) {
#pragma unroll
          for (int i = 0; i < RT; ++i)
            acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[t][j], af[t][i][0], acc[j][i], 0, 0, 0);
        } else if constexpr (P == P_MX4) {
          const v4i& w4 = wf[t][j];
          const v8i wv = __builtin_shufflevector(w4, w4, 0, 1, 2, 3, -1, -1, -1, -1);
          const int sw = (int)(wd[t][j] >> (8 * q));
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const v4i& a4 = af[t][i][0];
            const v8i av = __builtin_shufflevector(a4, a4, 0, 1, 2, 3, -1, -1, -1, -1);
            acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                wv, av, acc[j][i], 4, 4, 0, sw, 0, (int)(ad[t][i] >> (8 * q)));
          }
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
#pragma unroll
            for (int i = 0; i < RT; ++i)
              acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  wv, __builtin_bit_cast(v8bf, af[t][i][v]), acc[j][i], 0, 0, 0);
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < RT; ++i) part[wave][j * RT + i][lane] = acc[j][i];
  __syncthreads();

  // lane l of a tile holds activation row l % 16 and weight rows 4 (l / 16) + [0, 4)
  for (int idx = threadIdx.x; idx < NT * RT * 64; idx += 64 * kWaves) {
    const int tile = idx >> 6, l = idx & 63;
    Acc sum = part[0][tile][l];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += part[w][tile][l];
    const int m = m0 + (tile % RT) * 16 + (l & 15);
    const int n = n0 + (tile / RT) * 16 + 4 * (l >> 4);
    if (m >= p.M) continue;
    uint16_t* orow = p.out + (int64_t)m * p.ld_out;
    float sa = 0.f;
    if constexpr (P == P_I8) sa = *reinterpret_cast<const float*>(p.as + (int64_t)m * p.ldas);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e >= p.N) break;
      const int c = p.col_map ? p.col_map[n + e] : n + e;
      if (c < 0 || c >= p.n_out) continue;
      float v;
      if constexpr (P == P_I8) {
        const float sw = *reinterpret_cast<const float*>(p.ws + (int64_t)(n + e) * p.ldws);
        v = ((float)sum[e] * sa) * sw;
        if constexpr (!GRP) {
          const float* u = p.u + (int64_t)m * p.ld_u;
          const uint16_t* l2 = p.l2t + (int64_t)c * p.rank;
          for (int r = 0; r < p.rank; ++r) v = fmaf(u[r], bf16_bits_to_f32(l2[r]), v);
        }
      } else {
        v = P == P_BF4 ? sum[e] * 0.25f : sum[e];
      }
      if (p.bias) v += bf16_bits_to_f32(p.bias[c]);
      orow[c] = (uint16_t)f32_to_bf16_bits(v);
    }
  }
}

template <int P, int NT, int RT, bool GRP>
hipError_t go(GemmP p, hipStream_t s) {
  p.tiles_m = GRP ? (int)group_tiles_bound(p.M, p.groups, 16 * RT) : (p.M + 16 * RT - 1) / (16 * RT);
  p.tiles_n = (p.N + 16 * NT - 1) / (16 * NT);
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  gemm_few_kernel<P, NT, RT, GRP><<<(unsigned)tiles, 64 * kWaves, 0, s>>>(p);
  return hipGetLastError();
}

template <int P, int NT>
hipError_t by_rows(const GemmP& p, hipStream_t s) {
  if ((int64_t)p.M <= (int64_t)16 * p.groups) return go<P, NT, 1, true>(p, s);
  return go<P, NT, 2, true>(p, s);
}

}  // namespace

// Where this kernel is the faster one: up to 16 rows of a plain product (16 x
// 4096 x 4096 7.3 us against 8.9 with 64 x 64 tiles; 32 rows 9.2 against 8.8),
// up to 32 on average per group.
bool few_rows(const GemmArgs& a) {
  if (!a.goff) return a.M <= 16;
  return a.M <= 32 * a.groups;
}

hipError_t launch_gemm_few(const GemmArgs& a, hipStream_t s) {
  const GemmP p = gemm_params(a);
  if (!a.goff) return go<P_I8, 1, 1, false>(p, s);
  if (a.a_fmt == FMT_INT8) return by_rows<P_I8, 1>(p, s);
  if (a.a_fmt == FMT_MXFP4) return by_rows<P_MX4, 1>(p, s);
  return by_rows<P_BF4, 2>(p, s);
}

}  // namespace mxq
