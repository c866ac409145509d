// RMS norm of every query and key head with the position rotation, one pass:
//   n = v / sqrt(mean(v^2) + eps) * g,  (a, b) -> (a c - b s, b c + a s)
// for the pairs (i, i + R/2) or (2i, 2i + 1), i < R/2, with c, s the cosine
// and sine of the token's position; elements R .. D-1 are normalised only.
// Everything in fp32 from the loaded values, one rounding at the end.
//
// Bound by memory (every head read and written once).  A head is cut into
// units of 8 elements that hold whole pairs -- 4 elements of the first half
// and their 4 partners of the second, or 8 neighbours -- so the rotation stays
// inside a lane and only the sum of squares crosses lanes.  LPH lanes (the
// power of two at or above D / 8) take a head, a wave 64 / LPH heads of one
// token at a time, kHeads times, with all loads issued first; the token's
// cosines and sines and both gains stay in registers meanwhile.
//
// 16384 tokens x (32 + 8) heads x 128 in bf16: 69 us, 5.0 TB/s (a plain copy of a
// gigabyte runs at 5.2): one wave per workgroup (256 threads 75 us), streaming
// stores (cached ones 75 us: a sequence's heads are more than the L2s hold),
// four heads per lane (two 74 us, eight 94 us).  72-wide heads use 9 of 16
// lanes: 16384 x 32 heads 43 us, 3.6 TB/s (seven heads packed into a wave, with
// the sum by lane shifts: 41 us, not kept).
#include "device_common.h"
#include "gemm_pipe.h"
#include "kernels.h"

namespace mxq {
namespace {

constexpr int kThreads = 64;   // one wave: no wave waits for another
constexpr int kHeads = 4;   // heads per lane

struct QkParams {
  QkNormArgs a;
  int chunks;   // groups of heads per token
};

// 4 consecutive elements.
template <int DT>
__device__ __forceinline__ void load4(const void* p, int64_t i, float (&f)[4]) {
  if constexpr (DT == DT_BF16) {
    const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xFFFF0000u);
  } else {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
}

template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t i, const float (&f)[4]) {
  if constexpr (DT == DT_BF16) {
    typedef unsigned int v2u __attribute__((ext_vector_type(2)));
    const v2u v = {pack_bf16_rne(f[0], f[1]), pack_bf16_rne(f[2], f[3])};
    __builtin_nontemporal_store(v, reinterpret_cast<v2u*>(static_cast<uint16_t*>(p) + i));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

// 8 consecutive bf16 elements in one access.
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&f)[2][4]) {
  const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[e >> 1][2 * (e & 1)] = __uint_as_float(d[e] << 16);
    f[e >> 1][2 * (e & 1) + 1] = __uint_as_float(d[e] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void store8(void* p, int64_t i, const float (&f)[2][4]) {
  const v4u v = {pack_bf16_rne(f[0][0], f[0][1]), pack_bf16_rne(f[0][2], f[0][3]),
                 pack_bf16_rne(f[1][0], f[1][1]), pack_bf16_rne(f[1][2], f[1][3])};
  __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(static_cast<uint16_t*>(p) + i));
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
  if constexpr (LPH >= 2) v += xor_lane_f<1>(v);
  if constexpr (LPH >= 4) v += xor_lane_f<2>(v);
  if constexpr (LPH >= 8) v += xor_lane_f<4>(v);
  if constexpr (LPH >= 16) v += xor_lane_f<8>(v);
  if constexpr (LPH >= 32) v += xor_lane_f<16>(v);
  if constexpr (LPH >= 64) v += xor_lane_f<32>(v);
  return v;
}

template <int DT, bool INTER, int LPH>
__global__ __launch_bounds__(kThreads) void qk_norm_kernel(QkParams p) {
  const QkNormArgs& a = p.a;
  constexpr int HPW = 64 / LPH;   // heads of a wave at a time
  const int lane = threadIdx.x & 63;
  const int64_t task = (int64_t)block_index() * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t tok = task / p.chunks;
  if (tok >= a.tokens) return;   // whole waves leave
  const int h0 = (int)(task - tok * p.chunks) * HPW * kHeads + lane / LPH;
  const int u = lane % LPH;                       // unit of the head
  const int D = a.head_dim, heads = a.n_q + a.n_k;
  const bool act = 8 * u < D, rot = 8 * u < a.rot_dim;
  const int lo = !INTER && rot ? 4 * u : 8 * u;
  const int hi = !INTER && rot ? a.rot_dim / 2 + 4 * u : 8 * u + 4;

  float x[kHeads][2][4];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i * HPW;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[i][0][e] = x[i][1][e] = 0.f;
    if (act && h < heads) {
      const int64_t at = tok * a.ldx + (int64_t)h * D;
      if constexpr (INTER && DT == DT_BF16) {
        load8(a.x, at + lo, x[i]);
      } else {
        load4<DT>(a.x, at + lo, x[i][0]);
        load4<DT>(a.x, at + hi, x[i][1]);
      }
    }
  }
  float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.rot_dim > 0) {
    const int64_t pos = a.pos ? (int64_t)a.pos[tok] : tok;
    if (pos < 0 || pos >= a.n_pos) return;   // whole waves leave: the token is skipped
    if (rot) {
      load4<DT_F32>(a.cos, pos * (a.rot_dim / 2) + 4 * u, c);
      load4<DT_F32>(a.sin, pos * (a.rot_dim / 2) + 4 * u, s);
    }
  }
  float gq[2][4], gk[2][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) gq[0][e] = gq[1][e] = gk[0][e] = gk[1][e] = 1.f;
  if (act && a.wq) {
    load4<DT>(a.wq, lo, gq[0]);
    load4<DT>(a.wq, hi, gq[1]);
  }
  if (act && a.wk) {
    load4<DT>(a.wk, lo, gk[0]);
    load4<DT>(a.wk, hi, gk[1]);
  }
  const float inv_d = 1.0f / (float)D;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i * HPW;
    float sq = 0.f;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) sq = fmaf(x[i][b][e], x[i][b][e], sq);
    const float r = 1.0f / sqrtf(head_sum<LPH>(sq) * inv_d + a.eps);
    const bool is_q = h < a.n_q;
    float n[2][4], o[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) n[b][e] = x[i][b][e] * r * (is_q ? gq[b][e] : gk[b][e]);
    if constexpr (INTER) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float y = n[b][2 * e], z = n[b][2 * e + 1], cc = c[2 * b + e], ss = s[2 * b + e];
          o[b][2 * e] = y * cc - z * ss;
          o[b][2 * e + 1] = z * cc + y * ss;
        }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // a unit past the rotated part has c = 1, s = 0: it passes unchanged
        o[0][e] = n[0][e] * c[e] - n[1][e] * s[e];
        o[1][e] = n[1][e] * c[e] + n[0][e] * s[e];
      }
    }
    if (act && h < heads) {
      void* out = is_q ? a.q : a.k;
      const int64_t at = is_q ? tok * a.q_token + (int64_t)h * a.q_head
                              : tok * a.k_token + (int64_t)(h - a.n_q) * a.k_head;
      if constexpr (INTER && DT == DT_BF16) {
        store8(out, at + lo, o);
      } else {
        store4<DT>(out, at + lo, o[0]);
        store4<DT>(out, at + hi, o[1]);
      }
    }
  }
}

template <int DT, bool INTER, int LPH>
hipError_t go(QkParams p, hipStream_t s) {
  constexpr int PER = 64 / LPH * kHeads;   // heads per wave
  p.chunks = (p.a.n_q + p.a.n_k + PER - 1) / PER;
  const int64_t waves = p.a.tokens * p.chunks, blocks = (waves + kThreads / 64 - 1) / (kThreads / 64);
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  qk_norm_kernel<DT, INTER, LPH><<<grid_of(blocks), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

template <int DT, bool INTER>
hipError_t by_head(const QkParams& p, hipStream_t s) {
  const int units = p.a.head_dim / 8;
  if (units <= 8) return go<DT, INTER, 8>(p, s);
  if (units <= 16) return go<DT, INTER, 16>(p, s);
  if (units <= 32) return go<DT, INTER, 32>(p, s);
  return go<DT, INTER, 64>(p, s);
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormArgs& a, hipStream_t s) {
  const QkParams p{a, 0};
  if (a.dtype == DT_BF16) return a.interleaved ? by_head<DT_BF16, true>(p, s) : by_head<DT_BF16, false>(p, s);
  return a.interleaved ? by_head<DT_F32, true>(p, s) : by_head<DT_F32, false>(p, s);
}

}  // namespace mxq
