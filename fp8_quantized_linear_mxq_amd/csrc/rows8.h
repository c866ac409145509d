// Rows taken 8 consecutive elements to a lane: loads, the block Hadamard rotation
// and the largest magnitude, shared by the quantizes whose scales cover whole rows
// or runs of 128.
#pragma once

#include "device_common.h"

#include <type_traits>

namespace mxq {

// A lane's 8 consecutive values as loaded: two fp32 quads, or one quad of
// packed bf16 pairs.
template <int DT> struct Raw { uint4 lo, hi; };
template <> struct Raw<DT_BF16> { uint4 lo; };

// Elements col .. col + 7 of the row that begins at element `first`; zeros past the row's end.
template <int DT>
__device__ __forceinline__ Raw<DT> load8(const void* x, int64_t first, int col, int cols) {
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  if constexpr (DT == DT_BF16) {
    if (col < cols) lo = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + first + col);
    return {lo};
  } else {
    if (col < cols) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(x) + first + col);
      lo = q[0];
      hi = q[1];
    }
    return {lo, hi};
  }
}

template <int DT>
__device__ __forceinline__ void unpack8(const Raw<DT>& r, float (&f)[8]) {
  if constexpr (DT == DT_BF16) {
    const uint32_t d[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(d[i] << 16);
      f[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
  } else {
    const uint32_t d[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(d[i]);
  }
}

// n-point block Hadamard of a lane's 8 values and its neighbours': distances
// 1, 2, 4 in registers, 8 .. n/2 across lanes (lane distance 1 .. n/16); sums
// exact in float64, r = RN_fp32(RN_fp64(c_n S)), a zero sum is +0.
template <int HAD>
__device__ __forceinline__ void hadamard8(float (&f)[8], int lane) {
  double h[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] = (double)f[e];
#pragma unroll
  for (int d = 1; d < 8; d <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e & d) continue;
      const double a = h[e], b = h[e + d];
      h[e] = a + b;
      h[e + d] = a - b;
    }
  auto across = [&](auto m) __attribute__((always_inline)) {
    constexpr int M = decltype(m)::value;
    const bool upper = (lane & M) != 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double o = xor_lane_d<M>(h[e]);
      h[e] = upper ? (o - h[e]) : (h[e] + o);
    }
  };
  if constexpr (HAD >= 16) across(std::integral_constant<int, 1>{});
  if constexpr (HAD >= 32) across(std::integral_constant<int, 2>{});
  if constexpr (HAD >= 128) {
    across(std::integral_constant<int, 4>{});
    across(std::integral_constant<int, 8>{});
  }
  // float64 nearest to 1/sqrt(n): 1/4, sqrt(2)/8, sqrt(2)/16
  constexpr double c = HAD == 16 ? 0.25 : HAD == 32 ? 0x1.6a09e667f3bcdp-3 : 0x1.6a09e667f3bcdp-4;
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = (float)(c * (h[e] + 0.0));
}

__device__ __forceinline__ float amax8(const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(f[e]));
  return m;
}

template <int N>
__device__ __forceinline__ void flag_nonfinite(const float (&f)[N], unsigned* dbg) {
  if (!dbg) return;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < N; ++e) bad |= !__builtin_isfinite(f[e]);
  if (bad) atomicOr(dbg, 1u);
}

}  // namespace mxq
