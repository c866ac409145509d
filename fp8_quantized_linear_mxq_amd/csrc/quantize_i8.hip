// Row-wise symmetric int8 quantization: one fp32 scale per row (an activation
// token, or a weight's output channel).
//
//   r = x, or x H_bd (block-diagonal Hadamard, as in quantize.hip)
//   s = RN_fp32(max_k |r_k| / 127),  q_k = clamp(RNE(r_k / s), -127, 127)
//
// decided on the exact real quotient like every other format (s = 0 gives
// q = 0).  The quotient is formed as t = r * (1 / s): both roundings move it
// by less than 2**-16, so RNE(t) is RNE(r / s) unless t lies that close to a
// half-integer.  A lane keeps its smallest distance to one, and only lanes
// inside the window (a few in 10000) redo their values with the float64
// quotient, which is exact enough to decide every case (r / s differs from a
// half-integer by 2**-25 at least, or is one).
//
// Bound by memory: 2 (bf16) or 4 (fp32) bytes read and one written per
// element.  A row is held in registers between the amax and the encoding, so
// x is read once (rows of up to 16384 columns; longer rows are read twice).
// A lane takes 8 consecutive elements at a time, so a wave's load is one
// contiguous kilobyte of bf16; a row belongs to one wave when there are rows
// enough to fill the GPU, else to the four waves of a workgroup.
#include "device_common.h"
#include "kernels.h"

namespace mxq {
namespace {

constexpr int kThreads = 256;

struct I8Params {
  const void* x;
  int64_t rows, ldx;
  int cols;
  int8_t* codes;
  int64_t ld_codes;
  uint8_t* scales;
  int64_t ld_scales;   // bytes
  unsigned* dbg;
};

// A lane's 8 consecutive values as loaded (bf16 pairs stay packed).
template <int DT> struct Raw { uint4 v[DT == DT_F32 ? 2 : 1]; };

template <int DT>
__device__ __forceinline__ void load8(const I8Params& p, int64_t row, int col, Raw<DT>& r) {
  const bool act = col < p.cols;
  if constexpr (DT == DT_BF16) {
    r.v[0] = make_uint4(0, 0, 0, 0);
    if (act) r.v[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + row * p.ldx + col);
  } else {
    r.v[0] = r.v[1] = make_uint4(0, 0, 0, 0);
    if (act) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p.x) + row * p.ldx + col);
      r.v[0] = q[0];
      r.v[1] = q[1];
    }
  }
}

template <int DT>
__device__ __forceinline__ void unpack8(const Raw<DT>& r, float (&f)[8]) {
  if constexpr (DT == DT_BF16) {
    const uint32_t d[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(d[i] << 16);
      f[2 * i + 1] = __uint_as_float(d[i] & 0xFFFF0000u);
    }
  } else {
    const uint32_t d[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w,
                           r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
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

// 8 codes of a row with scale s (inv = 1 / s, usable when `fast`).
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float s, float inv, bool fast) {
  // t + 1.5 * 2**23 rounds t to the nearest integer, ties to even, and holds
  // its two's complement in the low mantissa bits
  constexpr float kMagic = 12582912.0f;
  uint32_t u[8];
  float near = 1.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = f[e] * inv;
    const float a = t + kMagic;
    u[e] = __float_as_uint(a);
    near = fminf(near, fabsf(fabsf(t - (a - kMagic)) - 0.5f));
  }
  if (!fast || near < 0x1p-15f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double q = s == 0.f ? 0.0 : rint((double)f[e] / (double)s);
      u[e] = (uint32_t)(int)fmin(127.0, fmax(-127.0, q));
    }
  }
  // low bytes of four words into one
  auto pack = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
    return lo | hi;
  };
  return make_uint2(pack(u[0], u[1], u[2], u[3]), pack(u[4], u[5], u[6], u[7]));
}

template <int N>
__device__ __forceinline__ void flag_nonfinite(const float (&f)[N], unsigned* dbg) {
  if (!dbg) return;
  bool bad = false;
#pragma unroll
  for (int e = 0; e < N; ++e) bad |= !__builtin_isfinite(f[e]);
  if (bad) atomicOr(dbg, 1u);
}

// J 8-element pieces per lane held in registers, WPR waves per row; J = 0
// reads rows of any length twice instead.
template <int DT, int HAD, int J, int WPR>
__global__ __launch_bounds__(kThreads) void quantize_i8_kernel(I8Params p) {
  constexpr int RPB = kThreads / 64 / WPR;   // rows per workgroup
  constexpr int STEP = WPR * 64 * 8;         // columns per piece of the row's waves
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = (int64_t)blockIdx.x * RPB + wave / WPR;
  const bool live = row0 < p.rows;
  const int64_t row = live ? row0 : p.rows - 1;
  const int c0 = ((wave % WPR) * 64 + lane) * 8;

  // without a rotation the loaded words are kept, with one the rotated values
  Raw<DT> raw[J > 0 && HAD == 0 ? J : 1];
  float rot[J > 0 && HAD > 0 ? J : 1][8];
  float m = 0.f;
  if constexpr (J > 0) {
    Raw<DT> in[HAD > 0 ? J : 1];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if constexpr (HAD > 0) load8<DT>(p, row, c0 + j * STEP, in[j]);
      else load8<DT>(p, row, c0 + j * STEP, raw[j]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float f[8];
      if constexpr (HAD > 0) {
        unpack8<DT>(in[j], rot[j]);
        flag_nonfinite(rot[j], p.dbg);
        hadamard8<HAD>(rot[j], lane);
        m = fmaxf(m, amax8(rot[j]));
      } else {
        unpack8<DT>(raw[j], f);
        flag_nonfinite(f, p.dbg);
        m = fmaxf(m, amax8(f));
      }
    }
  } else {
    for (int c = c0; c - lane * 8 < p.cols; c += STEP) {   // whole waves stay in the loop
      Raw<DT> r;
      float f[8];
      load8<DT>(p, row, c, r);
      unpack8<DT>(r, f);
      flag_nonfinite(f, p.dbg);
      if constexpr (HAD > 0) hadamard8<HAD>(f, lane);
      m = fmaxf(m, amax8(f));
    }
  }
  m = group_max<64>(m);
  if constexpr (WPR > 1) {
    __shared__ float red[kThreads / 64];
    if (lane == 0) red[wave] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < WPR; ++w) m = fmaxf(m, red[w]);
  }
  const float s = (float)((double)m / 127.0);
  // below 2**-120 the reciprocal nears overflow: take the float64 quotients
  const bool fast = s == 0.f || s >= 0x1p-120f;
  const float inv = s == 0.f ? 0.f : 1.0f / s;
  if (!live) return;
  if (c0 == 0) *reinterpret_cast<float*>(p.scales + row * p.ld_scales) = s;
  int8_t* out = p.codes + row * p.ld_codes;
  if constexpr (J > 0) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = c0 + j * STEP;
      float f[8];
      if constexpr (HAD > 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = rot[j][e];
      } else {
        unpack8<DT>(raw[j], f);
      }
      if (c < p.cols) *reinterpret_cast<uint2*>(out + c) = encode8(f, s, inv, fast);
    }
  } else {
    for (int c = c0; c - lane * 8 < p.cols; c += STEP) {
      Raw<DT> r;
      float f[8];
      load8<DT>(p, row, c, r);
      unpack8<DT>(r, f);
      if constexpr (HAD > 0) hadamard8<HAD>(f, lane);
      if (c < p.cols) *reinterpret_cast<uint2*>(out + c) = encode8(f, s, inv, fast);
    }
  }
}

template <int DT, int HAD, int J, int WPR>
hipError_t go(const I8Params& p, hipStream_t s) {
  constexpr int RPB = kThreads / 64 / WPR;
  quantize_i8_kernel<DT, HAD, J, WPR><<<(unsigned)((p.rows + RPB - 1) / RPB), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

template <int DT, int HAD, int WPR>
hipError_t by_pieces(const I8Params& p, hipStream_t s) {
  const int j = (p.cols + WPR * 512 - 1) / (WPR * 512);
  if (j <= 1) return go<DT, HAD, 1, WPR>(p, s);
  if (j <= 2) return go<DT, HAD, 2, WPR>(p, s);
  if (j <= 3) return go<DT, HAD, 3, WPR>(p, s);
  if (j <= 4) return go<DT, HAD, 4, WPR>(p, s);
  if (j <= 6) return go<DT, HAD, 6, WPR>(p, s);
  if (j <= 8) return go<DT, HAD, 8, WPR>(p, s);
  if constexpr (WPR == 4) return go<DT, HAD, 0, WPR>(p, s);
  return hipErrorInvalidValue;
}

template <int DT, int HAD>
hipError_t by_rows(const I8Params& p, hipStream_t s) {
  // a wave per row needs rows for every compute unit's waves
  if (p.rows >= 2048 && p.cols <= 4096) return by_pieces<DT, HAD, 1>(p, s);
  return by_pieces<DT, HAD, 4>(p, s);
}

template <int DT>
hipError_t by_rotation(const I8Params& p, int had, hipStream_t s) {
  switch (had) {
    case 0: return by_rows<DT, 0>(p, s);
    case 16: return by_rows<DT, 16>(p, s);
    case 32: return by_rows<DT, 32>(p, s);
    default: return by_rows<DT, 128>(p, s);
  }
}

}  // namespace

hipError_t launch_quantize_i8(const QuantizeArgs& a, hipStream_t s) {
  I8Params p;
  p.x = a.x;
  p.rows = a.rows;
  p.ldx = a.ldx;
  p.cols = (int)a.cols;
  p.codes = reinterpret_cast<int8_t*>(a.codes);
  p.ld_codes = a.ld_codes;
  p.scales = a.scales;
  p.ld_scales = a.ld_scales;
  p.dbg = a.dbg;
  const hipError_t e = a.dtype == DT_BF16 ? by_rotation<DT_BF16>(p, a.hadamard_n, s)
                                          : by_rotation<DT_F32>(p, a.hadamard_n, s);
  if (e != hipSuccess || !a.lr) return e;
  return launch_lora_down(*a.lr, s);
}

}  // namespace mxq
