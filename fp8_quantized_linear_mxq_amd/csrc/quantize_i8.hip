// Row-wise symmetric int8 quantization: one fp32 scale per row (an activation
// token, or a weight's output channel).
//
//   r = x, or x H_bd (block-diagonal Hadamard, as in quantize.hip)
//   s = RN_fp32(max_k |r_k| / 127),  q_k = clamp(RNE(r_k / s), -127, 127)
//
// decided on the exact real quotient like every other format (s = 0 gives
// q = 0).  The quotient is formed as t = r * (1 / s): both roundings move it
// by less than 2**-16, so q = RNE(t) is RNE(r / s) unless t lies that close to
// a half-integer.  A lane keeps its smallest distance to one, and only lanes
// inside the window (one in 2000) look at the remainder r - q s: near a tie it
// is exact in fp32 (a multiple of the smaller of r's and s's last places, and
// at most about s / 2), so comparing it with s / 2 decides.  Deciding there by
// float64 quotients instead cost a fifth of the kernel: 25% of the waves hold
// such a lane.  Scales below 2**-120, whose reciprocal nears overflow, take
// float64 quotients (r / s is 2**-25 away from a half-integer at least, or is one).
//
// Bound by memory: 2 (bf16) or 4 (fp32) bytes read and one written per
// element.  A row is held in registers between the amax and the encoding, so
// x is read once (rows of up to 32768 columns, 16384 rotated; longer rows are
// read twice).  A lane takes 8 consecutive elements at a time, so a wave's load
// is one contiguous kilobyte of bf16; a row belongs to one wave up to 2048
// columns, else to the four waves of a workgroup.  16384 x 4608 bf16: 41 us, 5.5
// TB/s (a plain copy of a gigabyte runs at 5.2), with the 16-point rotation 56
// us (float64 butterflies); 4096 x 4096 fp32 14 us.
#include "device_common.h"
#include "kernels.h"
#include "rows8.h"

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

template <int DT>
__device__ __forceinline__ Raw<DT> load8(const I8Params& p, int64_t row, int col) {
  return mxq::load8<DT>(p.x, row * p.ldx, col, p.cols);
}

// 8 codes of a row of DT values with scale s (inv = 1 / s, usable when `fast`).
template <int DT>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float s, float inv, bool fast) {
  // t + 1.5 * 2**23 rounds t to the nearest integer, ties to even, and holds
  // its two's complement in the low mantissa bits
  constexpr float kMagic = 12582912.0f;
  uint32_t u[8];
  float near = 1.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // a NaN keeps its payload, whose low byte may be -128: it is made -127, below
    // which no other value lies (bf16 NaNs have no such bits)
    const float t = DT == DT_F32 ? fmaxf(f[e] * inv, -127.0f) : f[e] * inv;
    const float a = t + kMagic;
    u[e] = __float_as_uint(a);
    near = fminf(near, fabsf(fabsf(t - (a - kMagic)) - 0.5f));
  }
  if (!fast) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double q = s == 0.f ? 0.0 : rint((double)f[e] / (double)s);
      u[e] = (uint32_t)(int)fmin(127.0, fmax(-127.0, q));
    }
  } else if (near < 0x1p-15f) {
    const float h = 0.5f * s;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = __builtin_fmaf(-(__uint_as_float(u[e]) - kMagic), s, f[e]);
      const bool past = fabsf(r) > h || (fabsf(r) == h && (u[e] & 1u));
      u[e] += past ? (r > 0.f ? 1u : ~0u) : 0u;
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

// J 8-element pieces per lane held in registers, WPR waves per row; J = 0
// reads rows of any length twice instead.
template <int DT, int HAD, int J, int WPR>
__global__ __launch_bounds__(kThreads) void quantize_i8_kernel(I8Params p) {
  constexpr int RPB = kThreads / 64 / WPR;   // rows per workgroup
  constexpr int STEP = WPR * 64 * 8;         // columns per piece of the row's waves
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = (int64_t)block_index() * RPB + wave / WPR;
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
      if constexpr (HAD > 0) in[j] = load8<DT>(p, row, c0 + j * STEP);
      else raw[j] = load8<DT>(p, row, c0 + j * STEP);
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
      float f[8];
      unpack8<DT>(load8<DT>(p, row, c), f);
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
      if (c < p.cols) *reinterpret_cast<uint2*>(out + c) = encode8<DT>(f, s, inv, fast);
    }
  } else {
    for (int c = c0; c - lane * 8 < p.cols; c += STEP) {
      float f[8];
      unpack8<DT>(load8<DT>(p, row, c), f);
      if constexpr (HAD > 0) hadamard8<HAD>(f, lane);
      if (c < p.cols) *reinterpret_cast<uint2*>(out + c) = encode8<DT>(f, s, inv, fast);
    }
  }
}

template <int DT, int HAD, int J, int WPR>
hipError_t go(const I8Params& p, hipStream_t s) {
  constexpr int RPB = kThreads / 64 / WPR;
  quantize_i8_kernel<DT, HAD, J, WPR><<<grid_of((p.rows + RPB - 1) / RPB), kThreads, 0, s>>>(p);
  return hipGetLastError();
}

template <int DT, int HAD, int WPR>
hipError_t by_pieces(const I8Params& p, hipStream_t s) {
  const int j = (p.cols + WPR * 512 - 1) / (WPR * 512);
  if (j <= 1) return go<DT, HAD, 1, WPR>(p, s);
  if (j <= 2) return go<DT, HAD, 2, WPR>(p, s);
  if (j <= 3) return go<DT, HAD, 3, WPR>(p, s);
  if (j <= 4) return go<DT, HAD, 4, WPR>(p, s);
  if constexpr (WPR > 1) {
    if (j <= 6) return go<DT, HAD, 6, WPR>(p, s);
    if (j <= 8) return go<DT, HAD, 8, WPR>(p, s);
    if constexpr (HAD == 0) {   // rotated rows are held as fp32 values: no registers for more
      if (j <= 12) return go<DT, HAD, 12, WPR>(p, s);
      if (j <= 16) return go<DT, HAD, 16, WPR>(p, s);
    }
    return go<DT, HAD, 0, WPR>(p, s);
  }
  return hipErrorInvalidValue;   // not reached: one wave takes up to 2048 columns
}

template <int DT, int HAD>
hipError_t by_rows(const I8Params& p, hipStream_t s) {
  // narrow rows leave most of four waves idle (bf16 4096 x 1152 5.8 us with one
  // wave per row, 10.3 with four), wide ones too few waves per compute unit
  // (2048 x 4096 10.4 / 7.7)
  if (p.cols <= 2048) return by_pieces<DT, HAD, 1>(p, s);
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
