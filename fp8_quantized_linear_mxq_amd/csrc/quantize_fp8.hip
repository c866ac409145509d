// E4M3 quantization with one fp32 scale per block of 128 columns: of one row
// (FP8, activations) or of 128 rows (FP8_TILE, weights).
//
//   r = x, or x H_bd (block-diagonal Hadamard, as in quantize.hip)
//   s = RN_fp32(max over the block |r| / 448),  q = RNE_E4M3(r / s)
//
// decided on the exact real quotient (s = 0 gives zeros).  The quotient is formed
// as t = r * (1 / s), which the hardware's reciprocal (one unit) and the product move
// by at most 3 units of its last place, and converted by the hardware.  A code can only be wrong where t
// lies within 4 units of the middle between two codes (bits 0x80000 below the
// three that E4M3 keeps) or is subnormal in E4M3 (below 2**-6, where the middles
// lie elsewhere); a lane that holds such an element compares it with the middle
// exactly: fma(-middle, s, r) has the sign of r / s - middle.  bf16 inputs tie
// often (both mantissas are short), so this path costs no float64.  Scales below
// 2**-100, where the remainder could underflow, take float64 quotients.
//
// Bound by memory: 2 (bf16) or 4 (fp32) bytes read and one written per element; a
// block is held in registers between its maximum and its codes.  A lane takes 8
// consecutive elements, 16 lanes a row's block.
#include "device_common.h"
#include "kernels.h"
#include "rows8.h"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32;   // rows of a workgroup of the row-wise format: 8 per wave

struct Fp8Params {
  const void* x;
  int64_t rows, ldx;
  int cols, col_groups;
  uint8_t* codes;
  int64_t ld_codes;
  uint8_t* scales;
  int64_t ld_scales;   // bytes between K-blocks (FP8) or row blocks (FP8_TILE)
  unsigned* dbg;
};

// Codes of two values.
__device__ __forceinline__ uint32_t cvt2(float a, float b) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}

// t, whose true value is f / s, moved off the middle between two codes to the side
// that f / s lies on.
__device__ __forceinline__ float settle(float t, float f, float s) {
  const uint32_t b = __float_as_uint(t);
  const float a = fabsf(t), m = fabsf(f);
  if (a >= 0x1p-6f) {
    if (((b - 0x7FFFCu) & 0xFFFFFu) > 8u) return t;
    const uint32_t mid = (b & ~0xFFFFFu) | 0x80000u;
    const float r = __builtin_fmaf(-fabsf(__uint_as_float(mid)), s, m);
    return __uint_as_float(r > 0.f ? mid + 1u : r < 0.f ? mid - 1u : mid);
  }
  // subnormal codes: multiples of 2**-9, 2**-6 among them
  const float fl = floorf(a * 512.f), mid = (fl + 0.5f) * 0x1p-9f;
  const float r = __builtin_fmaf(-mid, s, m);
  const bool up = r > 0.f || (r == 0.f && ((int)fl & 1));
  return copysignf((fl + (up ? 1.f : 0.f)) * 0x1p-9f, t);
}

// 8 codes of values with scale s (inv = 1 / s, usable when `fast`).
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float s, float inv, bool fast) {
  float t[8];
  uint32_t mid = ~0u, low = ~0u;   // smallest distance to a middle, smallest nonzero magnitude
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t[e] = f[e] * inv;
    const uint32_t b = __float_as_uint(t[e]);
    mid = min(mid, (b - 0x7FFFCu) & 0xFFFFFu);
    low = min(low, (b & 0x7FFFFFFFu) - 1u);
  }
  uint32_t c[4];
  if (!fast) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t q[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float v = f[2 * e + k];
        q[k] = s == 0.f ? 0u : e4m3_encode_f64(fabs((double)v / (double)s));
        q[k] |= (__float_as_uint(v) >> 24) & 0x80u;
      }
      c[e] = q[0] | q[1] << 8;
    }
  } else {
    if (mid <= 8u || low < 0x3C7FFFFFu) {   // 2**-6 - 1 unit
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = settle(t[e], f[e], s);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = cvt2(t[2 * e], t[2 * e + 1]);
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// RN_fp32(amax / 448): the compiler's fp32 division is correctly rounded; quotients
// that are subnormal, where it may flush, take float64 (whose rounding to fp32 is
// right for a quotient of two fp32 values).
__device__ __forceinline__ float scale_of(float amax) {
  return amax >= 0x1p-100f ? amax / 448.0f : (float)((double)amax / 448.0);
}

// A workgroup takes 32 rows x 4 blocks: lane group l / 16 of a wave one block of
// the row, so a wave's load is one contiguous kilobyte of bf16, eight rows in
// flight.  The scales of a K-block lie together for all rows (the matrix product
// reads one per lane), so they leave through LDS as 128-byte runs.
template <int DT, int HAD>
__global__ __launch_bounds__(kThreads) void quantize_fp8_kernel(Fp8Params p) {
  constexpr int U = kRows / 4;
  __shared__ float sc[4][kRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t bid = block_index();
  const int64_t row0 = (int64_t)(bid / (uint32_t)p.col_groups) * kRows;
  const int c = (int)(bid % (uint32_t)p.col_groups) * 512 + lane * 8;
  if (row0 >= p.rows) return;
  const int live = (int)min((int64_t)kRows, p.rows - row0);
  Raw<DT> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u * 4 + wave < live) raw[u] = load8<DT>(p.x, (row0 + u * 4 + wave) * p.ldx, c, p.cols);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = u * 4 + wave;
    if (r >= live) continue;
    float f[8];
    unpack8<DT>(raw[u], f);
    flag_nonfinite(f, p.dbg);
    if constexpr (HAD > 0) hadamard8<HAD>(f, lane);
    const float s = scale_of(group_max<16>(amax8(f)));
    const bool fast = s >= 0x1p-100f;
    if ((lane & 15) == 0) sc[lane >> 4][r] = s;
    if (c < p.cols)
      *reinterpret_cast<uint2*>(p.codes + (row0 + r) * p.ld_codes + c) = encode8(f, s, fast ? __builtin_amdgcn_rcpf(s) : 0.f, fast);
  }
  __syncthreads();
  const int t = threadIdx.x, kb = t / kRows, r = t % kRows;
  const int64_t block = (int64_t)(bid % (uint32_t)p.col_groups) * 4 + kb;
  if (kb < 4 && r < live && block * 128 < p.cols)
    *reinterpret_cast<float*>(p.scales + block * p.ld_scales + (row0 + r) * 4) = sc[kb][r];
}

// A workgroup takes one tile of 128 x 128, 16 rows at a time.
template <int DT, int HAD>
__global__ __launch_bounds__(kThreads) void quantize_fp8_tile_kernel(Fp8Params p) {
  __shared__ float red[kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t bid = block_index();
  const uint32_t tr = bid / (uint32_t)p.col_groups, tc = bid % (uint32_t)p.col_groups;
  const int64_t row0 = (int64_t)tr * 128;
  if (row0 >= p.rows) return;
  const int c = (int)tc * 128 + (lane & 15) * 8;
  const int64_t r0 = row0 + wave * 4 + (lane >> 4);
  Raw<DT> raw[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) raw[u] = load8<DT>(p.x, min(r0 + 16 * u, p.rows - 1) * p.ldx, c, p.cols);
  float m = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {   // rows past the end repeat the last one
    float f[8];
    unpack8<DT>(raw[u], f);
    flag_nonfinite(f, p.dbg);
    if constexpr (HAD > 0) hadamard8<HAD>(f, lane);
    m = fmaxf(m, amax8(f));
  }
  m = group_max<64>(m);
  if (lane == 0) red[wave] = m;
  __syncthreads();
  const float s = scale_of(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
  if (threadIdx.x == 0) *reinterpret_cast<float*>(p.scales + (int64_t)tr * p.ld_scales + (int64_t)tc * 4) = s;
  const bool fast = s >= 0x1p-100f;
  const float inv = fast ? __builtin_amdgcn_rcpf(s) : 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float f[8];
    unpack8<DT>(raw[u], f);
    if constexpr (HAD > 0) hadamard8<HAD>(f, lane);
    const int64_t r = r0 + 16 * u;
    if (r < p.rows && c < p.cols)
      *reinterpret_cast<uint2*>(p.codes + r * p.ld_codes + c) = encode8(f, s, inv, fast);
  }
}

template <int DT, int HAD>
hipError_t go(Fp8Params p, bool tile, hipStream_t s) {
  if (tile) {
    p.col_groups = (p.cols + 127) / 128;
    quantize_fp8_tile_kernel<DT, HAD><<<grid_of((p.rows + 127) / 128 * p.col_groups), kThreads, 0, s>>>(p);
  } else {
    p.col_groups = (p.cols + 511) / 512;
    quantize_fp8_kernel<DT, HAD><<<grid_of((p.rows + kRows - 1) / kRows * p.col_groups), kThreads, 0, s>>>(p);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t by_rotation(const Fp8Params& p, int had, bool tile, hipStream_t s) {
  switch (had) {
    case 0: return go<DT, 0>(p, tile, s);
    case 16: return go<DT, 16>(p, tile, s);
    case 32: return go<DT, 32>(p, tile, s);
    default: return go<DT, 128>(p, tile, s);
  }
}

}  // namespace

hipError_t launch_quantize_fp8(const QuantizeArgs& a, hipStream_t s) {
  Fp8Params p;
  p.x = a.x;
  p.rows = a.rows;
  p.ldx = a.ldx;
  p.cols = (int)a.cols;
  p.col_groups = 0;
  p.codes = a.codes;
  p.ld_codes = a.ld_codes;
  p.scales = a.scales;
  p.ld_scales = a.ld_scales;
  p.dbg = a.dbg;
  const bool tile = a.fmt == FMT_FP8_TILE;
  return a.dtype == DT_BF16 ? by_rotation<DT_BF16>(p, a.hadamard_n, tile, s)
                            : by_rotation<DT_F32>(p, a.hadamard_n, tile, s);
}

}  // namespace mxq
