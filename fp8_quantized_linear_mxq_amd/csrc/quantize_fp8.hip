// E4M3 quantization with one fp32 scale per block of 128 columns: of one row
// (FP8, activations) or of 128 rows (FP8_TILE, weights).
//
//   r = x, or x H_bd (block-diagonal Hadamard, as in quantize.hip)
//   s = RN_fp32(max over the block |r| / 448),  q = RNE_E4M3(r / s)
//
// decided on the exact real quotient (s = 0 gives zeros).  The quotient is formed
// as t = r * (1 / s), which the hardware's reciprocal (one unit) and the product move
// by at most 3 units of its last place, and converted by the hardware.  A code can
// only be wrong where t lies within 4 units of the middle between two codes (bits
// 0x80000 below the three that E4M3 keeps; below 2**-6, where codes are 2**-9 apart,
// of t + 2**-6); a lane that holds such an element compares it with the middle
// exactly: fma(-middle, s, r) has the sign of r / s - middle.  bf16 inputs tie often
// (both mantissas are short), so this path costs no float64.  Scales below 2**-100,
// where the remainder could underflow, take float64 quotients.
//
// A block with an infinity has an infinite scale; its quotients in float64 are 0, and
// 448 for the infinite ones (with the reciprocal they would be NaN).
//
// Bound by memory: 2 (bf16) or 4 (fp32) bytes read and one written per element; a
// block is held in registers between its maximum and its codes.  A lane takes 8
// consecutive elements, 16 lanes a row's block, and the maxima are those of the bit
// patterns, two bf16 to an integer instruction.  Measured: 16384 x 4608 bf16 49 us, 4.7
// TB/s (57 .. 59 with inputs from HBM only), 2048 x 4608 in 8.9, 37 x 1184 in 3.2 .. 4.0; with a
// division per block and float64 near ties 62, 15.2 and 11.2.  Tiles: 11008 x 4096 bf16 34 us
// from HBM, 4.0 TB/s.  Rotations add float64 sums: 16384 x 4608 by 16, 32 and 128 59, 65 and 76
// us, tiles, which form them twice, 11008 x 4096 by 16 and 128 74 and 138.
#include "device_common.h"
#include "kernels.h"
#include "rows8.h"

namespace mxq {
namespace {

constexpr int kThreads = 256;

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

// Whether r * (1 / s) and the exact remainder decide a code.
__device__ __forceinline__ bool fast_scale(float s) { return s >= 0x1p-100f && s <= 0x1.fffffep127f; }

// 8 codes of values with scale s (inv = 1 / s, usable when `fast`).
__device__ __forceinline__ uint2 encode8(const float (&f)[8], float s, float inv, bool fast) {
  if (!fast) {
    uint32_t q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      q[e] = s == 0.f ? 0u : e4m3_encode_f64(fabs((double)f[e] / (double)s));
      q[e] |= (__float_as_uint(f[e]) >> 24) & 0x80u;
    }
    return make_uint2(q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24, q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24);
  }
  float t[8];
  uint32_t v[8], near = ~0u;   // smallest distance to a middle
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t[e] = f[e] * inv;
    // subnormal codes are as far apart as those of the first binade, 2**-6 on
    const float a = fabsf(t[e]);
    v[e] = __float_as_uint(a < 0x1p-6f ? a + 0x1p-6f : a);
    near = min(near, (v[e] - 0x7FFFCu) & 0xFFFFFu);
  }
  if (near <= 8u) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // f / s against the middle, exactly; t goes to the side it lies on, or onto the
      // middle, from which the conversion rounds to even
      const float m = __uint_as_float((v[e] & ~0xFFFFFu) | 0x80000u), mid = fabsf(t[e]) < 0x1p-6f ? m - 0x1p-6f : m;
      const float r = __builtin_fmaf(-mid, s, fabsf(f[e]));
      const float to = r > 0.f ? mid * 1.0009765625f : r < 0.f ? mid * 0.9990234375f : mid;
      if (((v[e] - 0x7FFFCu) & 0xFFFFFu) <= 8u) t[e] = copysignf(to, t[e]);
    }
  }
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false), hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[4], t[5], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(t[6], t[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// RN_fp32(amax / 448) from the product with the reciprocal and its exact remainder
// (right for every mantissa: compared over all 2**23); amax whose remainder could
// underflow, or is infinite (the remainder would be NaN), takes float64, whose
// quotient of two fp32 values rounds rightly.
__device__ __forceinline__ float scale_of(float amax) {
  if (!(amax >= 0x1p-90f && amax <= 0x1.fffffep127f)) return (float)((double)amax / 448.0);
  constexpr float r = 1.0f / 448.0f;
  const float q = amax * r;
  return __builtin_fmaf(__builtin_fmaf(-q, 448.0f, amax), r, q);
}

// Largest magnitude of a lane's elements as bits: an integer maximum, packed for bf16
// (magnitudes are in the order of their bits, a NaN above all).
template <int DT>
__device__ __forceinline__ uint32_t amax_bits(const Raw<DT>& w) {
  if constexpr (DT == DT_BF16) {
    typedef unsigned short v2us __attribute__((ext_vector_type(2)));
    const uint32_t d[4] = {w.lo.x, w.lo.y, w.lo.z, w.lo.w};
    v2us m = __builtin_bit_cast(v2us, d[0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(v2us, d[i] & 0x7FFF7FFFu));
    return (uint32_t)max(m.x, m.y) << 16;
  } else {
    const uint32_t d[8] = {w.lo.x, w.lo.y, w.lo.z, w.lo.w, w.hi.x, w.hi.y, w.hi.z, w.hi.w};
    uint32_t m = d[0] & 0x7FFFFFFFu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, d[i] & 0x7FFFFFFFu);
    return m;
  }
}

// Maximum over G consecutive lanes.
template <int G>
__device__ __forceinline__ uint32_t lanes_max(uint32_t b) {
  b = max(b, (uint32_t)xor_lane<1>((int)b));
  b = max(b, (uint32_t)xor_lane<2>((int)b));
  b = max(b, (uint32_t)xor_lane<4>((int)b));
  b = max(b, (uint32_t)xor_lane<8>((int)b));
  if constexpr (G == 64) {
    b = max(b, (uint32_t)xor_lane<16>((int)b));
    b = max(b, (uint32_t)xor_lane<32>((int)b));
  }
  return b;
}

// The lane's values, rotated with HAD > 0, and the bits of their largest magnitude.
template <int DT, int HAD>
__device__ __forceinline__ uint32_t values(const Raw<DT>& w, float (&f)[8], int lane, unsigned* dbg) {
  unpack8<DT>(w, f);
  flag_nonfinite(f, dbg);
  if constexpr (HAD > 0) {
    hadamard8<HAD>(f, lane);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    return m;
  } else {
    return amax_bits<DT>(w);
  }
}

// A workgroup takes 4 U rows x 4 blocks: lane group l / 16 of a wave one block of
// the row, so a wave's load is one contiguous kilobyte of bf16, U rows in
// flight.  The scales of a K-block lie together for all rows (the matrix product
// reads one per lane), so they leave through LDS as runs of 4 U.
template <int DT, int HAD, int U>
__global__ __launch_bounds__(kThreads) void quantize_fp8_kernel(Fp8Params p) {
  constexpr int kRows = 4 * U;
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
    const float s = scale_of(__uint_as_float(lanes_max<16>(values<DT, HAD>(raw[u], f, lane, p.dbg))));
    const bool fast = fast_scale(s);
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
  __shared__ uint32_t red[kThreads / 64];
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
  uint32_t bits = 0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {   // rows past the end repeat the last one
    float f[8];
    bits = max(bits, values<DT, HAD>(raw[u], f, lane, p.dbg));
  }
  const uint32_t m = lanes_max<64>(bits);
  if (lane == 0) red[wave] = m;
  __syncthreads();
  const float s = scale_of(__uint_as_float(max(max(red[0], red[1]), max(red[2], red[3]))));
  if (threadIdx.x == 0) *reinterpret_cast<float*>(p.scales + (int64_t)tr * p.ld_scales + (int64_t)tc * 4) = s;
  const bool fast = fast_scale(s);
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
    p.col_groups = (int)((p.cols + (int64_t)127) / 128);
    quantize_fp8_tile_kernel<DT, HAD><<<grid_of((p.rows + 127) / 128 * p.col_groups), kThreads, 0, s>>>(p);
  } else {
    p.col_groups = (int)((p.cols + (int64_t)511) / 512);
    // one row to a wave while that leaves compute units idle, and of fp32 (4096 x 4096
    // 17.4 us, with two 19.0), else two
    if (DT == DT_F32 || (p.rows + 3) / 4 * p.col_groups <= 2048)
      quantize_fp8_kernel<DT, HAD, 1><<<grid_of((p.rows + 3) / 4 * p.col_groups), kThreads, 0, s>>>(p);
    else
      quantize_fp8_kernel<DT, HAD, 2><<<grid_of((p.rows + 7) / 8 * p.col_groups), kThreads, 0, s>>>(p);
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
