// Layer norm over the rows of a matrix and its gradients:
//   mean = sum x / C,  rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),
//   h = (x - mean) rstd,  y = h w + b;
//   with t = dy w:  dx = rstd (t - sum t / C - h sum (t h) / C),
//   dw = sum over rows of dy h,  db = sum over rows of dy.
// Everything in fp32 from the loaded values, one rounding at the end.  The
// variance is taken from the deviations (a second pass over registers): the
// difference of two sums would lose a row whose mean is large.
//
// Bound by memory.  Forward: a row is held in registers, one wave to a row while
// it fits, else four (16384 x 4096 bf16 54 us, 5.0 TB/s; one row of 1152 3.5).
// Backward: a persistent grid; a workgroup walks over rows with x and dy of a row in
// registers and keeps its share of dw and db there too, so both inputs are read once
// (8192 x 4096 bf16 44 us, 4.6 TB/s).  Each workgroup writes its sums to a row of the
// workspace and a second kernel adds those in a fixed order (no atomics: results do
// not depend on the order of workgroups; 5 us there).
//
// Rows of whole 8-element pieces at 16-byte alignment move as such (V = 8),
// others one element per lane (V = 1).  J pieces per lane in registers; J = 0
// reads a row of any length several times instead.
#include "device_common.h"
#include "gemm_pipe.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace mxq {
namespace {

template <int DT, int V>
__device__ __forceinline__ void load_v(const void* p, int64_t i, float (&f)[V]) {
  if constexpr (V == 1) {
    if constexpr (DT == DT_BF16) f[0] = bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
    else f[0] = static_cast<const float*>(p)[i];
  } else if constexpr (DT == DT_BF16) {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(d[e] << 16);
      f[2 * e + 1] = __uint_as_float(d[e] & 0xFFFF0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

template <int DT, int V>
__device__ __forceinline__ void store_v(void* p, int64_t i, const float (&f)[V]) {
  if constexpr (V == 1) {
    if constexpr (DT == DT_BF16) static_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16_rne(f[0], 0.f);
    else static_cast<float*>(p)[i] = f[0];
  } else if constexpr (DT == DT_BF16) {
    const v4u v = {pack_bf16_rne(f[0], f[1]), pack_bf16_rne(f[2], f[3]), pack_bf16_rne(f[4], f[5]),
                   pack_bf16_rne(f[6], f[7])};
    __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(static_cast<uint16_t*>(p) + i));
  } else {
    v4f* q = reinterpret_cast<v4f*>(static_cast<float*>(p) + i);
    __builtin_nontemporal_store(v4f{f[0], f[1], f[2], f[3]}, q);
    __builtin_nontemporal_store(v4f{f[4], f[5], f[6], f[7]}, q + 1);
  }
}

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += xor_lane_f<1>(v);
  v += xor_lane_f<2>(v);
  v += xor_lane_f<4>(v);
  v += xor_lane_f<8>(v);
  v += xor_lane_f<16>(v);
  return v + xor_lane_f<32>(v);
}

// Sum over the W waves of a row (W > 1: through LDS, all waves of the workgroup
// take part; a buffer is used again only after another barrier).
template <int W>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (W > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    const float* r = red + wave / W * W;
    v = r[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += r[w];
  }
  return v;
}

constexpr int kFwdThreads = 256;

template <int DT, int V, int J, int W>
__global__ __launch_bounds__(kFwdThreads) void layer_norm_kernel(LayerNormArgs a) {
  constexpr int ROWS = kFwdThreads / 64 / W, STEP = W * 64 * V;
  __shared__ float red[2][kFwdThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = (int64_t)block_index() * ROWS + wave / W;
  const bool live = row0 < a.rows;
  const int64_t row = live ? row0 : a.rows - 1;
  const int c0 = (wave % W * 64 + lane) * V, C = (int)a.cols;
  const float inv_c = 1.0f / (float)C;
  const int64_t xr = row * a.ldx, yr = row * a.ldy;

  float x[J > 0 ? J : 1][V];
  float sum = 0.f;
  auto each = [&](auto f) __attribute__((always_inline)) {   // f(piece, first column)
    if constexpr (J > 0) {
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (c0 + j * STEP < C) f(x[j], c0 + j * STEP);
    } else {
      for (int c = c0; c < C; c += STEP) {
        load_v<DT, V>(a.x, xr + c, x[0]);
        f(x[0], c);
      }
    }
  };
  if constexpr (J > 0) {
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (c0 + j * STEP < C) load_v<DT, V>(a.x, xr + c0 + j * STEP, x[j]);
  }
  each([&](const float (&v)[V], int) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < V; ++e) sum += v[e];
  });
  const float mean = row_sum<W>(sum, red[0]) * inv_c;
  float sq = 0.f;
  each([&](const float (&v)[V], int) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < V; ++e) sq = fmaf(v[e] - mean, v[e] - mean, sq);
  });
  const float rstd = rsqrtf(row_sum<W>(sq, red[1]) * inv_c + a.eps);
  if (!live) return;
  if (a.stats && c0 == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean, rstd);
  each([&](const float (&v)[V], int c) __attribute__((always_inline)) {
    float w[V], b[V], y[V];
    if (a.weight) load_v<DT, V>(a.weight, c, w);
    if (a.bias) load_v<DT, V>(a.bias, c, b);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      y[e] = (v[e] - mean) * rstd;
      if (a.weight) y[e] *= w[e];
      if (a.bias) y[e] += b[e];
    }
    store_v<DT, V>(a.y, yr + c, y);
  });
}

// ---- backward -------------------------------------------------------------

// One workgroup to a compute unit, so as few rows of sums as there are units: the two
// kernels 44 + 5 us at 8192 x 4096, with 512 threads and twice the rows 38 + 10.
constexpr int kBwdThreads = 1024;

// A wave's W-wave group takes rows group, group + groups, ...; all groups of the
// grid make the same number of steps, so that barriers are met by every wave.
template <int DT, int V, int J, int W>
__global__ __launch_bounds__(kBwdThreads) void layer_norm_bwd_kernel(LayerNormBwdArgs a) {
  constexpr int GR = kBwdThreads / 64 / W, STEP = W * 64 * V, P = J > 0 ? J : 1;
  __shared__ float red[2][2][kBwdThreads / 64];
  __shared__ float fold[J > 0 && GR > 1 ? GR * P * STEP : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, grp = wave / W;
  const int c0 = (wave % W * 64 + lane) * V, C = (int)a.cols;
  const float inv_c = 1.0f / (float)C;
  const bool params = a.partial != nullptr;
  float* const part_w = a.partial + (int64_t)blockIdx.x * 2 * C;   // this workgroup's dw, then db
  float* const part_b = part_w + C;

  float w[P][V], dw[P][V], db[P][V];
#pragma unroll
  for (int j = 0; j < P; ++j) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[j][e] = 1.f;
      dw[j][e] = db[j][e] = 0.f;
    }
    if constexpr (J > 0) {
      if (a.weight && c0 + j * STEP < C) load_v<DT, V>(a.weight, c0 + j * STEP, w[j]);
    }
  }
  if constexpr (J == 0) {   // sums of rows of any length live in the workspace
    if (params) {
      for (int c = threadIdx.x; c < 2 * C; c += kBwdThreads) part_w[c] = 0.f;
      __syncthreads();
    }
  }
  const int64_t stride = (int64_t)gridDim.x * GR, steps = (a.rows + stride - 1) / stride;
  for (int64_t it = 0; it < steps; ++it) {
    const int64_t row0 = it * stride + (int64_t)blockIdx.x * GR + grp;
    const bool live = row0 < a.rows;
    const int64_t row = live ? row0 : a.rows - 1;
    const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * row);
    const float mean = st.x, rstd = st.y;
    const int64_t xr = row * a.ldx, yr = row * a.ld_dy;
    float x[P][V], g[P][V];
    float s1 = 0.f, s2 = 0.f;
    auto add = [&](int j) __attribute__((always_inline)) {   // x becomes h
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[j][e] = (x[j][e] - mean) * rstd;
        const float t = g[j][e] * w[j][e];
        s1 += t;
        s2 = fmaf(t, x[j][e], s2);
      }
    };
    auto fetch = [&](int j, int c) __attribute__((always_inline)) {
      load_v<DT, V>(a.x, xr + c, x[j]);
      load_v<DT, V>(a.dy, yr + c, g[j]);
    };
    if constexpr (J > 0) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int e = 0; e < V; ++e) x[j][e] = g[j][e] = 0.f;
        if (c0 + j * STEP < C) fetch(j, c0 + j * STEP);
      }
#pragma unroll
      for (int j = 0; j < J; ++j)
        if (c0 + j * STEP < C) add(j);
    } else {
      for (int c = c0; c < C; c += STEP) {
        fetch(0, c);
        if (a.weight) load_v<DT, V>(a.weight, c, w[0]);
        add(0);
      }
    }
    if (a.dx) {
      // the two sums share a barrier; buffers alternate, so one is not written
      // while a slower wave still reads it
      float* const r1 = red[it & 1][0];
      float* const r2 = red[it & 1][1];
      s1 = wave_sum(s1);
      s2 = wave_sum(s2);
      if constexpr (W > 1) {
        if (lane == 0) {
          r1[wave] = s1;
          r2[wave] = s2;
        }
        __syncthreads();
        s1 = s2 = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
          s1 += r1[grp * W + k];
          s2 += r2[grp * W + k];
        }
      }
      s1 *= inv_c;
      s2 *= inv_c;
    }
    if (!live) continue;
    auto finish = [&](int j, int c) __attribute__((always_inline)) {
      float d[V];
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] = rstd * (g[j][e] * w[j][e] - s1 - x[j][e] * s2);
      if (a.dx) store_v<DT, V>(a.dx, row * a.ld_dx + c, d);
    };
    if constexpr (J > 0) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          dw[j][e] = fmaf(g[j][e], x[j][e], dw[j][e]);
          db[j][e] += g[j][e];
        }
        if (c0 + j * STEP < C) finish(j, c0 + j * STEP);
      }
    } else {
      for (int c = c0; c < C; c += STEP) {
        fetch(0, c);
        if (a.weight) load_v<DT, V>(a.weight, c, w[0]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[0][e] = (x[0][e] - mean) * rstd;
          if (params) {
            part_w[c + e] = fmaf(g[0][e], x[0][e], part_w[c + e]);
            part_b[c + e] += g[0][e];
          }
        }
        finish(0, c);
      }
    }
  }
  if constexpr (J > 0) {
    if (!params) return;
    // the groups' sums of a column meet in LDS, dw and db in turn
    auto out = [&](float (&acc)[P][V], float* to) __attribute__((always_inline)) {
      if constexpr (GR > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) fold[grp * P * STEP + c0 + j * STEP + e] = acc[j][e];
        __syncthreads();
        for (int c = threadIdx.x; c < C; c += kBwdThreads) {
          float v = fold[c];
#pragma unroll
          for (int k = 1; k < GR; ++k) v += fold[k * P * STEP + c];
          to[c] = v;
        }
      } else {
#pragma unroll
        for (int j = 0; j < P; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e)
            if (c0 + j * STEP + e < C) to[c0 + j * STEP + e] = acc[j][e];
      }
    };
    out(dw, part_w);
    out(db, part_b);
  }
}

// Column sums of the workgroups' rows [groups][2 C]: 64 columns of a workgroup,
// 16 waves taking every 16th row.
constexpr int kSumWaves = 16;

template <int DT>
__global__ __launch_bounds__(64 * kSumWaves) void layer_norm_sum_kernel(const float* partial, int groups, int C,
                                                                       void* dw, void* db) {
  __shared__ float red[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < 2 * (int64_t)C) {
#pragma unroll 8
    for (int g = wave; g < groups; g += kSumWaves) s += partial[(int64_t)g * 2 * C + c];
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= 2 * (int64_t)C) return;
#pragma unroll
  for (int w = 1; w < kSumWaves; ++w) s += red[w][lane];
  void* const to = c < C ? dw : db;
  const float v[1] = {s};
  if (to) store_v<DT, 1>(to, c < C ? c : c - C, v);
}

// Pieces per lane and waves per row of a row of `cols` elements: f(J, W).
template <int J> using I = std::integral_constant<int, J>;

template <int DT, int V, class F>
hipError_t fwd_shape(int64_t cols, F f) {
  // one wave: no barrier in the row's way, all of its loads in flight
  constexpr int64_t one = 64 * V;
  if (cols <= one) return f(I<1>{}, I<1>{});
  if (cols <= 2 * one) return f(I<2>{}, I<1>{});
  if (cols <= 4 * one) return f(I<4>{}, I<1>{});
  if (cols <= 8 * one) return f(I<2>{}, I<4>{});
  if (cols <= 16 * one) return f(I<4>{}, I<4>{});
  if (cols <= 32 * one) return f(I<8>{}, I<4>{});
  return f(I<0>{}, I<4>{});
}

template <int DT, int V, class F>
hipError_t bwd_shape(int64_t cols, F f) {
  constexpr int64_t one = 64 * V;
  constexpr int J = 16 / V > 2 ? 8 : 2;
  if (cols <= one) return f(I<1>{}, I<1>{});
  if (cols <= J * one) return f(I<J>{}, I<1>{});
  if (cols <= 2 * J * one) return f(I<J>{}, I<2>{});
  if (cols <= 4 * J * one) return f(I<J>{}, I<4>{});
  if (cols <= 8 * J * one) return f(I<J>{}, I<8>{});
  if (cols <= 16 * J * one) return f(I<J>{}, I<16>{});
  return f(I<0>{}, I<16>{});
}

template <int DT, int V>
hipError_t forward(const LayerNormArgs& a, hipStream_t s) {
  return fwd_shape<DT, V>(a.cols, [&](auto j, auto w) {
    constexpr int J = decltype(j)::value, W = decltype(w)::value, ROWS = kFwdThreads / 64 / W;
    layer_norm_kernel<DT, V, J, W><<<grid_of((a.rows + ROWS - 1) / ROWS), kFwdThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

template <int DT, int V>
hipError_t backward(const LayerNormBwdArgs& a, hipStream_t s) {
  int groups = 0;
  hipError_t e = hipSuccess;
  if (a.rows > 0)
    e = bwd_shape<DT, V>(a.cols, [&](auto j, auto w) {
      constexpr int J = decltype(j)::value, W = decltype(w)::value, GR = kBwdThreads / 64 / W;
      groups = (int)std::min<int64_t>((a.rows + GR - 1) / GR, kLayerNormGroups);
      layer_norm_bwd_kernel<DT, V, J, W><<<groups, kBwdThreads, 0, s>>>(a);
      return hipGetLastError();
    });
  if (e != hipSuccess || !a.partial) return e;
  layer_norm_sum_kernel<DT><<<grid_of((2 * a.cols + 63) / 64), 64 * kSumWaves, 0, s>>>(a.partial, groups, (int)a.cols,
                                                                                  a.dweight, a.dbias);
  return hipGetLastError();
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s) {
  const bool vec = a.cols % 8 == 0 && a.ldx % 8 == 0 && a.ldy % 8 == 0 && al16(a.x) && al16(a.y) && al16(a.weight) &&
                   al16(a.bias);
  if (a.dtype == DT_BF16) return vec ? forward<DT_BF16, 8>(a, s) : forward<DT_BF16, 1>(a, s);
  return vec ? forward<DT_F32, 8>(a, s) : forward<DT_F32, 1>(a, s);
}

hipError_t launch_layer_norm_bwd(const LayerNormBwdArgs& a, hipStream_t s) {
  const bool vec = a.cols % 8 == 0 && a.ldx % 8 == 0 && a.ld_dy % 8 == 0 && (!a.dx || a.ld_dx % 8 == 0) && al16(a.x) &&
                   al16(a.dy) && al16(a.dx) && al16(a.weight);
  if (a.dtype == DT_BF16) return vec ? backward<DT_BF16, 8>(a, s) : backward<DT_BF16, 1>(a, s);
  return vec ? backward<DT_F32, 8>(a, s) : backward<DT_F32, 1>(a, s);
}

}  // namespace mxq
