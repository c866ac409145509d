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
// it fits, else four (16384 x 4096 bf16 54 .. 58 us, 4.8 TB/s, fp32 107; one row of 1152 3.5).
// Backward: a persistent grid; a workgroup walks over rows with x and dy of a row in
// registers and keeps its share of dw and db there too, so both inputs are read once
// (8192 x 4096 bf16 44 us, 4.6 TB/s).  Each workgroup writes its sums to a row of the
// workspace and a second kernel adds those in a fixed order (no atomics: results do
// not depend on the order of workgroups; 5 us there).
//
// A lane's pieces are 8 elements, moved as vectors: aligned and streaming where all
// rows are whole pieces at 16-byte alignment, else (ANY) at the alignment of one
// element, the last piece of a row by single ones; short rows and very long ones of
// that kind move as single elements (V = 1).  J pieces per lane in registers; J = 0 reads a row of any
// length several times instead.
#include "device_common.h"
#include "gemm_pipe.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace mxq {
namespace {

// Vectors at the alignment of one element.
typedef uint32_t v4u_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float v4f_any __attribute__((ext_vector_type(4), aligned(4)));

// Elements of a piece at column c that exist.
template <int V, bool ANY>
__device__ __forceinline__ int count(int c, int cols) { return ANY ? min(V, cols - c) : V; }

// n elements from p[i] on, zeros behind them.
template <int DT, int V, bool ANY>
__device__ __forceinline__ void load(const void* p, int64_t i, int n, float (&f)[V]) {
  if constexpr (V == 1) {
    if constexpr (DT == DT_BF16) f[0] = bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
    else f[0] = static_cast<const float*>(p)[i];
  } else if (ANY && n < V) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      f[e] = 0.f;
      if (e < n) {
        if constexpr (DT == DT_BF16) f[e] = bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i + e]);
        else f[e] = static_cast<const float*>(p)[i + e];
      }
    }
  } else if constexpr (DT == DT_BF16) {
    const uint16_t* const q = static_cast<const uint16_t*>(p) + i;
    v4u d;
    if constexpr (ANY) d = *reinterpret_cast<const v4u_any*>(q);
    else d = *reinterpret_cast<const v4u*>(q);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(d[e] << 16);
      f[2 * e + 1] = __uint_as_float(d[e] & 0xFFFF0000u);
    }
  } else {
    const float* const q = static_cast<const float*>(p) + i;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4f d;
      if constexpr (ANY) d = *reinterpret_cast<const v4f_any*>(q + 4 * h);
      else d = *reinterpret_cast<const v4f*>(q + 4 * h);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[4 * h + e] = d[e];
    }
  }
}

template <int DT>
__device__ __forceinline__ void store_one(void* p, int64_t i, float f) {
  if constexpr (DT == DT_BF16) static_cast<uint16_t*>(p)[i] = (uint16_t)pack_bf16_rne(f, 0.f);
  else static_cast<float*>(p)[i] = f;
}

template <int DT, int V, bool ANY>
__device__ __forceinline__ void store(void* p, int64_t i, int n, const float (&f)[V]) {
  if constexpr (V == 1) {
    store_one<DT>(p, i, f[0]);
  } else if (ANY && n < V) {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < n) store_one<DT>(p, i + e, f[e]);
  } else if constexpr (DT == DT_BF16) {
    const v4u v = {pack_bf16_rne(f[0], f[1]), pack_bf16_rne(f[2], f[3]), pack_bf16_rne(f[4], f[5]),
                   pack_bf16_rne(f[6], f[7])};
    uint16_t* const q = static_cast<uint16_t*>(p) + i;
    if constexpr (ANY) *reinterpret_cast<v4u_any*>(q) = v;
    else __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(q));
  } else {
    float* const q = static_cast<float*>(p) + i;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4f v = {f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]};
      if constexpr (ANY) *reinterpret_cast<v4f_any*>(q + 4 * h) = v;
      else __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(q + 4 * h));
    }
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

template <int DT, int V, bool ANY, int J, int W>
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
        load<DT, V, ANY>(a.x, xr + c, count<V, ANY>(c, C), x[0]);
        f(x[0], c);
      }
    }
  };
  if constexpr (J > 0) {
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (c0 + j * STEP < C) load<DT, V, ANY>(a.x, xr + c0 + j * STEP, count<V, ANY>(c0 + j * STEP, C), x[j]);
  }
  each([&](const float (&v)[V], int) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < V; ++e) sum += v[e];
  });
  const float mean = row_sum<W>(sum, red[0]) * inv_c;
  float sq = 0.f;
  each([&](const float (&v)[V], int c) __attribute__((always_inline)) {
    const int n = count<V, ANY>(c, C);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float d = e < n ? v[e] - mean : 0.f;
      sq = fmaf(d, d, sq);
    }
  });
  const float rstd = rsqrtf(row_sum<W>(sq, red[1]) * inv_c + a.eps);
  if (!live) return;
  if (a.stats && c0 == 0) *reinterpret_cast<float2*>(a.stats + 2 * row) = make_float2(mean, rstd);
  each([&](const float (&v)[V], int c) __attribute__((always_inline)) {
    const int n = count<V, ANY>(c, C);
    float w[V], b[V], y[V];
    if (a.weight) load<DT, V, ANY>(a.weight, c, n, w);
    if (a.bias) load<DT, V, ANY>(a.bias, c, n, b);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      y[e] = (v[e] - mean) * rstd;
      if (a.weight) y[e] *= w[e];
      if (a.bias) y[e] += b[e];
    }
    store<DT, V, ANY>(a.y, yr + c, n, y);
  });
}

// ---- backward -------------------------------------------------------------

// One workgroup to a compute unit, so as few rows of sums as there are units: the two
// kernels 44 + 5 us at 8192 x 4096, with 512 threads and twice the rows 38 + 10.
constexpr int kBwdThreads = 1024;

// A wave's W-wave group takes rows group, group + groups, ...; all groups of the
// grid make the same number of steps, so that barriers are met by every wave.
template <int DT, int V, bool ANY, int J, int W>
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
      if (a.weight && c0 + j * STEP < C) load<DT, V, ANY>(a.weight, c0 + j * STEP, count<V, ANY>(c0 + j * STEP, C), w[j]);
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
      const int n = count<V, ANY>(c, C);
      load<DT, V, ANY>(a.x, xr + c, n, x[j]);
      load<DT, V, ANY>(a.dy, yr + c, n, g[j]);   // zeros behind the row add nothing to its sums
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
        if (a.weight) load<DT, V, ANY>(a.weight, c, count<V, ANY>(c, C), w[0]);
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
      if (a.dx) store<DT, V, ANY>(a.dx, row * a.ld_dx + c, count<V, ANY>(c, C), d);
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
        if (a.weight) load<DT, V, ANY>(a.weight, c, count<V, ANY>(c, C), w[0]);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[0][e] = (x[0][e] - mean) * rstd;
          if (params && e < count<V, ANY>(c, C)) {
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
  if (to) store_one<DT>(to, c < C ? c : c - C, s);
}

// Pieces per lane and waves per row of a row of `cols` elements: f(J, W).
template <int J> using I = std::integral_constant<int, J>;

// Rows that are not whole, aligned pieces move as single elements up to kShort columns,
// and in the backward pass past kAnyMost, where it sums in memory (J = 0).
constexpr int64_t kShort = 1024, kAnyMost = 16384;

template <int V, bool ANY, class F>
hipError_t fwd_shape(int64_t cols, F f) {
  // one wave: no barrier in the row's way, all of its loads in flight
  constexpr int64_t one = 64 * V;
  if constexpr (!ANY) {
    if (cols <= one) return f(I<1>{}, I<1>{});
    if (cols <= 2 * one) return f(I<2>{}, I<1>{});
  }
  if (cols <= 4 * one) return f(I<4>{}, I<1>{});
  if (cols <= 8 * one) return f(I<2>{}, I<4>{});
  if constexpr (V == 1) {
    return f(I<4>{}, I<4>{});
  } else {
    if (cols <= 16 * one) return f(I<4>{}, I<4>{});
    if (cols <= 32 * one) return f(I<8>{}, I<4>{});
    return f(I<0>{}, I<4>{});
  }
}

template <int V, bool ANY, class F>
hipError_t bwd_shape(int64_t cols, F f) {
  constexpr int64_t one = 64 * V;
  constexpr int J = V == 1 ? 8 : 2;
  if constexpr (!ANY) {
    if (cols <= one) return f(I<1>{}, I<1>{});
    if (cols <= J * one) return f(I<J>{}, I<1>{});
  }
  if (cols <= 2 * J * one) return f(I<J>{}, I<2>{});
  if constexpr (V > 1) {
    if (cols <= 4 * J * one) return f(I<J>{}, I<4>{});
    if (cols <= 8 * J * one) return f(I<J>{}, I<8>{});
    if (ANY || cols <= 16 * J * one) return f(I<J>{}, I<16>{});
  }
  return f(I<0>{}, I<16>{});
}

template <int DT, int V, bool ANY>
hipError_t forward(const LayerNormArgs& a, hipStream_t s) {
  return fwd_shape<V, ANY>(a.cols, [&](auto j, auto w) {
    constexpr int J = decltype(j)::value, W = decltype(w)::value, ROWS = kFwdThreads / 64 / W;
    layer_norm_kernel<DT, V, ANY, J, W><<<grid_of((a.rows + ROWS - 1) / ROWS), kFwdThreads, 0, s>>>(a);
    return hipGetLastError();
  });
}

template <int DT, int V, bool ANY>
hipError_t backward(const LayerNormBwdArgs& a, hipStream_t s) {
  int groups = 0;
  hipError_t e = hipSuccess;
  if (a.rows > 0)
    e = bwd_shape<V, ANY>(a.cols, [&](auto j, auto w) {
      constexpr int J = decltype(j)::value, W = decltype(w)::value, GR = kBwdThreads / 64 / W;
      groups = (int)std::min<int64_t>((a.rows + GR - 1) / GR, kLayerNormGroups);
      layer_norm_bwd_kernel<DT, V, ANY, J, W><<<groups, kBwdThreads, 0, s>>>(a);
      return hipGetLastError();
    });
  if (e != hipSuccess || !a.partial) return e;
  layer_norm_sum_kernel<DT><<<grid_of((2 * a.cols + 63) / 64), 64 * kSumWaves, 0, s>>>(a.partial, groups, (int)a.cols,
                                                                                  a.dweight, a.dbias);
  return hipGetLastError();
}

template <int DT, int V, bool ANY>
hipError_t run(const LayerNormArgs& a, hipStream_t s) { return forward<DT, V, ANY>(a, s); }
template <int DT, int V, bool ANY>
hipError_t run(const LayerNormBwdArgs& a, hipStream_t s) { return backward<DT, V, ANY>(a, s); }

template <int DT, class A>
hipError_t pieces(const A& a, bool vec, hipStream_t s) {
  if (vec) return run<DT, 8, false>(a, s);
  // single elements against vectors at any alignment, 96 x 583 bf16 3.4 / 5.2 us forward and
  // 7.2 / 9.4 backward, 6081 x 525 fp32 9.9 / 10.4 and 15.9 / 19.4; 5366 x 4090 bf16 60 / 27 and
  // 80 / 45; rows too long for the registers 1000 x 20001 99 / 36 and 150 / 227
  if (a.cols > kShort && (std::is_same_v<A, LayerNormArgs> || a.cols <= kAnyMost)) return run<DT, 8, true>(a, s);
  return run<DT, 1, false>(a, s);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t s) {
  const bool vec = a.cols % 8 == 0 && a.ldx % 8 == 0 && a.ldy % 8 == 0 && al16(a.x) && al16(a.y) && al16(a.weight) &&
                   al16(a.bias);
  return a.dtype == DT_BF16 ? pieces<DT_BF16>(a, vec, s) : pieces<DT_F32>(a, vec, s);
}

hipError_t launch_layer_norm_bwd(const LayerNormBwdArgs& a, hipStream_t s) {
  const bool vec = a.cols % 8 == 0 && a.ldx % 8 == 0 && a.ld_dy % 8 == 0 && (!a.dx || a.ld_dx % 8 == 0) && al16(a.x) &&
                   al16(a.dy) && al16(a.dx) && al16(a.weight);
  return a.dtype == DT_BF16 ? pieces<DT_BF16>(a, vec, s) : pieces<DT_F32>(a, vec, s);
}

}  // namespace mxq
