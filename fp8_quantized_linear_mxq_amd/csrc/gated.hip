// The gated feed-forward on bf16 operands and its gradients:
//   g = x Wg^T,  u = x Wu^T,  y = f(g) u;
//   dg = dy u f'(g),  du = dy f(g),
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x.
//
// Forward: one product whose workgroup tiles hold gate and up columns of the same
// outputs (block_gemm.h), so neither g nor u leaves the registers unless a
// backward pass needs them; then they are kept in fp32, since bf16 ones would add
// two more roundings to every gradient (a relative 2**-9 each on dg and du, next to
// the one that dg and du themselves take as operands of the matrix cores).
//
// Backward: one pass over dy, g and u forms P = [dg | du] in bf16, its halves
// padded with zeros to whole K-tiles of 64 columns and its rows to 64, so that dx is
// one product over 2 N and both weight gradients are one product over the rows of
// x, and neither has a K-tile cut short.  8192 x 2048 x 5632: forward 354 .. 398 us with
// the card, the pass 102 (bound by memory: 14 bytes to an element, 6.3 TB/s), dx 286 .. 303, dW
// 331 .. 348.
#include "block_gemm.h"

#include <algorithm>

namespace mxq {
namespace {

constexpr int kGradThreads = 256;

struct GradP {
  const uint16_t* dy; int64_t ld_dy;
  const float* gate; const float* up; int64_t ld_saved;
  uint16_t* p;       // [rows][2 np]
  int M, N, np, act;
};

// A thread takes V columns of a row: 8, with rows of dy, g and u at 16-byte alignment
// and N a multiple of 8, else 2 (a wave's loads then are runs of a row, whatever its
// alignment: 1111 x 2003 17 us with 8).
template <int V>
__global__ __launch_bounds__(kGradThreads) void gated_grad_kernel(GradP a, int64_t pieces) {
  const int64_t t = (int64_t)block_index() * kGradThreads + threadIdx.x;
  if (t >= pieces) return;
  const uint32_t per = a.np / V;
  const int64_t row = t / per;
  const int c = (int)(t % per) * V;
  float dg[V], du[V];
#pragma unroll
  for (int e = 0; e < V; ++e) dg[e] = du[e] = 0.f;
  if (row < a.M && c < a.N) {
    float dy[V], g[V], u[V];
    const uint16_t* const y = a.dy + row * a.ld_dy + c;
    const float* const gr = a.gate + row * a.ld_saved + c;
    const float* const ur = a.up + row * a.ld_saved + c;
    if constexpr (V == 8) {
      const v4u v = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(y));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dy[2 * e] = __uint_as_float(v[e] << 16);
        dy[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4f gv = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(gr + 4 * h));
        const v4f uv = __builtin_nontemporal_load(reinterpret_cast<const v4f*>(ur + 4 * h));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[4 * h + e] = gv[e];
          u[4 * h + e] = uv[e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int k = c + e < a.N ? e : 0;
        dy[e] = bf16_bits_to_f32(y[k]);
        g[e] = gr[k];
        u[e] = ur[k];
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (V == 2 && c + e >= a.N) continue;
      float d;
      const float f = activation<true>(a.act, g[e], &d);
      dg[e] = dy[e] * u[e] * d;
      du[e] = dy[e] * f;
    }
  }
  uint16_t* const o = a.p + row * 2 * a.np + c;
  uint32_t pg[V / 2], pu[V / 2];
#pragma unroll
  for (int e = 0; e < V / 2; ++e) {
    pg[e] = pack_bf16_rne(dg[2 * e], dg[2 * e + 1]);
    pu[e] = pack_bf16_rne(du[2 * e], du[2 * e + 1]);
  }
  if constexpr (V == 8) {
    *reinterpret_cast<uint4*>(o) = make_uint4(pg[0], pg[1], pg[2], pg[3]);
    *reinterpret_cast<uint4*>(o + a.np) = make_uint4(pu[0], pu[1], pu[2], pu[3]);
  } else {
    *reinterpret_cast<uint32_t*>(o) = pg[0];
    *reinterpret_cast<uint32_t*>(o + a.np) = pu[0];
  }
}

// [rows][cols] bf16 zeros: the gradients of a product without terms.
__global__ __launch_bounds__(kGradThreads) void zero_rows_kernel(uint16_t* p, int64_t ld, int64_t cols, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * kGradThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kGradThreads)
    p[i / cols * ld + i % cols] = 0;
}

hipError_t zero_rows(uint16_t* p, int64_t ld, int64_t rows, int64_t cols, hipStream_t s) {
  const int64_t n = rows * cols;
  if (n == 0) return hipSuccess;
  zero_rows_kernel<<<(int)std::min<int64_t>((n + kGradThreads - 1) / kGradThreads, 4096), kGradThreads, 0, s>>>(p, ld, cols, n);
  return hipGetLastError();
}

// Times of the tile kernels, fits as in gemm_fp8.hip: 256 x 256, 128 x 128, and with whole
// K-tiles in flight 64 x 128 (M x K x N 4096 x 4096 x 4096 gated 218 / 269 / 451 us, 512 x 4096 x
// 4096 81 / 55 / 62, 256 x 4096 x 4096 82 / 53 / 34).
constexpr TileShape kForward[] = {{{7.3, 1.1, 8.0, 1.6, 256, true}, 256, 128},
                                  {{0.5, 0.84, 4.0, 1.02, 512, false}, 128, 64},
                                  {{1.0, 0.5, 2.0, 0.48, 256, false}, 64, 64}};

double tiles_of(const TileShape& t, int M, int N) { return (double)((M + t.rows - 1) / t.rows) * ((N + t.cols - 1) / t.cols); }

// In one launch (8300 x 2056 x 2200 in one and in two, as the gradients, 181 / 182 us).
hipError_t gated_tiles(const BlockP& p, hipStream_t s) {
  const double kt = (p.K + 63) / 64;
  double time[3];
  for (int i = 0; i < 3; ++i) time[i] = tile_time(kForward[i].cost, tiles_of(kForward[i], p.M, p.N), kt);
  const TilePart all{0, 0, p.M, p.N, 0, 1};
  if (time[0] < time[1] && time[0] < time[2])
    return launch_block_gemm<EL_BF16, LAY_ROW, LAY_ROW, EP_GATED, false, 4, 2, 2, 4>(p, all, s);
  if (time[1] < time[2]) return launch_block_gemm<EL_BF16, LAY_ROW, LAY_ROW, EP_GATED, false, 2, 2, 2, 2>(p, all, s);
  return launch_block_gemm<EL_BF16, LAY_ROW, LAY_ROW, EP_GATED, false, 1, 2, 2, 2, 4>(p, all, s);
}

// A gradient's product: its tile shapes and over how many workgroups its K-tiles are
// split (fp32 sums in the workspace, added in order by a second kernel): dx has few
// tiles where there are few rows, and 2 N of K.  Only a last part is ever split.
TilePlan grad_plan(const BlockP& p, bool dw, int64_t room) {
  const TileShape shapes[] = {{kForward[0].cost, 256, 256}, {kForward[1].cost, 128, 128}, {kForward[2].cost, 64, 128}};
  const double kt = p.K / 64;
  return tile_plan(p.M, p.N, shapes[0], kt, [&](int M, int N) {
    TileChoice best{1e30, 0, 1};
    const double mn = (double)M * N;
    // the weights' gradients take no 64-row tiles (four swizzled segments to a K-row)
    for (int i = 0; i < (dw ? 2 : 3); ++i)
      for (int s = 1; s <= 16 && s * 4 <= std::max(kt, 4.); s *= 2) {
        if (s > 1 && (double)s * mn * 4 > (double)room) break;
        // the sums: written, read and rounded at some 4 TB/s, and a launch
        const double t = tile_time(shapes[i].cost, tiles_of(shapes[i], M, N) * s, std::ceil(kt / s)) +
                         (s > 1 ? 3.0 + s * mn * 8 / 4e6 : 0.);
        if (t < best.time) best = {t, i, s};
      }
    return best;
  });
}

struct SumP {
  const float* part;
  int m0, n0, M, N, splits;   // rows [m0, M), columns [n0, N)
  uint16_t* out; uint16_t* out2; int64_t ld_out;
  int m_split, m_rows;
};

// Rows of out (and from m_split on of out2) from the splits' sums, four columns to a thread.
__global__ __launch_bounds__(kGradThreads) void split_sum_kernel(SumP p) {
  const int64_t t = (int64_t)block_index() * kGradThreads + threadIdx.x, cols = p.N - p.n0, rows = p.M - p.m0, quads = cols / 4;
  if (t >= rows * quads) return;
  const int64_t in = t / quads;
  const int c = p.n0 + (int)(t % quads) * 4;
  const float* const from = p.part + in * cols + (c - p.n0);
  int64_t row = p.m0 + in;
  uint16_t* o = p.out;
  if (row >= p.m_split) {
    row -= p.m_split;
    o = p.out2;
  }
  if (row >= p.m_rows) return;
  v4f s = *reinterpret_cast<const v4f*>(from);
  for (int k = 1; k < p.splits; ++k) s += *reinterpret_cast<const v4f*>(from + k * rows * cols);
  o += row * p.ld_out + c;
  const uint32_t lo = pack_bf16_rne(s[0], s[1]), hi = pack_bf16_rne(s[2], s[3]);
  if ((reinterpret_cast<uintptr_t>(o) & 7) == 0) {
    *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
  } else {
    o[0] = (uint16_t)lo;
    o[1] = (uint16_t)(lo >> 16);
    o[2] = (uint16_t)hi;
    o[3] = (uint16_t)(hi >> 16);
  }
}

template <int AL, int EP>
hipError_t grad_product(BlockP p, float* part, int64_t room, hipStream_t s) {
  constexpr bool dw = EP == EP_SPLIT;
  const TilePlan plan = grad_plan(p, dw, room);
  const int kt = p.K / 64;
  for (int i = 0; i < plan.parts; ++i) {
    const TilePart& t = plan.part[i];
    p.k_per = (kt + t.splits - 1) / t.splits;
    p.splits = (kt + p.k_per - 1) / p.k_per;
    p.part = p.splits > 1 ? part : nullptr;
    hipError_t e;
    if (t.shape == 0) e = launch_block_gemm<EL_BF16, AL, LAY_COL, EP, false, 4, 2, 2, 4>(p, t, s);
    else if (t.shape == 1 || dw) e = launch_block_gemm<EL_BF16, AL, LAY_COL, EP, false, 2, 2, 2, 2>(p, t, s);
    else if constexpr (!dw) e = launch_block_gemm<EL_BF16, AL, LAY_COL, EP, false, 1, 2, 2, 2, 4>(p, t, s);
    if (e != hipSuccess) return e;
    if (!p.part) continue;
    const SumP q{p.part, t.m0, t.n0, p.M, p.N, p.splits, p.out, p.out2, p.ld_out, dw ? p.m_split : p.M, dw ? p.m_rows : p.M};
    const int64_t pieces = (int64_t)(p.M - t.m0) * ((p.N - t.n0) / 4);
    split_sum_kernel<<<grid_of((pieces + kGradThreads - 1) / kGradThreads), kGradThreads, 0, s>>>(q);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

namespace {

// P; then, shared by the two products in turn, the splits' sums: both shapes are
// known, so this is what grad_plan() asks for given any room.
int64_t p_bytes(int64_t M, int64_t N) { return pad64(M) * 2 * pad64(N) * 2; }

BlockP dx_shape(int64_t M, int64_t N, int64_t K) {
  BlockP p{};
  p.M = (int)M; p.N = p.n_out = (int)K; p.K = (int)(2 * pad64(N));
  return p;
}

BlockP dw_shape(int64_t M, int64_t N, int64_t K) {
  BlockP p{};
  p.M = (int)(2 * pad64(N)); p.N = p.n_out = (int)K; p.K = (int)pad64(M);
  return p;
}

int64_t split_bytes(const BlockP& p, bool dw) {
  const TilePlan plan = grad_plan(p, dw, INT64_MAX);
  const TilePart& t = plan.part[plan.parts - 1];
  return t.splits > 1 ? (int64_t)t.splits * (p.M - t.m0) * (p.N - t.n0) * 4 : 0;
}

}  // namespace

int64_t gated_backward_workspace(int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0 || K == 0) return p_bytes(M, N);
  return p_bytes(M, N) + std::max(split_bytes(dx_shape(M, N, K), false), split_bytes(dw_shape(M, N, K), true));
}

hipError_t launch_gated_bf16(const GatedArgs& a, hipStream_t s) {
  BlockP p{};
  p.a = a.g.a_codes; p.lda = a.g.lda;
  p.w = a.g.w_codes; p.ldw = a.g.ldw;
  p.w2 = a.w2_codes; p.ldw2 = a.ldw2;
  p.M = (int)a.g.M; p.N = (int)a.g.N; p.K = (int)a.g.K;
  p.out = a.g.out; p.ld_out = a.g.ld_out; p.n_out = (int)a.g.N;
  p.gate = a.gate; p.up = a.up; p.ld_saved = a.ld_saved; p.act = a.act;
  p.saved_vec = p.N % 4 == 0 && al16(a.gate);
  if (block_few(p, true)) return launch_block_few(p, EL_BF16, true, s);
  return gated_tiles(p, s);
}

hipError_t launch_gated_backward(const GatedBwdArgs& a, hipStream_t s) {
  const int64_t np = pad64(a.N), mp = pad64(a.M);
  if (a.M == 0 || a.N == 0) {
    hipError_t e = a.dx ? zero_rows(a.dx, a.ld_dx, a.M, a.K, s) : hipSuccess;
    if (e == hipSuccess && a.dwg) e = zero_rows(a.dwg, a.ld_dw, a.N, a.K, s);
    if (e == hipSuccess && a.dwg) e = zero_rows(a.dwu, a.ld_dw, a.N, a.K, s);
    return e;
  }
  GradP g;
  g.dy = a.dy; g.ld_dy = a.ld_dy;
  g.gate = a.gate; g.up = a.up; g.ld_saved = a.ld_saved;
  g.p = static_cast<uint16_t*>(a.ws);
  g.M = (int)a.M; g.N = (int)a.N; g.np = (int)np; g.act = a.act;
  const bool vec = a.N % 8 == 0 && a.ld_dy % 8 == 0 && a.ld_saved % 4 == 0 && al16(a.dy) && al16(a.gate) && al16(a.up);
  const int64_t pieces = mp * (np / (vec ? 8 : 2));
  const dim3 grid = grid_of((pieces + kGradThreads - 1) / kGradThreads);
  if (vec) gated_grad_kernel<8><<<grid, kGradThreads, 0, s>>>(g, pieces);
  else gated_grad_kernel<2><<<grid, kGradThreads, 0, s>>>(g, pieces);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t room = a.ws_bytes - p_bytes(a.M, a.N);
  float* const part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.ws) + p_bytes(a.M, a.N));
  if (a.dx) {   // P [M, 2 np] x [Wg; Wu]
    BlockP p = dx_shape(a.M, a.N, a.K);
    p.a = static_cast<const uint8_t*>(a.ws); p.lda = 4 * np;
    p.w = a.wg; p.ldw = a.ldw; p.w2 = a.wu; p.ldw2 = a.ldw2;
    p.k_split = (int)np; p.k_rows = (int)a.N;
    p.out = a.dx; p.ld_out = a.ld_dx;
    e = grad_product<LAY_ROW, EP_LINEAR>(p, part, room, s);
    if (e != hipSuccess) return e;
  }
  if (a.dwg) {   // P^T [2 np, M] x x
    BlockP p = dw_shape(a.M, a.N, a.K);
    p.a = static_cast<const uint8_t*>(a.ws); p.lda = 4 * np;
    p.w = p.w2 = a.x; p.ldw = p.ldw2 = a.ldx;
    p.k_split = (int)mp; p.k_rows = (int)a.M;
    p.out = a.dwg; p.out2 = a.dwu; p.ld_out = a.ld_dw;
    p.m_split = (int)np; p.m_rows = (int)a.N;
    e = grad_product<LAY_COL, EP_SPLIT>(p, part, room, s);
  }
  return e;
}

}  // namespace mxq
