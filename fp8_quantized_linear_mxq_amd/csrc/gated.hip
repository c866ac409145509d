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
// x, and neither has a K-tile cut short.
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

// A thread takes 8 columns of a row.  VEC: rows of dy, g and u at 16-byte alignment.
template <bool VEC>
__global__ __launch_bounds__(kGradThreads) void gated_grad_kernel(GradP a, int64_t pieces) {
  const int64_t t = (int64_t)block_index() * kGradThreads + threadIdx.x;
  if (t >= pieces) return;
  const int per = a.np / 8;
  const int64_t row = t / per;
  const int c = (int)(t % per) * 8;
  float dg[8], du[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dg[e] = du[e] = 0.f;
  if (row < a.M) {
    float dy[8], g[8], u[8];
    const uint16_t* const y = a.dy + row * a.ld_dy + c;
    const float* const gr = a.gate + row * a.ld_saved + c;
    const float* const ur = a.up + row * a.ld_saved + c;
    if (VEC && c < a.N) {   // N is a multiple of 8
      const uint4 v = *reinterpret_cast<const uint4*>(y);
      const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        dy[2 * e] = __uint_as_float(d[e] << 16);
        dy[2 * e + 1] = __uint_as_float(d[e] & 0xFFFF0000u);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const v4f gv = *reinterpret_cast<const v4f*>(gr + 4 * h), uv = *reinterpret_cast<const v4f*>(ur + 4 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[4 * h + e] = gv[e];
          u[4 * h + e] = uv[e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (c + e >= a.N) continue;
      if (!VEC) {
        dy[e] = bf16_bits_to_f32(y[e]);
        g[e] = gr[e];
        u[e] = ur[e];
      }
      float d;
      const float f = activation<true>(a.act, g[e], &d);
      dg[e] = dy[e] * u[e] * d;
      du[e] = dy[e] * f;
    }
  }
  uint16_t* const o = a.p + row * 2 * a.np + c;
  auto pack = [](const float (&v)[8]) {
    return make_uint4(pack_bf16_rne(v[0], v[1]), pack_bf16_rne(v[2], v[3]), pack_bf16_rne(v[4], v[5]),
                      pack_bf16_rne(v[6], v[7]));
  };
  *reinterpret_cast<uint4*>(o) = pack(dg);
  *reinterpret_cast<uint4*>(o + a.np) = pack(du);
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

int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

int64_t gated_backward_workspace(int64_t M, int64_t N) { return pad64(M) * 2 * pad64(N) * 2; }

hipError_t launch_gated_bf16(const GatedArgs& a, hipStream_t s) {
  BlockP p{};
  p.a = a.g.a_codes; p.lda = a.g.lda;
  p.w = a.g.w_codes; p.ldw = a.g.ldw;
  p.w2 = a.w2_codes; p.ldw2 = a.ldw2;
  p.M = (int)a.g.M; p.N = (int)a.g.N; p.K = (int)a.g.K;
  p.out = a.g.out; p.ld_out = a.g.ld_out; p.n_out = (int)a.g.N;
  p.gate = a.gate; p.up = a.up; p.ld_saved = a.ld_saved; p.act = a.act;
  p.saved_vec = p.N % 4 == 0 && al16(a.gate);
  if (block_few(p)) return launch_block_few(p, EL_BF16, true, s);
  if (gemm_tiles(a.g, 256, 128) >= 200)
    return launch_block_gemm<EL_BF16, LAY_ROW, LAY_ROW, EP_GATED, false, 4, 2, 2, 4>(p, s);
  return launch_block_gemm<EL_BF16, LAY_ROW, LAY_ROW, EP_GATED, false, 2, 2, 2, 2>(p, s);
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
  const int64_t pieces = mp * (np / 8);
  const bool vec = a.N % 8 == 0 && a.ld_dy % 8 == 0 && a.ld_saved % 4 == 0 && al16(a.dy) && al16(a.gate) && al16(a.up);
  const dim3 grid = grid_of((pieces + kGradThreads - 1) / kGradThreads);
  if (vec) gated_grad_kernel<true><<<grid, kGradThreads, 0, s>>>(g, pieces);
  else gated_grad_kernel<false><<<grid, kGradThreads, 0, s>>>(g, pieces);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.dx) {   // P [M, 2 np] x [Wg; Wu]
    BlockP p{};
    p.a = reinterpret_cast<const uint8_t*>(a.ws); p.lda = 4 * np;
    p.w = a.wg; p.ldw = a.ldw; p.w2 = a.wu; p.ldw2 = a.ldw2;
    p.M = (int)a.M; p.N = p.n_out = (int)a.K; p.K = (int)(2 * np);
    p.k_split = (int)np; p.k_rows = (int)a.N;
    p.out = a.dx; p.ld_out = a.ld_dx;
    const double tiles = (double)((p.M + 255) / 256) * ((p.N + 255) / 256);
    e = tiles >= 200 ? launch_block_gemm<EL_BF16, LAY_ROW, LAY_COL, EP_LINEAR, false, 4, 2, 2, 4>(p, s)
                     : launch_block_gemm<EL_BF16, LAY_ROW, LAY_COL, EP_LINEAR, false, 2, 2, 2, 2>(p, s);
    if (e != hipSuccess) return e;
  }
  if (a.dwg) {   // P^T [2 np, M] x x
    BlockP p{};
    p.a = reinterpret_cast<const uint8_t*>(a.ws); p.lda = 4 * np;
    p.w = p.w2 = a.x; p.ldw = p.ldw2 = a.ldx;
    p.M = (int)(2 * np); p.N = p.n_out = (int)a.K; p.K = (int)mp;
    p.k_split = (int)mp; p.k_rows = (int)a.M;
    p.out = a.dwg; p.out2 = a.dwu; p.ld_out = a.ld_dw;
    p.m_split = (int)np; p.m_rows = (int)a.N;
    const double tiles = (double)((p.M + 255) / 256) * ((p.N + 255) / 256);
    e = tiles >= 200 ? launch_block_gemm<EL_BF16, LAY_COL, LAY_COL, EP_SPLIT, false, 4, 2, 2, 4>(p, s)
                     : launch_block_gemm<EL_BF16, LAY_COL, LAY_COL, EP_SPLIT, false, 2, 2, 2, 2>(p, s);
  }
  return e;
}

}  // namespace mxq
