// Products of E4M3 codes with fp32 block scales (block_gemm.h): the FP8 layer
//   y[m][n] = RN_bf16(sum over K-blocks b of sa[b][m] sw[n / 128][b] sum_{k in b} a[m][k] w[n][k] + bias[n]),
// the same grouped by expert, and the gated pair of projections.  8192^3 takes 479 .. 505 us
// with the card (2.18 .. 2.30 PFLOP/s), 4096 x 4096 x 11008 gated 376 .. 384 (1.92 .. 1.97: 5.4
// rounds of tiles take six), 777 x 1184 x 1001 7.7 .. 8.1; 16384 rows of 32 experts, K 2048, N
// 4096, 170 even (1.62 PFLOP/s) and 225 with half of them one expert's.
#include "block_gemm.h"

namespace mxq {
namespace {

BlockP params(const GemmArgs& a) {
  BlockP p{};
  p.a = a.a_codes; p.lda = a.lda;
  p.w = a.w_codes; p.ldw = a.ldw;
  p.as = reinterpret_cast<const float*>(a.a_scales); p.ldas = a.ld_as / 4;
  p.ws = reinterpret_cast<const float*>(a.w_scales); p.ldws = a.ld_ws / 4;
  p.M = (int)a.M; p.N = (int)a.N; p.K = (int)a.K;
  p.col_map = a.col_map;
  p.bias = a.bias;
  p.out = a.out; p.ld_out = a.ld_out; p.n_out = (int)a.n_out;
  p.goff = a.goff; p.groups = (int)a.groups;
  return p;
}

// The tile kernels: 256 x 256, 128 x 128, and 64 x 64 with whole K-tiles in flight.
// Larger tiles load fewer bytes per product, smaller ones fill the GPU: M x K x N 4096^3
// 72 / 85 / 157 us, 1024 x 4096 x 4096 51 / 27 / 36, 256 x 4096 x 4096 50 / 24 / 16, 2048 x
// 1152 x 1024 20 / 11.2 / 8.7.  The constants are fits to 32 .. 8192 rows, 512 .. 4608
// columns and K = 512 .. 8192, operands from HBM, within some 20%.
template <int EP, bool GRP>
hipError_t tiles(const BlockP& p, const GemmArgs& a, hipStream_t s) {
  constexpr int half = EP == EP_GATED ? 2 : 1;
  constexpr TileShape shapes[] = {{{6.5, 1.4, 6.0, 1.95, 256, true}, 256, 256 / half},
                                  {{3.4, 0.7, 5.5, 1.19, 512, false}, 128, 128 / half},
                                  {{2.2, 0.5, 1.5, 0.55, 512, false}, 64, 64 / half}};
  const double kt = (p.K + 127) / 128;
  const auto best = [&](int M, int N) {
    TileChoice c{1e30, 0, 1};
    for (int i = 0; i < 3; ++i) {
      const TileShape& t = shapes[i];
      const double tn = (N + t.cols - 1) / t.cols;
      const double n = GRP ? (double)group_tiles_bound(M, a.groups, t.rows) * tn : (double)((M + t.rows - 1) / t.rows) * tn;
      const double time = tile_time(t.cost, n, kt);
      if (time < c.time) c = {time, i, 1};
    }
    return c;
  };
  // Two launches for a K of 4096 and more: with short sums the outputs' way out weighs
  // more than the estimate says (4400 x 1024 x 4400 in one and in two 38 / 42 us); not
  // for groups, whose rows are known to the GPU only.
  TilePlan plan{{{0, 0, p.M, p.N, best(p.M, p.N).shape, 1}, {}}, 1};
  if (!GRP && kt >= 32) plan = tile_plan(p.M, p.N, shapes[0], kt, best);
  for (int i = 0; i < plan.parts; ++i) {
    const TilePart& t = plan.part[i];
    hipError_t e;
    if (t.shape == 0) e = launch_block_gemm<EL_FP8, LAY_ROW, LAY_ROW, EP, GRP, 8, 4, 2, 4>(p, t, s);
    else if (t.shape == 1) e = launch_block_gemm<EL_FP8, LAY_ROW, LAY_ROW, EP, GRP, 4, 4, 2, 2>(p, t, s);
    else e = launch_block_gemm<EL_FP8, LAY_ROW, LAY_ROW, EP, GRP, 2, 2, 2, 2, 4>(p, t, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_gemm_fp8(const GemmArgs& a, hipStream_t s) {
  const BlockP p = params(a);
  if (block_few(p, false)) return launch_block_few(p, EL_FP8, false, s);
  return a.goff ? tiles<EP_LINEAR, true>(p, a, s) : tiles<EP_LINEAR, false>(p, a, s);
}

hipError_t launch_gated_fp8(const GatedArgs& a, hipStream_t s) {
  BlockP p = params(a.g);
  p.w2 = a.w2_codes; p.ldw2 = a.ldw2;
  p.ws2 = reinterpret_cast<const float*>(a.w2_scales); p.ldws2 = a.ld_ws2 / 4;
  p.gate = a.gate; p.up = a.up; p.ld_saved = a.ld_saved; p.act = a.act;
  if (block_few(p, true)) return launch_block_few(p, EL_FP8, true, s);
  return tiles<EP_GATED, false>(p, a.g, s);
}

}  // namespace mxq
