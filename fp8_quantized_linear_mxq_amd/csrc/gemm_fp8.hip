// Products of E4M3 codes with fp32 block scales (block_gemm.h): the FP8 layer
//   y[m][n] = RN_bf16(sum over K-blocks b of sa[b][m] sw[n / 128][b] sum_{k in b} a[m][k] w[n][k] + bias[n]),
// the same grouped by expert, and the gated pair of projections.
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

template <bool GRP, int TI, int TJ, int WM, int WN>
hipError_t linear(const BlockP& p, hipStream_t s) {
  return launch_block_gemm<EL_FP8, LAY_ROW, LAY_ROW, EP_LINEAR, GRP, TI, TJ, WM, WN>(p, s);
}

}  // namespace

hipError_t launch_gemm_fp8(const GemmArgs& a, hipStream_t s) {
  const BlockP p = params(a);
  if (block_few(p)) return launch_block_few(p, EL_FP8, false, s);
  const bool big = gemm_tiles(a, 256, 256) >= 200;
  if (a.goff) return big ? linear<true, 8, 4, 2, 4>(p, s) : linear<true, 4, 4, 2, 2>(p, s);
  return big ? linear<false, 8, 4, 2, 4>(p, s) : linear<false, 4, 4, 2, 2>(p, s);
}

hipError_t launch_gated_fp8(const GatedArgs& a, hipStream_t s) {
  BlockP p = params(a.g);
  p.w2 = a.w2_codes; p.ldw2 = a.ldw2;
  p.ws2 = reinterpret_cast<const float*>(a.w2_scales); p.ldws2 = a.ld_ws2 / 4;
  p.gate = a.gate; p.up = a.up; p.ld_saved = a.ld_saved; p.act = a.act;
  if (block_few(p)) return launch_block_few(p, EL_FP8, true, s);
  if (gemm_tiles(a.g, 256, 128) >= 200)
    return launch_block_gemm<EL_FP8, LAY_ROW, LAY_ROW, EP_GATED, false, 8, 4, 2, 4>(p, s);
  return launch_block_gemm<EL_FP8, LAY_ROW, LAY_ROW, EP_GATED, false, 4, 4, 2, 2>(p, s);
}

}  // namespace mxq
