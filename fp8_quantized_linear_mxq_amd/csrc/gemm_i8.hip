// int8 x int8 GEMM with one fp32 scale per activation row and per weight row
// (output channel):
//   y[m][n] = RN_bf16(sa[m] sw[n] sum_k a[m][k] w[n][k] [+ u L2] [+ bias]),
// and the same product grouped by expert (rows of a sorted by expert).
//
// The sum is exact: v_mfma_i32_32x32x32_i8 accumulates in int32, which holds
// 127 * 127 * K up to K = 2**17.  It is rounded to fp32 once, then multiplied
// by the two scales in turn, (acc * sa) * sw: the product of the scales alone
// could underflow where the result does not.
//
// Organisation (the pipeline of the MXFP4 kernel without its block scales):
//  * workgroup tile (32*TM*WGM) x (64*TN), waves in a WGM x 2 grid, each wave
//    (32*TM) x (32*TN); K-tile 128, so every row of a tile contributes one
//    whole 128-byte line per K-tile;
//  * code tiles stream into a 2-stage LDS ring with direct global->LDS loads
//    one K-tile ahead of the MFMAs, landing in the XOR-swizzled slots the
//    fragment reads expect;
//  * lane l of a 32x32x32 step supplies row l % 32 and the 16 codes K =
//    16 * (l / 32) + [0, 16);
//  * the MFMAs compute D^T = W A^T, so each lane holds four consecutive output
//    columns of one row, and the output leaves through LDS as whole rows.
#include "device_common.h"
#include "gemm_common.h"
#include "gemm_pipe.h"
#include "grouped.h"
#include "kernels.h"

namespace mxq {
namespace {

constexpr int BK = 128;           // K (and bytes per row) per K-tile
constexpr int RB = BK;
constexpr int CH = RB / 16;       // 16-byte chunks per row
constexpr int KS = BK / 32;       // MFMA K-steps per K-tile

template <int TM, int TN, int WGM, bool LR, bool GRP>
__global__ __launch_bounds__(128 * WGM, 1) void gemm_i8_kernel(GemmP p, int gm) {
  constexpr int NW = 2 * WGM;                      // waves: WGM (rows) x 2 (columns)
  constexpr int TBM = 32 * TM * WGM, TBN = 64 * TN, NTHR = 64 * NW;
  constexpr int A_STAGE = TBM * RB, W_STAGE = TBN * RB, STAGE = A_STAGE + W_STAGE;
  static_assert((TBM * CH / 64) % NW == 0 && (TBN * CH / 64) % NW == 0, "every wave the same loads");
  // two separate stages: reads of one are visibly independent of the loads in
  // flight into the other, so the compiler adds no wait for them
  __shared__ __attribute__((aligned(16))) uint8_t st0[STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t st1[STAGE];
  __shared__ __attribute__((aligned(16))) float scl[TBM + TBN];

  int tm, tn, m0;
  if constexpr (GRP) {
    const int tiles_m = group_tiles(p.goff, p.groups, p.M, TBM);
    if ((int)blockIdx.x >= tiles_m * p.tiles_n) return;
    tile_coords(blockIdx.x, tiles_m, p.tiles_n, gm, tm, tn);
    m0 = enter_group(p, TBM, tm);
    if (m0 < 0) return;
  } else {
    tile_coords(blockIdx.x, p.tiles_m, p.tiles_n, gm, tm, tn);
    m0 = tm * TBM;
  }
  const int n0 = tn * TBN;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, half = lane >> 5;
  const int KT = (p.K + BK - 1) / BK;
  const int last_ch = (p.K % BK) ? (p.K % BK) / 16 : CH;   // chunks of the last K-tile

  // the tile's scales, on their way while the first K-tiles load
  constexpr int NSC = (TBM + TBN + NTHR - 1) / NTHR;
  float my_scale[NSC];
#pragma unroll
  for (int t = 0; t < NSC; ++t) {
    const int i = t * NTHR + tid;
    const int ra = min(m0 + i, p.M - 1), rw = max(min(n0 + i - TBM, p.N - 1), 0);
    const uint8_t* pa = p.as + (int64_t)ra * p.ldas;
    const uint8_t* pw = p.ws + (int64_t)rw * p.ldws;
    my_scale[t] = *reinterpret_cast<const float*>(i < TBM ? pa : pw);
  }

  const uint8_t* zsrc = zero_src();
  const int swl = swz<CH>(l32);
  uint32_t a_base[KS], w_base[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const uint32_t c = ((2 * s + half) ^ swl) * 16;
    a_base[s] = (wm * 32 * TM + l32) * RB + c;
    w_base[s] = A_STAGE + (wn * 32 * TN + l32) * RB + c;
  }

  auto issue = [&](int kt, uint8_t* st) __attribute__((always_inline)) {
    const bool past = kt >= KT;   // past the end of K: a tile of zeros
    kt = past ? KT - 1 : kt;
    const int lim = kt == KT - 1 ? last_ch : CH;
    issue_tile<TBM, RB, NW>(p.a, p.lda, m0, p.M, kt, st, wave, lane, zsrc, past, nullptr, lim);
    issue_tile<TBN, RB, NW>(p.w, p.ldw, n0, p.N, kt, st + A_STAGE, wave, lane, zsrc, past, nullptr, lim);
  };

  v16i acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = v16i{};

  auto compute = [&](const uint8_t* st) __attribute__((always_inline)) {
    v4i fa[2][TM], fw[2][TN];
    auto frag = [&](int s, int b) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
        fw[b][j] = *reinterpret_cast<const v4i*>(st + w_base[s] + j * 32 * RB);
#pragma unroll
      for (int i = 0; i < TM; ++i)
        fa[b][i] = *reinterpret_cast<const v4i*>(st + a_base[s] + i * 32 * RB);
    };
    frag(0, 0);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if (s + 1 < KS) frag(s + 1, (s + 1) & 1);
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[s & 1][j], fa[s & 1][i], acc[i][j], 0, 0, 0);
    }
  };

  // One K-tile (tile t lives in stage t % 2): wait until K-tile kt has landed,
  // barrier (every wave is done reading the other stage), load K-tile kt+1
  // into that stage and multiply K-tile kt.  Whole 2-step groups, no branch
  // around the MFMAs; K-tiles past the end are loaded as zeros.
  constexpr int NT = tile_loads<TBM, RB, NW>() + tile_loads<TBN, RB, NW>();   // per wave per K-tile
  constexpr int N_MFMA = KS * TM * TN, N_DS0 = TM + TN, N_DS1 = (KS - 1) * (TM + TN);
  auto step = [&](int kt, const uint8_t* st_cur, uint8_t* st_nxt, bool first) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);   // nothing of the previous step sinks below the wait
    if (first) wait_vmcnt<NT>();
    else wait_vmcnt<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");   // no LDS read moves above the barrier
    if (!first) issue(kt + 1, st_nxt);
    compute(st_cur);
    __builtin_amdgcn_sched_group_barrier(0x100, N_DS0, 0);
#pragma unroll
    for (int k = 0; k < N_MFMA; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (k < N_DS1) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (k < NT) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  };
  issue(0, st0);
  issue(1, st1);
  step(0, st0, st1, true);
  step(1, st1, st0, false);
  for (int kt = 2; kt < KT; kt += 2) {
    step(kt, st0, st1, false);
    step(kt + 1, st1, st0, false);
  }
  wait_vmcnt<0>();   // the zero loads issued past the end
#pragma unroll
  for (int t = 0; t < NSC; ++t)
    if (t * NTHR + tid < TBM + TBN) scl[t * NTHR + tid] = my_scale[t];
  wait_lgkmcnt0();
  __syncthreads();

  v16f out[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    const float sa = scl[wm * 32 * TM + i * 32 + l32];
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const v4f sw = *reinterpret_cast<const v4f*>(&scl[TBM + wn * 32 * TN + j * 32 + 8 * g + 4 * half]);
#pragma unroll
        for (int e = 0; e < 4; ++e) out[i][j][4 * g + e] = ((float)acc[i][j][4 * g + e] * sa) * sw[e];
      }
  }
  const int row0 = m0 + wm * 32 * TM, col0 = n0 + wn * 32 * TN;
  if constexpr (LR) add_lowrank<TM, TN>(p, out, row0, col0, lane);
  // the whole output tile through LDS when its rows can leave as 16-byte
  // pieces (no column map, aligned rows), else each wave by itself
  constexpr int WRS = TBN * 2 + 16;
  if constexpr ((TBM / 2) * WRS <= STAGE) {
    if (!p.col_map && (p.ld_out & 7) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0) {
      epilogue_wg<TM, TN, WGM, STAGE>(p, out, m0, n0, wm, wn, lane, st0, st1);
      return;
    }
  }
  epilogue_tr<false, TM, TN>(p, out, 1.0f, row0, col0, lane);
}

template <int TM, int TN, int WGM>
hipError_t launch_cfg(GemmP p, hipStream_t s) {
  constexpr int TBM = 32 * TM * WGM, TBN = 64 * TN;
  const bool grp = p.goff != nullptr;
  p.tiles_m = grp ? (int)group_tiles_bound(p.M, p.groups, TBM) : (p.M + TBM - 1) / TBM;
  p.tiles_n = (p.N + TBN - 1) / TBN;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  // tile-rows per group: one XCD's share (tiles / 8) as a near-square block
  int gm = 1;
  while (gm * 2 <= p.tiles_m && (int64_t)gm * 2 * gm * 2 <= (tiles + 7) / 8) gm *= 2;
  const dim3 grid((unsigned)tiles);
  if (grp) gemm_i8_kernel<TM, TN, WGM, false, true><<<grid, 128 * WGM, 0, s>>>(p, gm);
  else if (p.rank > 0) gemm_i8_kernel<TM, TN, WGM, true, false><<<grid, 128 * WGM, 0, s>>>(p, gm);
  else gemm_i8_kernel<TM, TN, WGM, false, false><<<grid, 128 * WGM, 0, s>>>(p, gm);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_i8(const GemmArgs& a, hipStream_t s) {
  GemmP p = gemm_params(a);
  // rows a tile can fill: all of them, or a group's share
  const int64_t m = a.goff ? (a.M + a.groups - 1) / a.groups : a.M;
  const int64_t cu = 256;
  auto rounds = [&](int tbm, int tbn) {
    const int64_t t = ((m + tbm - 1) / tbm) * ((a.N + tbn - 1) / tbn) * (a.goff ? a.groups : 1);
    return (t + cu - 1) / cu;
  };
  const int64_t c44 = rounds(256, 256) * 16 * 10, c22 = rounds(128, 128) * 4 * 16;
  if (c44 <= c22) return launch_cfg<2, 4, 4>(p, s);
  if (((m + 127) / 128) * ((a.N + 127) / 128) * (a.goff ? a.groups : 1) < 128) return launch_cfg<1, 1, 2>(p, s);
  return launch_cfg<2, 2, 2>(p, s);
}

}  // namespace mxq
