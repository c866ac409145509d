// Matrix products on 8-bit floating point codes with block scales and on bf16, one
// kernel template for the FP8 layer and the gated feed-forward with its gradients.
//
// Operands.  A K-tile is 128 bytes of every row: 128 E4M3 codes or 64 bf16.  An
// operand lies row-wise (ROW: K contiguous) or column-wise (COL, bf16 only: the
// rows of the product contiguous, K strided), so that the gradients read
// activations and weights as they are stored:
//   forward   y  = x W^T        A ROW, W ROW
//   dx        = dp W            A ROW, W COL
//   dW        = dp^T x          A COL, W COL
// A ROW slot of LDS holds a row's eight 16-byte chunks at chunk ^ swz(row); a
// COL slot holds 64 K-rows of the tile, their 64-byte segments at segment ^ (k & 3),
// and its fragments come by transposing reads (ds_read_b64_tr_b16: 16 lanes fetch
// four K-rows of 16 columns and each gets the four K of its column), whose four
// rows then fall on different banks.
//
// Fragments.  Lane l of a 32-row MFMA operand holds row l % 32 and, of a K-tile,
// 64 bytes: for bf16 step s (16 K) the chunk 2 s + l / 32, for E4M3 step s (64 K)
// the chunks 4 s + 2 (l / 32) + {0, 1} (any order of K is right that both operands
// share).  The MFMAs compute D^T = W A^T: a lane holds four consecutive output
// columns of one row, so the row's scale is one register.
//
// E4M3 sums.  Within one MFMA the hardware adds products to about 2**-15 of the
// largest (measured: at most 2**-11.3 of it over 64 products, without bias, 1.3e-5
// of the sum's rms on normal data; profiles/mfma_probe.md).  Each block of 128 is
// therefore summed from a zero accumulator and enters the fp32 sum scaled,
// acc += (sa sw) * sum, so the error stays relative to the block's own products.
// Converting the codes to bf16 would be exact at 2.4 times the MFMA time.
#pragma once

#include "device_common.h"
#include "gated_act.h"
#include "gemm_common.h"
#include "gemm_pipe.h"
#include "grouped.h"
#include "kernels.h"

#include <type_traits>

namespace mxq {

enum : int { EL_FP8 = 0, EL_BF16 = 1 };
enum : int { LAY_ROW = 0, LAY_COL = 1 };
// outputs: the product (+ bias, column map); act(gate) * up; rows split over two outputs
enum : int { EP_LINEAR = 0, EP_GATED = 1, EP_SPLIT = 2 };

struct BlockP {
  const uint8_t* a; int64_t lda;             // bytes between rows (ROW) or K-rows (COL)
  const uint8_t* w; int64_t ldw;             // EP_GATED: the gate's weights, and
  const uint8_t* w2; int64_t ldw2;           // the up projection's; COL: rows of K from k_split on
  const float* as; int64_t ldas;             // FP8: [K / 128][ldas]
  const float* ws; int64_t ldws;             // FP8: [rows / 128][ldws]
  const float* ws2; int64_t ldws2;
  int M, N, K;          // rows of a, output columns, K (COL: a whole number of K-tiles)
  int k_split, k_rows;  // COL W: K-rows of each of w and w2, and how many of them exist
  int tiles_m, tiles_n;
  const int32_t* col_map;
  const uint16_t* bias;
  uint16_t* out; int64_t ld_out; int n_out;
  // EP_GATED: pre-activations, fp32 [M][ld_saved] each, or null
  float* gate; float* up; int64_t ld_saved;
  int act;
  // EP_SPLIT: rows [0, m_split) go to out, the others to out2, m_rows of each
  uint16_t* out2; int m_split, m_rows;
  const int32_t* goff; int groups;
};

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

// TI x TJ MFMA tiles of 32 x 32 per wave, WM x WN waves.
template <int EL, int AL, int WL, int EP, bool GRP, int TI, int TJ, int WM, int WN>
struct BlockGemm {
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int TBM = 32 * TI * WM, TBN = 32 * TJ * WN;      // rows of a and of w in a tile
  static constexpr int OUT_N = EP == EP_GATED ? TBN / 2 : TBN;      // output columns
  static constexpr int SLOT_A = TBM * 128, SLOT_W = TBN * 128;
  static constexpr int LA = SLOT_A / 1024 / NW, LW = SLOT_W / 1024 / NW;   // loads per wave
  static constexpr int KT_ELEMS = EL == EL_FP8 ? 128 : 64;
  static_assert(EP != EP_GATED || TJ % 2 == 0, "gate and up tiles in one wave");
  static_assert(EL == EL_BF16 || (AL == LAY_ROW && WL == LAY_ROW), "transposing reads are of 16-bit elements");
  static_assert((AL == LAY_ROW || TBM >= 128) && (WL == LAY_ROW || TBN >= 128), "four segments to swizzle");
  static_assert(SLOT_A % (1024 * NW) == 0 && SLOT_W % (1024 * NW) == 0, "whole loads");

  struct Frag { v4i f[4]; };

  static __device__ __forceinline__ Frag read_row(const uint8_t* slot, int row, const uint32_t (&c)[4]) {
    Frag r;
#pragma unroll
    for (int q = 0; q < 4; ++q) r.f[q] = *reinterpret_cast<const v4i*>(slot + row * 128 + c[q]);
    return r;
  }

  // Columns 32 tile .. 32 tile + 31 of a COL slot of TB columns.
  template <int TB>
  static __device__ __forceinline__ Frag read_col(uint8_t* slot, int tile, int lane) {
    Frag r;
    const int q = (lane >> 2) & 3;
    const uint32_t at = (8 * (lane >> 5) + q) * (2 * TB) + ((tile ^ q) * 64) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v4s h[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        h[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(slot + at + (16 * s + 4 * e) * (2 * TB)));
      r.f[s] = __builtin_bit_cast(v4i, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return r;
  }
};

template <int EL, int AL, int WL, int EP, bool GRP, int TI, int TJ, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void block_gemm_kernel(BlockP p, int gm) {
  using G = BlockGemm<EL, AL, WL, EP, GRP, TI, TJ, WM, WN>;
  using Frag = typename G::Frag;
  constexpr int NW = G::NW, TBM = G::TBM, TBN = G::TBN, OUT_N = G::OUT_N, LA = G::LA, LW = G::LW;
  __shared__ __attribute__((aligned(16))) uint8_t a0[G::SLOT_A], w0[G::SLOT_W], a1[G::SLOT_A], w1[G::SLOT_W];

  const int bid = (int)block_index();
  int tm, tn, m0;
  if constexpr (GRP) {
    const GroupScan gs(p.goff, p.groups, p.M, TBM);
    const int tiles_m = gs.tiles(p.tiles_m);
    if (bid >= tiles_m * p.tiles_n) return;
    tile_coords(bid, tiles_m, p.tiles_n, gm, tm, tn);
    GroupTile gt;
    if (!gs.find(tm, gt)) return;
    m0 = gt.row0;
    p.M = gt.row1;
    const int64_t first = (int64_t)gt.g * p.N;
    p.w += first * p.ldw;
    p.ws += first / 128 * p.ldws;
    if (p.bias) p.bias += first;
  } else {
    if (bid >= p.tiles_m * p.tiles_n) return;
    tile_coords(bid, p.tiles_m, p.tiles_n, gm, tm, tn);
    m0 = tm * TBM;
  }
  const int n0 = tn * OUT_N;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int l32 = lane & 31, half = lane >> 5;
  const int KF = p.K / G::KT_ELEMS;                       // whole K-tiles
  const int rest = (p.K % G::KT_ELEMS) * (EL == EL_FP8 ? 1 : 2) / 16;   // 16-byte chunks of a last one
  const int KT = KF + (rest > 0);

  // ---- loads ----
  // ROW: load t of a wave covers rows 8 (t NW + wave) + lane / 8; the lane's chunk
  // of its row is the same for every t.  Rows past the end re-read the last.
  // COL: load t covers 512 / TB K-rows; the lane's columns are the same for every t.
  const int lr = 8 * wave + (lane >> 3);
  const int lc = ((lane & 7) ^ swz<8>(lr)) * 16;
  uint32_t va[LA], vw[WL == LAY_ROW ? LW : 1];
  uint32_t ca = lc, cw = lc;    // the part of the offset within a row
  const uint8_t *abase, *wbase, *wbase2 = nullptr;
  if constexpr (AL == LAY_ROW) {
#pragma unroll
    for (int t = 0; t < LA; ++t)
      va[t] = (uint32_t)(min(m0 + 8 * NW * t + lr, p.M - 1) - m0) * (uint32_t)p.lda + lc;
    abase = p.a + (int64_t)m0 * p.lda;
  } else {
    constexpr int CPR = TBM / 8;
    const int kr = lane / CPR + (512 / TBM) * wave;
    const int seg = ((lane % CPR) >> 2) ^ (kr & 3), col = seg * 32 + (lane & 3) * 8;
    ca = 2 * (m0 + col < p.M ? col : 0);
#pragma unroll
    for (int t = 0; t < LA; ++t) va[t] = (uint32_t)(kr + (512 / TBM) * NW * t) * (uint32_t)p.lda + ca;
    abase = p.a + (int64_t)m0 * 2;
  }
  int kw = 0;   // the lane's K-row in a COL W tile's first load
  if constexpr (WL == LAY_ROW) {
#pragma unroll
    for (int t = 0; t < LW; ++t) {
      const int r = 8 * NW * t + lr;
      if constexpr (EP == EP_GATED) {
        // 32 TJ rows per wave column: its gate rows, then its up rows
        const int wc = r / (32 * TJ), in = r % (32 * TJ), n = n0 + wc * 16 * TJ + in % (16 * TJ);
        const bool second = in >= 16 * TJ;
        vw[t] = (uint32_t)(min(n, p.N - 1) - n0) * (uint32_t)(second ? p.ldw2 : p.ldw) + lc;
      } else {
        vw[t] = (uint32_t)(min(n0 + r, p.N - 1) - n0) * (uint32_t)p.ldw + lc;
      }
    }
    wbase = p.w + (int64_t)n0 * p.ldw;
    if constexpr (EP == EP_GATED) wbase2 = p.w2 + (int64_t)n0 * p.ldw2;
  } else {
    constexpr int CPR = TBN / 8;
    kw = lane / CPR + (512 / TBN) * wave;
    const int seg = ((lane % CPR) >> 2) ^ (kw & 3), col = seg * 32 + (lane & 3) * 8;
    cw = 2 * (n0 + col < p.N ? col : 0);
    wbase = p.w + (int64_t)n0 * 2;
    wbase2 = p.w2 + (int64_t)n0 * 2;
  }
  auto issue_a = [&](int kt, uint8_t* slot) __attribute__((always_inline)) {
    kt = kt < KT ? kt : KT - 1;
    const uint8_t* b = abase + (AL == LAY_ROW ? (int64_t)kt * 128 : (int64_t)kt * 64 * p.lda);
    // chunks past the end of K re-read the row's first chunk of the K-tile
    const uint32_t back = AL == LAY_ROW && kt == KF && lc >= rest * 16 ? lc : 0;
#pragma unroll
    for (int t = 0; t < LA; ++t)
      __builtin_amdgcn_global_load_lds(b + (uint64_t)(va[t] - back), (lds_void_t*)(slot + (t * NW + wave) * 1024), 16, 0, 0);
  };
  auto issue_w = [&](int kt, uint8_t* slot) __attribute__((always_inline)) {
    kt = kt < KT ? kt : KT - 1;
    if constexpr (WL == LAY_ROW) {
      const int64_t k = (int64_t)kt * 128;
      const uint32_t back = kt == KF && lc >= rest * 16 ? lc : 0;
#pragma unroll
      for (int t = 0; t < LW; ++t) {
        const uint8_t* b = wbase;
        if constexpr (EP == EP_GATED) {
          const int r = 8 * (NW * t + wave);   // a load's eight rows lie on one side
          if (r % (32 * TJ) >= 16 * TJ) b = wbase2;
        }
        __builtin_amdgcn_global_load_lds(b + k + (uint64_t)(vw[t] - back), (lds_void_t*)(slot + (t * NW + wave) * 1024), 16, 0, 0);
      }
    } else {
      int k0 = kt * 64;
      const bool second = k0 >= p.k_split;
      if (second) k0 -= p.k_split;
      const uint8_t* b = second ? wbase2 + (int64_t)k0 * p.ldw2 : wbase + (int64_t)k0 * p.ldw;
      const int rows = p.k_rows - k0;   // K-rows past the end re-read the K-tile's first
      const uint32_t ld = (uint32_t)(second ? p.ldw2 : p.ldw);
#pragma unroll
      for (int t = 0; t < LW; ++t) {
        const int kr = kw + (512 / TBN) * NW * t;
        __builtin_amdgcn_global_load_lds(b + (uint64_t)((kr < rows ? (uint32_t)kr * ld : 0u) + cw),
                                         (lds_void_t*)(slot + (t * NW + wave) * 1024), 16, 0, 0);
      }
    }
  };

  // ---- fragments ----
  uint32_t fc[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int c = EL == EL_FP8 ? 4 * (q >> 1) + 2 * half + (q & 1) : 2 * q + half;
    fc[q] = ((c ^ swz<8>(l32)) * 16);
  }
  auto read_a = [&](uint8_t* slot, int i) __attribute__((always_inline)) {
    if constexpr (AL == LAY_ROW) return G::read_row(slot, (wm * TI + i) * 32 + l32, fc);
    else return G::template read_col<TBM>(slot, wm * TI + i, lane);
  };
  auto read_w = [&](uint8_t* slot, int j) __attribute__((always_inline)) {
    if constexpr (WL == LAY_ROW) return G::read_row(slot, (wn * TJ + j) * 32 + l32, fc);
    else return G::template read_col<TBN>(slot, wn * TJ + j, lane);
  };
  // chunks past the end of K as zeros
  auto cut = [&](Frag& f) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = EL == EL_FP8 ? 4 * (q >> 1) + 2 * half + (q & 1) : 2 * q + half;
      if (c >= rest) f.f[q] = v4i{};
    }
  };

  v16f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v16f{};

  auto join = [](const v4i& a, const v4i& b) __attribute__((always_inline)) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto mma = [&](const Frag& w, const Frag& a, v16f c) __attribute__((always_inline)) {
    if constexpr (EL == EL_FP8) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        c = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(join(w.f[2 * s], w.f[2 * s + 1]), join(a.f[2 * s], a.f[2 * s + 1]),
                                                            c, 0, 0, 0, 127, 0, 127);
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, w.f[s]), __builtin_bit_cast(v8bf, a.f[s]), c, 0, 0, 0);
    }
    return c;
  };

  // FP8: the scales of a K-tile, one row of a per lane and MFMA tile, one block of
  // w's rows per wave (its 16 or 32 TJ rows lie in one block of 128)
  float sa[TI], sw[2];
  const float* as[TI];
  const float *ws = nullptr, *ws2 = nullptr;
  if constexpr (EL == EL_FP8) {
#pragma unroll
    for (int i = 0; i < TI; ++i) as[i] = p.as + min(m0 + (wm * TI + i) * 32 + l32, p.M - 1);
    const int nb = min(n0 + wn * (OUT_N / WN), p.N - 1) / 128;
    ws = p.ws + nb * p.ldws;
    if constexpr (EP == EP_GATED) ws2 = p.ws2 + nb * p.ldws2;
  }
  auto scales = [&](int kt) __attribute__((always_inline)) {
    kt = kt < KT ? kt : KT - 1;
#pragma unroll
    for (int i = 0; i < TI; ++i) sa[i] = as[i][(int64_t)kt * p.ldas];
    sw[0] = ws[kt];
    sw[1] = EP == EP_GATED ? ws2[kt] : sw[0];
  };

  auto compute = [&](uint8_t* A, uint8_t* W, bool last) __attribute__((always_inline)) {
    Frag fw[TJ];
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      fw[j] = read_w(W, j);
      if (last) cut(fw[j]);
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      Frag fa = read_a(A, i);
      if (last) cut(fa);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        if constexpr (EL == EL_FP8) {
          const v16f t = mma(fw[j], fa, v16f{});
          const float s = sa[i] * sw[EP == EP_GATED && j >= TJ / 2];
#pragma unroll
          for (int q = 0; q < 16; ++q) acc[i][j][q] = fmaf(t[q], s, acc[i][j][q]);
        } else {
          acc[i][j] = mma(fw[j], fa, acc[i][j]);
        }
      }
    }
  };

  issue_a(0, a0);
  issue_w(0, w0);
  for (int kt = 0; kt < KT; kt += 2) {
    if constexpr (EL == EL_FP8) scales(kt);
    wait_vmcnt<0>();
    __syncthreads();
    issue_a(kt + 1, a1);
    issue_w(kt + 1, w1);
    compute(a0, w0, kt == KF);
    if (kt + 1 >= KT) break;
    if constexpr (EL == EL_FP8) scales(kt + 1);
    wait_vmcnt<0>();
    __syncthreads();
    issue_a(kt + 2, a0);
    issue_w(kt + 2, w0);
    compute(a1, w1, kt + 1 == KF);
  }
  wait_vmcnt<0>();

  // ---- epilogue ----
  // lane: row i*32 + l32 of the wave, columns j*32 + 8 g + 4 half + [0, 4)
  constexpr int OJ = EP == EP_GATED ? TJ / 2 : TJ;
  const int n_lim = min(p.N, p.n_out);
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const int row = m0 + (wm * TI + i) * 32 + l32;
    if (row >= p.M) continue;
    uint16_t* orow = p.out + (int64_t)row * p.ld_out;
    if constexpr (EP == EP_SPLIT) {
      int r = row;
      uint16_t* o = p.out;
      if (r >= p.m_split) {
        r -= p.m_split;
        o = p.out2;
      }
      if (r >= p.m_rows) continue;
      orow = o + (int64_t)r * p.ld_out;
    }
#pragma unroll
    for (int j = 0; j < OJ; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = n0 + wn * (OUT_N / WN) + j * 32 + 8 * g + 4 * half;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int q = 4 * g + e, nn = n + e;
          if (nn >= p.N) continue;
          float v = acc[i][j][q];
          int c = nn;
          if constexpr (EP == EP_GATED) {
            const float u = acc[i][j + OJ][q];
            if (EL == EL_BF16 && p.gate) {
              p.gate[(int64_t)row * p.ld_saved + nn] = v;
              p.up[(int64_t)row * p.ld_saved + nn] = u;
            }
            v = activation<false>(p.act, v) * u;
          } else if constexpr (EP == EP_LINEAR) {
            if (p.col_map) c = p.col_map[nn];
            if (c < 0 || c >= p.n_out) continue;
            if (p.bias) v += bf16_bits_to_f32(p.bias[c]);
          }
          orow[c] = (uint16_t)pack_bf16_rne(v, 0.f);
        }
      }
  }
  (void)n_lim;
}

template <int EL, int AL, int WL, int EP, bool GRP, int TI, int TJ, int WM, int WN>
hipError_t launch_block_gemm(BlockP p, hipStream_t s) {
  using G = BlockGemm<EL, AL, WL, EP, GRP, TI, TJ, WM, WN>;
  p.tiles_m = GRP ? (int)group_tiles_bound(p.M, p.groups, G::TBM) : (p.M + G::TBM - 1) / G::TBM;
  p.tiles_n = (p.N + G::OUT_N - 1) / G::OUT_N;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  int gm = 1;
  while (gm * 2 <= p.tiles_m && (int64_t)gm * 2 * gm * 2 <= (tiles + 7) / 8) gm *= 2;
  block_gemm_kernel<EL, AL, WL, EP, GRP, TI, TJ, WM, WN><<<grid_of(tiles), G::THREADS, 0, s>>>(p, gm);
  return hipGetLastError();
}

}  // namespace mxq
