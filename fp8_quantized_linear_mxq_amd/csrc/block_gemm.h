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
// Fragments.  bf16: 32 x 32 x 16 MFMAs; lane l holds row l % 32 and, of step s of a
// K-tile's four, the chunk 2 s + l / 32.  E4M3: 16 x 16 x 128 MFMAs, a K-tile each;
// lane l holds row l % 16 and the chunks 2 (l / 16) + {0, 1}.  (Any order of K is
// right that both operands share.)  The MFMAs compute D^T = W A^T: a lane holds four
// consecutive output columns of one row, so the row's scale is one register.
//
// E4M3 sums.  An MFMA takes groups of eight consecutive K and cuts each product towards
// zero to a multiple of 2**-13 of the binade that leads its group (a code's exponent
// being at least -6), so a group loses less than 7 * 2**-13 of its largest product; the
// groups are added in fp32 (measured on every output of random and adverse codes;
// 1.4e-5 of the sum's rms on normal data, without bias).  Each block of 128 is
// therefore summed from a zero accumulator and enters the fp32 sum scaled,
// acc += (sa sw) * sum, so the error stays relative to the block's own products;
// that takes the vector units half as long as the MFMA the matrix cores, and runs
// under the MFMAs after it.
// Converting the codes to bf16 would be exact at 2.4 times the MFMA time.
//
// Large ones: FP8 8192^3 479 .. 505 us with the card, 2.18 .. 2.30 PFLOP/s, the MFMAs busy 55% of
// the time and LDS bank conflicts as long as the other LDS work (400 us on zeros; a loop of
// MFMAs on random codes in registers reaches 4.1 PFLOP/s, 3.5 with the blocks added; the library's
// product with one scale to a tensor takes 407 .. 420); bound by the MFMAs under the power limit,
// bf16 8192 x 2048 x 5632 gated with its pre-activations 354 .. 398 us, its dx 286 .. 303 and dW
// 331 .. 348, where the library's plain products take 400, 297 and 364.  Small ones wait for memory: a
// lone workgroup takes 0.84 us to a K-tile of 128 x 128, against 0.2 of MFMAs.
#pragma once

#include "device_common.h"
#include "gated_act.h"
#include "gemm_common.h"
#include "gemm_pipe.h"
#include "grouped.h"
#include "kernels.h"

#include <algorithm>
#include <cmath>
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
  // this launch's part of the outputs, from row m_base and column n_base on
  int m_base, n_base, tiles_m, tiles_n;
  const int32_t* col_map;
  const uint16_t* bias;
  uint16_t* out; int64_t ld_out; int n_out;
  // EP_GATED: pre-activations, fp32 [M][ld_saved] each, or null
  float* gate; float* up; int64_t ld_saved; bool saved_vec;   // saved_vec: rows of whole, aligned quads
  int act;
  // EP_SPLIT: rows [0, m_split) go to out, the others to out2, m_rows of each
  uint16_t* out2; int m_split, m_rows;
  const int32_t* goff; int groups;
  // COL W: K split over this many workgroups of k_per K-tiles each; with part the sums
  // of split s go there as fp32 [splits][M - m_base][N - n_base]
  int splits, k_per;
  float* part;
};

// Estimated time (us) of tile kernels: a workgroup alone (its K-tiles come at the
// latency of the way from memory), and rounds of as many as fit the GPU, of which
// the last may be partly filled.
struct TileCost {
  double lat0, lat1, fix, per;
  int slots;
  bool whole;   // one workgroup to a compute unit: rounds do not overlap
};
inline double tile_time(const TileCost& c, double tiles, double kt) {
  const double lat = c.lat0 + c.lat1 * kt, full = c.fix + c.per * kt, r = tiles / c.slots, n = std::floor(r);
  const double more = full > lat ? full - lat : 0.;
  if (r <= 1) return lat + more * r;
  if (c.whole) return n * full + (r > n ? lat + more * (r - n) : 0.) + 2.5;
  return std::max(r, std::ceil(r) - 0.4) * full + 2.5;
}

// Tile shapes to choose from, and a product as one launch or two: whole rounds of the
// largest tiles on its first columns (or rows), the rest, which would fill another
// round in part, in the shape that is best for it.  The order of every sum is that of
// K whatever the shape, so nothing but the time depends on this.
struct TileShape { TileCost cost; int rows, cols; };
struct TileChoice { double time; int shape, splits; };
struct TilePart { int m0, n0, m1, n1; int shape, splits; };
struct TilePlan { TilePart part[2]; int parts; };

// best(M, N): the choice for a product of this size in one launch.
template <class Best>
TilePlan tile_plan(int M, int N, const TileShape& big, double kt, Best best) {
  const TileChoice one = best(M, N);
  TilePlan plan{{{0, 0, M, N, one.shape, one.splits}, {}}, 1};
  // Only for a clear gain, a second launch's some 6 us counted: the estimate takes a
  // round filled in part for slower than it is (fewer units at work run at a higher
  // clock).  In one and in two launches: dW 11264 x 8192 x 2048 with its first pass 475 /
  // 430 us, 8832 x 2304 x 4104 210 / 196, dx 4400 x 10112 x 4104 459 / 395, FP8 4096 x 4096
  // x 6000 120 / 111; where less is estimated nothing was won (gated FP8 4096 x 4096 x
  // 11008 385 / 385).
  double least = 0.95 * one.time - 6;
  const int64_t tm = (M + big.rows - 1) / big.rows, tn = (N + big.cols - 1) / big.cols, rounds = tm * tn / big.cost.slots;
  for (int rows = 0; rows < 2; ++rows) {
    const int64_t across = rows ? tn : tm, n = rounds * big.cost.slots / across;
    if (n == 0 || n >= (rows ? tm : tn)) continue;
    const int m1 = rows ? (int)n * big.rows : M, n1 = rows ? N : (int)n * big.cols, m0 = rows ? m1 : 0, n0 = rows ? 0 : n1;
    const TileChoice rest = best(M - m0, N - n0);
    const double t = tile_time(big.cost, (double)(n * across), kt) + rest.time;
    if (t >= least) continue;
    least = t;
    plan = {{{0, 0, m1, n1, 0, 1}, {m0, n0, M, N, rest.shape, rest.splits}}, 2};
  }
  return plan;
}

// Products of few rows (block_few.hip).
hipError_t launch_block_few(const BlockP& p, int el, bool gated, hipStream_t s);
bool block_few(const BlockP& p, bool gated);

typedef short v4s __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4s lds_v4s;

// The tile product: TI x TJ MFMA tiles of R x R per wave, WM x WN waves, the LDS a
// ring.
//
// DEEP = 0: five slots, each the A or the W half of a K-tile (equal halves: square
// tiles).  K-tile t has A in slot 2t % 5 and W in slot (2t + 1) % 5; W is loaded one
// K-tile ahead, A nearly two.  DEEP = S: S slots of whole K-tiles, S - 1 on their way,
// for grids that leave a compute unit one workgroup and no other that would hide the
// way from memory.  The slots are arrays of their own and the loop has as many
// K-tiles, so every read is visibly independent of the loads in flight and the
// compiler adds no wait; the K-tiles left over follow it in line.
//
// A wave walks over its MFMA tiles row by row with the fragments of one row of a and
// of all TJ rows of w in registers, reading those of the next row meanwhile.  By the
// last row of a K-tile every wave has read all of it: one barrier there releases its
// slots and, with the next K-tile's loads waited for, opens that one, whose first
// fragments are read under the last row's MFMAs.  Loads go out one or two to a row or
// tile: all of a slot's at once fill the queue to memory, and the wave that issues
// them stands still with its MFMAs behind them (8192^3 FP8: a fifth of the time).
template <int EL, int AL, int WL, int EP, bool GRP, int TI, int TJ, int WM, int WN, int DEEP>
struct BlockGemm {
  static constexpr int NW = WM * WN, THREADS = 64 * NW;
  static constexpr int R = EL == EL_FP8 ? 16 : 32;                  // rows of an MFMA tile
  static constexpr int TBM = R * TI * WM, TBN = R * TJ * WN;        // rows of a and of w in a tile
  static constexpr int OUT_N = EP == EP_GATED ? TBN / 2 : TBN;      // output columns
  static constexpr int SLOT_A = TBM * 128, SLOT_W = TBN * 128;
  static constexpr int LA = SLOT_A / 1024 / NW, LW = SLOT_W / 1024 / NW;   // loads per wave
  static constexpr int KT_ELEMS = EL == EL_FP8 ? 128 : 64;
  static constexpr int SLOTS = DEEP ? DEEP : 5, SLOT = DEEP ? SLOT_A + SLOT_W : SLOT_A;
  static constexpr int PER_EU = SLOTS * SLOT * 2 <= 160 * 1024 ? 2 * NW / 4 : NW / 4;   // waves of a SIMD
  // the output tile in LDS: whole rows of bf16, this many to a slot
  static constexpr int ROW_BYTES = 2 * OUT_N, ROWS = SLOT / ROW_BYTES / 32 * 32;
  // Steps of a K-tile that loads are dealt to: rows (E4M3) or MFMA tiles; the
  // barrier is before step `OPEN`.
  static constexpr int STEPS = EL == EL_FP8 ? TI : TI * TJ, OPEN = EL == EL_FP8 ? TI - 1 : (TI - 1) * TJ;
  // The W loads go out first, two to a step where there are enough, then the A loads,
  // the first at step OPEN.
  static constexpr int W_STEPS = (LW + 1) / 2 < (STEPS + 1) / 2 ? (LW + 1) / 2 : (STEPS + 1) / 2;
  static constexpr int PER_W = (LW + W_STEPS - 1) / W_STEPS, PER_A = (LA + STEPS - W_STEPS - 1) / (STEPS - W_STEPS);
  static constexpr int turn(int t) { return t >= OPEN ? t - OPEN : t + STEPS - OPEN; }   // steps since the barrier
  static constexpr int first_w(int t) { return turn(t) < W_STEPS ? PER_W * turn(t) : LW; }
  static constexpr int last_w(int t) { return turn(t) < W_STEPS && PER_W * turn(t) + PER_W < LW ? PER_W * turn(t) + PER_W : LW; }
  static constexpr int first_a(int t) { return turn(t) < W_STEPS ? 0 : (turn(t) - W_STEPS) * PER_A < LA ? (turn(t) - W_STEPS) * PER_A : LA; }
  static constexpr int last_a(int t) { return turn(t) < W_STEPS ? 0 : (turn(t) - W_STEPS + 1) * PER_A < LA ? (turn(t) - W_STEPS + 1) * PER_A : LA; }
  // W loads of the K-tile after next that are out before K-tile 0 begins
  static constexpr int AHEAD_W = last_w(STEPS - 1), AHEAD_A = last_a(STEPS - 1);
  static_assert(WM == 2 && TJ >= 2 && (EL == EL_BF16 ? TI % 2 == 0 || DEEP % 2 == 0 : TI % 2 == 0 && TI * TJ % 4 == 0), "the walk's fragment buffers");
  static_assert(DEEP > 0 || TBM == TBN, "five equal slots");
  static_assert(DEEP == 0 || DEEP >= 3, "one K-tile in use, one landed, others on their way");
  static_assert(EL == EL_BF16 || (AL == LAY_ROW && WL == LAY_ROW), "transposing reads are of 16-bit elements");
  static_assert((AL == LAY_ROW || TBM >= 128) && (WL == LAY_ROW || TBN >= 128), "four segments to swizzle");
  static_assert(SLOT_A % (1024 * NW) == 0 && SLOT_W % (1024 * NW) == 0, "whole loads");
  static_assert(TBM <= ROWS * SLOTS, "the output tile fits the slots");

  struct Frag { v4i f[EL == EL_FP8 ? 2 : 4]; };

  // A lane's fragment of MFMA tile `tile` of the wave.  `at` is its address of the
  // first chunk (ROW) or K-row (COL) in the wave's tile 0, relative to the slot; the
  // others differ in bits that the swizzles flip.  It is made opaque at every read:
  // left alone the compiler keeps the sums with every slot's address in registers,
  // which spill.
  template <int LAY, int TB>
  static __device__ __forceinline__ Frag read(uint8_t* slot, uint32_t at, int tile) {
    Frag r;
    asm volatile("" : "+v"(at));
    if constexpr (EL == EL_FP8) {
#pragma unroll
      for (int q = 0; q < 2; ++q) r.f[q] = *reinterpret_cast<const v4i*>(slot + (at ^ (16 * q)) + tile * 2048);
    } else if constexpr (LAY == LAY_ROW) {
#pragma unroll
      for (int q = 0; q < 4; ++q) r.f[q] = *reinterpret_cast<const v4i*>(slot + (at ^ (32 * q)) + tile * 4096);
    } else {
      at ^= tile * 64;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        v4s h[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          h[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(slot + at + (16 * s + 4 * e) * (2 * TB)));
        r.f[s] = __builtin_bit_cast(v4i, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
      }
    }
    return r;
  }

  // `at` for the MFMA tiles from tile0 (a multiple of their number in a wave) on.
  template <int LAY, int TB>
  static __device__ __forceinline__ uint32_t first(int tile0, int lane) {
    const int r = lane % R, part = lane / R;
    if constexpr (LAY == LAY_ROW) {
      return (tile0 * R + r) * 128 + (((EL == EL_FP8 ? 2 * part : part) ^ swz<8>(r)) * 16);
    } else {
      const int q = (lane >> 2) & 3;
      return (8 * part + q) * (2 * TB) + ((tile0 ^ q) * 64) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
    }
  }
};

// Stores the tile in LDS (at(r, c): the address of element c of row r) to the rows
// that to(r) gives (null: not stored), columns n0 + [0, n_lim), in pieces of V
// elements, neighbours by neighbouring threads; up to eight are read before they
// are stored.
template <int V, int ROWS, int COLS, int THREADS, class At, class To>
__device__ __forceinline__ void store_tile(int n_lim, int tid, At at, To to) {
  using Piece = std::conditional_t<V == 8, v4u, std::conditional_t<V == 4, uint2, std::conditional_t<V == 2, uint32_t, uint16_t>>>;
  constexpr int PER = COLS / V, N = ROWS * PER / THREADS, U = N % 8 == 0 ? 8 : N % 4 == 0 ? 4 : N % 2 == 0 ? 2 : 1;
  static_assert(ROWS * PER % THREADS == 0, "whole rounds");
  for (int t = 0; t < N; t += U) {
    Piece v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int idx = (t + k) * THREADS + tid;
      v[k] = *reinterpret_cast<const Piece*>(at(idx / PER, idx % PER * V));
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int idx = (t + k) * THREADS + tid, c = idx % PER * V;
      uint16_t* const o = to(idx / PER);
      if (!o || c >= n_lim) continue;
      if (c + V <= n_lim) {
        if constexpr (V == 8) __builtin_nontemporal_store(v[k], reinterpret_cast<Piece*>(o + c));
        else *reinterpret_cast<Piece*>(o + c) = v[k];
      } else {
        uint16_t e[V];
        __builtin_memcpy(e, &v[k], sizeof(Piece));
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c + i < n_lim) o[c + i] = e[i];
      }
    }
  }
}

// Keeps the compiler from moving a wave's LDS accesses across this point, where its lanes
// exchange values: the hardware keeps a wave's LDS accesses in order, but a lane's own
// addresses do not tell the compiler of the others'.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <int EL, int AL, int WL, int EP, bool GRP, int TI, int TJ, int WM, int WN, int DEEP>
__global__ __launch_bounds__(64 * WM * WN, (BlockGemm<EL, AL, WL, EP, GRP, TI, TJ, WM, WN, DEEP>::PER_EU))
void block_gemm_kernel(BlockP p, int gm) {
  using G = BlockGemm<EL, AL, WL, EP, GRP, TI, TJ, WM, WN, DEEP>;
  using Frag = typename G::Frag;
  constexpr int NW = G::NW, TBM = G::TBM, TBN = G::TBN, OUT_N = G::OUT_N, LA = G::LA, LW = G::LW;
  constexpr int S = G::SLOTS;
  __shared__ __attribute__((aligned(16))) uint8_t s0[G::SLOT], s1[G::SLOT], s2[G::SLOT], s3[S > 3 ? G::SLOT : 16],
      s4[S > 4 ? G::SLOT : 16];
  uint8_t* const slots[5] = {s0, s1, s2, s3, s4};

  int bid = (int)block_index(), split = 0;
  if constexpr (WL == LAY_COL) {
    const int tiles = p.tiles_m * p.tiles_n;
    split = bid / tiles;
    bid -= split * tiles;
    if (split >= p.splits) return;
  }
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
    m0 = p.m_base + tm * TBM;
  }
  // uniform, but from divisions, which the vector units do
  m0 = __builtin_amdgcn_readfirstlane(m0);
  const int n0 = __builtin_amdgcn_readfirstlane(p.n_base + tn * OUT_N);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  constexpr int R = G::R;
  const int rl = lane % R, part = lane / R;
  int KF = p.K / G::KT_ELEMS;                             // whole K-tiles
  int k_first = 0;                                        // the first of this workgroup's
  if constexpr (WL == LAY_COL) {
    k_first = __builtin_amdgcn_readfirstlane(split * p.k_per);
    KF = min(p.k_per, KF - k_first);
  }
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
        // R TJ rows per wave column: its gate rows, then its up rows
        const int wc = r / (R * TJ), in = r % (R * TJ), n = n0 + wc * (R * TJ / 2) + in % (R * TJ / 2);
        const bool second = in >= R * TJ / 2;
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
  // held in scalar registers: a kernel argument loaded again in the loop would, as a
  // scalar load in flight, drain every LDS wait
  uint32_t lda = (uint32_t)p.lda, ldw = (uint32_t)p.ldw, ldw2 = (uint32_t)p.ldw2;
  int k_split = p.k_split, k_rows = p.k_rows;
  if constexpr (AL == LAY_COL) asm volatile("" : "+s"(lda));
  if constexpr (WL == LAY_COL) {
    asm volatile("" : "+s"(ldw), "+s"(k_rows));
    if constexpr (EP == EP_LINEAR) asm volatile("" : "+s"(ldw2), "+s"(k_split), "+s"(wbase2));
  }
  // loads [t0, t1) of a K-tile's A or W; chunks past the end of K re-read the row's
  // first chunk of the K-tile, K-rows past it the last K-row (and are cut below)
  auto issue_a = [&](int kt, uint8_t* slot, int t0, int t1) __attribute__((always_inline)) {
    kt = kt < KT ? kt : KT - 1;
    const int k = kt + k_first;
    const uint8_t* b = abase + (AL == LAY_ROW ? (int64_t)k * 128 : (int64_t)k * 64 * lda);
    const uint32_t back = WL == LAY_ROW && AL == LAY_ROW && kt == KF && lc >= rest * 16 ? lc : 0;
#pragma unroll
    for (int t = 0; t < LA; ++t)
      if (t >= t0 && t < t1)
        __builtin_amdgcn_global_load_lds(b + (uint64_t)(va[t] - back), (lds_void_t*)(slot + (t * NW + wave) * 1024), 16, 0, 0);
  };
  auto issue_w = [&](int kt, uint8_t* slot, int t0, int t1) __attribute__((always_inline)) {
    kt = kt < KT ? kt : KT - 1;
    if constexpr (WL == LAY_ROW) {
      const int64_t k = (int64_t)kt * 128;
      const uint32_t back = kt == KF && lc >= rest * 16 ? lc : 0;
#pragma unroll
      for (int t = 0; t < LW; ++t) {
        if (t < t0 || t >= t1) continue;
        const uint8_t* b = wbase;
        if constexpr (EP == EP_GATED) {
          const int r = 8 * (NW * t + wave);   // a load's eight rows lie on one side
          if (r % (R * TJ) >= R * TJ / 2) b = wbase2;
        }
        __builtin_amdgcn_global_load_lds(b + k + (uint64_t)(vw[t] - back), (lds_void_t*)(slot + (t * NW + wave) * 1024), 16, 0, 0);
      }
    } else {
      int k0 = (kt + k_first) * 64;
      const uint8_t* b = wbase;
      uint32_t ld = ldw;
      if constexpr (EP == EP_LINEAR) {
        const bool second = k0 >= k_split;
        k0 -= second ? k_split : 0;
        b = second ? wbase2 : wbase;
        ld = second ? ldw2 : ldw;
      }
      b += (int64_t)k0 * ld;
      const int last = k_rows - 1 - k0;
#pragma unroll
      for (int t = 0; t < LW; ++t)
        if (t >= t0 && t < t1)
          __builtin_amdgcn_global_load_lds(b + (uint64_t)((uint32_t)min(kw + (512 / TBN) * NW * t, last) * ld + cw),
                                           (lds_void_t*)(slot + (t * NW + wave) * 1024), 16, 0, 0);
    }
  };

  // COL W: the K-tiles that end in a half's last K-row, of this workgroup's the next one.  Its
  // K-rows past the end, by each wave those that it has loaded, become zeros before the barrier
  // that opens it: A's are zeros, but the row in their place may hold an infinity.  (As
  // loads from a row of zeros, which take addresses of 64 bits to a lane, 3% slower.)
  int cut_kt = -1, cut_later = -1;
  if constexpr (WL == LAY_COL) {
    if (k_rows % 64) {
      cut_kt = k_rows / 64 - k_first;
      if constexpr (EP == EP_LINEAR) cut_later = cut_kt + k_split / 64;
      if (cut_kt < 0) cut_kt = cut_later;
    }
    asm volatile("" : "+s"(cut_kt), "+s"(cut_later));
  }
  auto cut_rows = [&](int kt, uint8_t* slot) __attribute__((always_inline)) {
    if constexpr (WL == LAY_COL) {
      if (__builtin_expect(kt != cut_kt, 1)) return;
#pragma unroll
      for (int t = 0; t < LW; ++t)
        if (kw + (512 / TBN) * NW * t >= k_rows % 64) *reinterpret_cast<v4i*>(slot + (t * NW + wave) * 1024 + lane * 16) = v4i{};
      wait_lgkmcnt0();
      cut_kt = cut_later;
    }
  };

  // ---- fragments ----
  const uint32_t at_a = G::template first<AL, TBM>(wm * TI, lane), at_w = G::template first<WL, TBN>(wn * TJ, lane);
  auto read_a = [&](uint8_t* slot, int i) __attribute__((always_inline)) { return G::template read<AL, TBM>(slot, at_a, i); };
  auto read_w = [&](uint8_t* slot, int j) __attribute__((always_inline)) { return G::template read<WL, TBN>(slot, at_w, j); };
  // chunks past the end of K as zeros
  auto cut = [&](Frag f) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < (int)(sizeof(f.f) / 16); ++q)
      if ((EL == EL_FP8 ? 2 * part + q : 2 * q + part) >= rest) f.f[q] = v4i{};
    return f;
  };

  using Acc = std::conditional_t<EL == EL_FP8, v4f, v16f>;
  Acc acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = Acc{};

  // FP8 scales.  Of a K-tile a lane loads those of the rows 64 r + lane of the wave
  // (one line each, the rows of a K-block lie together) and swaps quarters of the
  // wave when it comes to them; the wave's columns lie in one block of w's rows, and
  // lane l holds that block's scale of the loop's K-tile l.
  constexpr int RAW = EL == EL_FP8 ? (TI + 3) / 4 : 1;
  float raw[RAW], raw_next[RAW], sa[4], sw_of[2], sw_next[2], sw[2], row_scale[2] = {0.f, 0.f}, old_scale[2] = {0.f, 0.f};
  const float *as = nullptr, *ws = nullptr, *ws2 = nullptr;
  if constexpr (EL == EL_FP8) {
    as = p.as + m0;
    const int nb = __builtin_amdgcn_readfirstlane(min(n0 + wn * (OUT_N / WN), p.N - 1) / 128);
    ws = p.ws + nb * p.ldws;
    if constexpr (EP == EP_GATED) ws2 = p.ws2 + nb * p.ldws2;
  }
  auto row_scales = [&](int kt) __attribute__((always_inline)) {   // into raw_next
    kt = kt < KT ? kt : KT - 1;
    const uint8_t* const b = reinterpret_cast<const uint8_t*>(as + (int64_t)kt * p.ldas);
#pragma unroll
    for (int r = 0; r < RAW; ++r) {
      // clamped before the product with 4, which for a last row past 2**30 is no 32-bit number
      const uint32_t row = wm * TI * 16 + 64 * r + (TI < 4 ? lane & 31 : lane);
      raw_next[r] = *reinterpret_cast<const float*>(b + 4 * min(row, (uint32_t)(p.M - 1 - m0)));
    }
  };
  auto block_scales = [&](int kt) __attribute__((always_inline)) {   // K-tiles kt and on, into sw_next
    const int k = min(kt + lane, KT - 1);
    sw_next[0] = ws[k];
    if constexpr (EP == EP_GATED) sw_next[1] = ws2[k];
  };
  auto open_scales = [&](int number) __attribute__((always_inline)) {   // of K-tile `number` of the loop's
#pragma unroll
    for (int r = 0; r < RAW; ++r) raw[r] = raw_next[r];
#pragma unroll
    for (int h = 0; h < (EP == EP_GATED ? 2 : 1); ++h)
      sw[h] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw_of[h]), number));
  };
  auto turn_scales = [&](int kt) __attribute__((always_inline)) {   // the loop begins at K-tile kt
    sw_of[0] = sw_next[0];
    sw_of[1] = sw_next[1];
    block_scales(kt + S);
  };
  // the scales of rows 64 r + 16 e + lane % 16 from those of rows 64 r + lane
  auto spread = [&](float v) __attribute__((always_inline)) {
    const uint32_t u = __float_as_uint(v);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);       // quarters 0 1 0 1, 2 3 2 3
    const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    sa[0] = __uint_as_float(lo[0]);
    sa[1] = __uint_as_float(lo[1]);
    sa[2] = __uint_as_float(hi[0]);
    sa[3] = __uint_as_float(hi[1]);
  };

  Frag fa[2], fw[TJ];
  // FP8: the block sums of the last two MFMA tiles, added under the next ones
  v4f blk[4] = {v4f{}, v4f{}, v4f{}, v4f{}};
  auto add_block = [&](int n) __attribute__((always_inline)) {   // MFMA tile n of the K-tile (negative: the one before)
    const int t = n < 0 ? n + TI * TJ : n, i = t / TJ, j = t % TJ;
    const float s = (n < 0 || j >= TJ - 2 ? old_scale : row_scale)[EP == EP_GATED && j >= TJ / 2];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(blk[t % 4][e], s, acc[i][j][e]);
  };
  // MFMA tile (i, j) of a K-tile on fragments a
  auto tile = [&](int i, int j, const Frag& a) __attribute__((always_inline)) {
    if constexpr (EL == EL_FP8) {
      const int n = i * TJ + j;
      if (j == 0) {
        if (i % 4 == 0) spread(raw[i / 4]);
        old_scale[0] = row_scale[0];
        row_scale[0] = sa[i % 4] * sw[0];
        if constexpr (EP == EP_GATED) {
          old_scale[1] = row_scale[1];
          row_scale[1] = sa[i % 4] * sw[1];
        }
      }
      const v8i wv = __builtin_shufflevector(fw[j].f[0], fw[j].f[1], 0, 1, 2, 3, 4, 5, 6, 7);
      const v8i av = __builtin_shufflevector(a.f[0], a.f[1], 0, 1, 2, 3, 4, 5, 6, 7);
      blk[n % 4] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, av, v4f{}, 0, 0, 0, 127, 0, 127);
      add_block(n - 2);
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, fw[j].f[s]),
                                                            __builtin_bit_cast(v8bf, a.f[s]), acc[i][j], 0, 0, 0);
    }
  };

  constexpr int PAR = TI & 1;   // a K-tile of one row leaves the next in the other buffer
  // K-tile kt, number I of the loop's; fa[P] and all but the last of fw hold its first fragments
  auto step = [&](auto number, int kt) __attribute__((always_inline)) {
    constexpr int I = decltype(number)::value, P = PAR ? I & 1 : 0;
    uint8_t* const A = DEEP ? slots[I % S] : slots[(2 * I) % 5];
    uint8_t* const W = DEEP ? slots[I % S] + G::SLOT_A : slots[(2 * I + 1) % 5];
    uint8_t* const A1 = DEEP ? slots[(I + 1) % S] : slots[(2 * I + 2) % 5];
    uint8_t* const W1 = DEEP ? slots[(I + 1) % S] + G::SLOT_A : slots[(2 * I + 3) % 5];
    // loads of step t: what the last barrier released
    auto issue = [&](int t) __attribute__((always_inline)) {
      if constexpr (DEEP) {
        uint8_t* const to = t >= G::OPEN ? A : slots[(I + S - 1) % S];
        const int k = t >= G::OPEN ? kt + DEEP : kt + DEEP - 1;
        issue_w(k, to + G::SLOT_A, G::first_w(t), G::last_w(t));
        issue_a(k, to, G::first_a(t), G::last_a(t));
      } else {
        issue_w(t >= G::OPEN ? kt + 2 : kt + 1, t >= G::OPEN ? A : W1, G::first_w(t), G::last_w(t));
        issue_a(t >= G::OPEN ? kt + 3 : kt + 2, t >= G::OPEN ? W : slots[(2 * I + 4) % 5], G::first_a(t), G::last_a(t));
      }
    };
    if constexpr (EL == EL_FP8) {
      if constexpr (I == 0) turn_scales(kt);
      open_scales(I);
      row_scales(kt + 1);
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const Frag& a = fa[(i + P) & 1];
      if (i == 0) fw[TJ - 1] = read_w(W, TJ - 1);   // with one row, too, before the barrier
      if (i == TI - 1) {
        // every fragment of K-tile kt is read and K-tile kt+1 has landed
        wait_lgkmcnt0();
        wait_vmcnt<DEEP ? (DEEP - 2) * (LA + LW) : LA>();
        asm volatile("" ::: "memory");
        cut_rows(kt + 1, W1);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        if (j == 0) fa[(i + 1 + P) & 1] = i + 1 < TI ? read_a(A, i + 1) : read_a(A1, 0);
        if (i == TI - 1 && j > 0) fw[j - 1] = read_w(W1, j - 1);
        if (EL == EL_BF16) issue(i * TJ + j);
        else if (j == 1) issue(i);
        tile(i, j, a);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  if constexpr (EL == EL_FP8) {
    row_scales(0);
    block_scales(0);
  }
  if constexpr (DEEP) {
#pragma unroll
    for (int t = 0; t + 1 < DEEP; ++t) {
      issue_w(t, slots[t] + G::SLOT_A, 0, LW);
      issue_a(t, slots[t], 0, LA);
    }
    issue_w(DEEP - 1, slots[DEEP - 1] + G::SLOT_A, 0, G::AHEAD_W);
    issue_a(DEEP - 1, slots[DEEP - 1], 0, G::AHEAD_A);
    wait_vmcnt<(DEEP - 2) * (LA + LW) + G::AHEAD_W + G::AHEAD_A>();
  } else {
    issue_a(0, s0, 0, LA);
    issue_w(0, s1, 0, LW);
    issue_a(1, s2, 0, LA);
    issue_w(1, s3, 0, G::AHEAD_W);
    issue_a(2, s4, 0, G::AHEAD_A);
    wait_vmcnt<LA + G::AHEAD_W + G::AHEAD_A>();
  }
  asm volatile("" ::: "memory");
  cut_rows(0, DEEP ? s0 + G::SLOT_A : s1);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  if (KF > 0) {
    fa[0] = read_a(s0, 0);
#pragma unroll
    for (int j = 0; j + 1 < TJ; ++j) fw[j] = read_w(DEEP ? s0 + G::SLOT_A : s1, j);
    int kt = 0;
    for (; kt + S <= KF; kt += S) {
      step(std::integral_constant<int, 0>{}, kt);
      step(std::integral_constant<int, 1>{}, kt + 1);
      step(std::integral_constant<int, 2>{}, kt + 2);
      if constexpr (S > 3) step(std::integral_constant<int, 3>{}, kt + 3);
      if constexpr (S > 4) step(std::integral_constant<int, 4>{}, kt + 4);
    }
    if (kt < KF) step(std::integral_constant<int, 0>{}, kt);
    if (kt + 1 < KF) step(std::integral_constant<int, 1>{}, kt + 1);
    if constexpr (S > 3) if (kt + 2 < KF) step(std::integral_constant<int, 2>{}, kt + 2);
    if constexpr (S > 4) if (kt + 3 < KF) step(std::integral_constant<int, 3>{}, kt + 3);
  }
  wait_vmcnt<0>();
  wait_lgkmcnt0();
  __syncthreads();
  if (AL == LAY_ROW && rest > 0) {   // a last K-tile that K ends in
    const int ia = DEEP ? KF % S : (2 * KF) % 5, iw = DEEP ? ia : (2 * KF + 1) % 5;
    auto at = [&](int i) __attribute__((always_inline)) { return i == 0 ? s0 : i == 1 ? s1 : i == 2 ? s2 : i == 3 ? s3 : s4; };
    uint8_t* const A = at(ia);
    uint8_t* const W = at(iw) + (DEEP ? G::SLOT_A : 0);
    if constexpr (EL == EL_FP8) {
      if (KF % S == 0) turn_scales(KF);
      open_scales(KF % S);
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) fw[j] = cut(read_w(W, j));
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const Frag a = cut(read_a(A, i));
#pragma unroll
      for (int j = 0; j < TJ; ++j) tile(i, j, a);
    }
    __syncthreads();
  }
  if constexpr (EL == EL_FP8) {   // the last two block sums
    old_scale[0] = row_scale[0];
    old_scale[1] = row_scale[1];
    add_block(-2);
    add_block(-1);
  }

  // ---- epilogue ----
  // A lane holds quads of four consecutive columns of one row.  The tile goes through
  // LDS in bf16, 16-byte chunks swizzled by the row, and leaves as whole rows.
  constexpr int OJ = EP == EP_GATED ? TJ / 2 : TJ;
  if constexpr (WL == LAY_COL) {
    if (p.part) {   // N is a multiple of 8: whole quads
      const int64_t rows = p.M - p.m_base, cols = p.N - p.n_base;
      float* const sums = p.part + (split * rows - p.m_base) * cols - p.n_base;
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int m = m0 + (wm * TI + i) * R + rl;
#pragma unroll
        for (int j = 0; j < OJ; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int c = n0 + wn * (OUT_N / WN) + j * R + 8 * g + 4 * part;
            if (m < p.M && c < p.N)
              *reinterpret_cast<v4f*>(sums + m * cols + c) =
                  v4f{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
          }
      }
      return;
    }
  }
  if constexpr (EP == EP_GATED && EL == EL_BF16) {
    // Pre-activations: MFMA tiles of 32 x 32 pass through a part of a slot that is the
    // wave's own and leave as 128-byte runs, a quad to a lane where rows are whole,
    // aligned quads, else a number (a lane's quads stored from its registers are 32
    // bytes of a row: 23% more bytes written).
    if (p.gate) {
      constexpr int PER_SLOT = G::SLOT / (32 * 144);   // rows of 128 bytes, 16 apart
      static_assert(PER_SLOT * (S - 1) >= NW, "a part for every wave, beside the slots of the output");
      const int at = wave / PER_SLOT;
      uint8_t* const own = (at == 0 ? slots[S - 1] : at == 1 ? slots[S - 2] : slots[S - 3]) + wave % PER_SLOT * (32 * 144);
      for (int side = 0; side < 2; ++side) {
        float* const to = side ? p.up : p.gate;
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int j = 0; j < OJ; ++j) {
            const int mt = m0 + (wm * TI + i) * R, ct = n0 + wn * (OUT_N / WN) + j * R;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              v4f q;
#pragma unroll
              for (int e = 0; e < 4; ++e) q[e] = side ? acc[i][j + OJ][4 * g + e] : acc[i][j][4 * g + e];
              *reinterpret_cast<v4f*>(own + rl * 144 + (8 * g + 4 * part) * 4) = q;
            }
            wave_order();   // lanes read what others wrote
            // rows of the tile from the lane's first on, its columns among those that exist
            const bool vec = p.saved_vec;
            const int r0 = vec ? lane >> 3 : lane >> 5, c = vec ? (lane & 7) * 4 : lane & 31;
            const int rows = ct + c < p.N ? p.M - mt - r0 : 0;
            float* o = to + (int64_t)(mt + r0) * p.ld_saved + (ct + c);
            const uint8_t* from = own + r0 * 144 + c * 4;
            if (vec) {
#pragma unroll
              for (int t = 0; t < 4; ++t, o += 8 * p.ld_saved)
                if (8 * t < rows) __builtin_nontemporal_store(*reinterpret_cast<const v4f*>(from + t * 8 * 144), reinterpret_cast<v4f*>(o));
            } else {
#pragma unroll 8
              for (int t = 0; t < 16; ++t, o += 2 * p.ld_saved)
                if (2 * t < rows) *o = *reinterpret_cast<const float*>(from + t * 2 * 144);
            }
            wave_order();   // before the next tile's values take the place
          }
      }
    }
  }
  constexpr int SWM = OUT_N / 8 < 16 ? OUT_N / 8 - 1 : 15;
  const int n_lim = min(p.N, p.n_out) - n0;   // columns of the tile that exist
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    uint8_t* const slot = wm ? slots[(TI + i) * R / G::ROWS] : slots[i * R / G::ROWS];
    uint8_t* const row = slot + (((wm * TI + i) * R) % G::ROWS + rl) * G::ROW_BYTES;
#pragma unroll
    for (int j = 0; j < OJ; ++j)
#pragma unroll
      for (int g = 0; g < R * R / 256; ++g) {
        const int c = wn * (OUT_N / WN) + j * R + (EL == EL_FP8 ? 0 : 8 * g) + 4 * part;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * g + e];
        if constexpr (EP == EP_GATED) {
          float u[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) u[e] = acc[i][j + OJ][4 * g + e];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = activation<false>(p.act, v[e]) * u[e];
        }
        if constexpr (EP == EP_LINEAR) {
          if (p.bias) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int n = min(n0 + c + e, p.N - 1), to = p.col_map ? p.col_map[n] : n;
              if (to >= 0 && to < p.n_out) v[e] += bf16_bits_to_f32(p.bias[to]);
            }
          }
        }
        *reinterpret_cast<uint2*>(row + (((c >> 3) ^ (rl & SWM)) * 16) + (c & 4) * 2) =
            make_uint2(pack_bf16_rne(v[0], v[1]), pack_bf16_rne(v[2], v[3]));
      }
  }
  __syncthreads();
  auto at = [&](int r, int c) __attribute__((always_inline)) {
    const int q = r / G::ROWS;
    uint8_t* const slot = G::ROWS >= TBM || q == 0 ? s0 : q == 1 ? s1 : q == 2 ? s2 : s3;
    return slot + (r % G::ROWS) * G::ROW_BYTES + (((c >> 3) ^ (r & SWM)) * 16) + (c & 7) * 2;
  };
  if (EP == EP_LINEAR && p.col_map) {   // one column per thread
    const int c = tid % OUT_N, to = n0 + c < p.N ? p.col_map[n0 + c] : -1;
    if (to < 0 || to >= p.n_out) return;
    const int rows = min(TBM, p.M - m0);
#pragma unroll 8
    for (int r = tid / OUT_N; r < rows; r += G::THREADS / OUT_N)
      p.out[(int64_t)(m0 + r) * p.ld_out + to] = *reinterpret_cast<const uint16_t*>(at(r, c));
    return;
  }
  uint16_t* const out = p.out + n0;
  auto to = [&](int r) __attribute__((always_inline)) -> uint16_t* {
    int row = m0 + r;
    if (row >= p.M) return nullptr;
    uint16_t* o = out;
    if constexpr (EP == EP_SPLIT) {
      if (row >= p.m_split) {
        row -= p.m_split;
        o = p.out2 + n0;
      }
      if (row >= p.m_rows) return nullptr;
    }
    return o + (int64_t)row * p.ld_out;
  };
  uint64_t low = (uint64_t)p.ld_out * 2 | reinterpret_cast<uintptr_t>(p.out);
  if constexpr (EP == EP_SPLIT) low |= reinterpret_cast<uintptr_t>(p.out2);
  if ((low & 15) == 0) store_tile<8, TBM, OUT_N, G::THREADS>(n_lim, tid, at, to);
  else if ((low & 7) == 0) store_tile<4, TBM, OUT_N, G::THREADS>(n_lim, tid, at, to);
  else if ((low & 3) == 0) store_tile<2, TBM, OUT_N, G::THREADS>(n_lim, tid, at, to);
  else store_tile<1, TBM, OUT_N, G::THREADS>(n_lim, tid, at, to);
}

template <int EL, int AL, int WL, int EP, bool GRP, int TI, int TJ, int WM, int WN, int DEEP = 0>
hipError_t launch_block_gemm(BlockP p, const TilePart& part, hipStream_t s) {
  using G = BlockGemm<EL, AL, WL, EP, GRP, TI, TJ, WM, WN, DEEP>;
  p.m_base = part.m0;
  p.n_base = part.n0;
  p.tiles_m = GRP ? (int)group_tiles_bound(p.M, p.groups, G::TBM) : (part.m1 - part.m0 + G::TBM - 1) / G::TBM;
  p.tiles_n = (part.n1 - part.n0 + G::OUT_N - 1) / G::OUT_N;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n, blocks = tiles * std::max(p.splits, 1);
  if (blocks > INT32_MAX) return hipErrorInvalidValue;
  int gm = 1;
  while (gm * 2 <= p.tiles_m && (int64_t)gm * 2 * gm * 2 <= (tiles + 7) / 8) gm *= 2;
  block_gemm_kernel<EL, AL, WL, EP, GRP, TI, TJ, WM, WN, DEEP><<<grid_of(blocks), G::THREADS, 0, s>>>(p, gm);
  return hipGetLastError();
}

}  // namespace mxq
