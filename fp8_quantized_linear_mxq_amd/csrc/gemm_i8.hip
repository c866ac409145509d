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
// Organisation: workgroup tiles of 64 T x 64 T for T = 1, 2 or 4, four waves of
// 32 T x 32 T each; K-tile 128, so every row of a tile contributes one whole
// 128-byte line per K-tile.  Code tiles stream into LDS with direct
// global->LDS loads, landing in XOR-swizzled slots; lane l of a 32x32x32 step
// supplies row l % 32 and the 16 codes K = 16 * (l / 32) + [0, 16) of it; the
// MFMAs compute D^T = W A^T, so a lane holds four consecutive output columns of
// one row, and the output leaves through LDS as whole rows.
//
// What bounds it: on random codes a stream of these MFMAs from registers
// reaches 2.9 Pop/s with one wave per SIMD (3.4 with two; 4.5 and 4.8 on
// zeros: the clock drops under the switching power).  8192^3 runs at 2.54
// Pop/s (432 us), 1.51 us per K-tile and round of 256 tiles (2.84 Pop/s) plus
// some 10 us a round to fill the pipeline and write the output.
#include "device_common.h"
#include "gemm_common.h"
#include "gemm_pipe.h"
#include "grouped.h"
#include "kernels.h"

#include <algorithm>
#include <cmath>
#include <type_traits>

namespace mxq {
namespace {

constexpr int BK = 128;           // K (and bytes per row) per K-tile
constexpr int RB = BK;
constexpr int CH = RB / 16;       // 16-byte chunks per row
constexpr int KS = BK / 32;       // MFMA K-steps per K-tile

// The pipeline.  A T = 4 wave (128 x 128) reads 8 KB of fragments from LDS for
// 16 MFMAs, a 64 x 128 one 6 KB for 8, which with the loads' own LDS writes
// would keep the LDS as busy as the matrix cores; its accumulators take 256 of
// the 512 registers that one wave per SIMD has.
//
// Two stages of whole K-tiles leave the loads one K-tile of MFMAs to arrive,
// less than their latency plus 64 KB (T = 4) at the rate one compute unit
// streams: 2.06 us per K-tile, against 1.51 now.  So the LDS is a ring of five
// slots, each the A or the W half of a K-tile: K-tile t has A in slot 2t % 5
// and W in slot (2t + 1) % 5, A is loaded two K-tiles ahead and W one.  Each
// wave holds the fragments of one K-step in registers while it reads those of
// the next, so by the last K-step of K-tile t every wave has read all of it:
// one barrier there releases its slots and, with the loads of K-tile t+1 waited
// for, opens the next K-tile, whose first fragments are read under the MFMAs
// of the last K-step.  The slots are five arrays and the loop has five
// K-tiles, so every read is visibly independent of the loads in flight and the
// compiler adds no wait; the K-tiles left over follow it in line (leaving the
// loop from its middle instead costs 80 spilled registers).
//
// DEEP (T = 1): for grids that leave a compute unit one or two workgroups, so
// that nothing else hides the way from memory.  kStages stages of whole K-tiles,
// all but one of them on their way, and a K-tile's fragments read into registers
// at once under the MFMAs of the one before.  512 x 2048 x 4096 with operands
// from HBM 21.9 -> 12.5 us, 1024 x 2048 x 4096 (two workgroups) 22.9 -> 19.8; eight
// stages 12.6 and 23.1, T = 2 with five 22.9 and 23.0.
template <int T, bool LR, bool GRP, bool DEEP = false>
__global__ __launch_bounds__(256, T == 4 ? 1 : T == 2 || DEEP ? 2 : 4) void gemm_i8_ring_kernel(GemmP p, int gm) {
  constexpr int TB = 64 * T, HB = 32 * T;   // workgroup and wave tile
  constexpr int LD = TB * CH / 64 / 4;      // loads per wave per slot
  constexpr int kSlot = TB * RB;
  constexpr int kStages = 4;
  constexpr int kBuf = DEEP ? 2 * kSlot : kSlot;
  __shared__ __attribute__((aligned(16))) uint8_t s0[kBuf], s1[kBuf], s2[kBuf], s3[kBuf], s4[kSlot];
  uint8_t* const slots[5] = {s0, s1, s2, s3, s4};

  const int bid = (int)block_index();
  int tm, tn, m0;
  if constexpr (GRP) {
    const GroupScan gs(p.goff, p.groups, p.M, TB);
    const int tiles_m = gs.tiles(p.tiles_m);
    if (bid >= tiles_m * p.tiles_n) return;
    tile_coords(bid, tiles_m, p.tiles_n, gm, tm, tn);
    m0 = enter_group(p, gs, tm);
    if (m0 < 0) return;
  } else {
    if (bid >= p.tiles_m * p.tiles_n) return;
    tile_coords(bid, p.tiles_m, p.tiles_n, gm, tm, tn);
    m0 = tm * TB;
  }
  const int n0 = tn * TB;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int l32 = lane & 31, half = lane >> 5;
  const int KF = p.K / BK, rest = (p.K % BK) / 32;   // whole K-tiles, K-steps of a last one
  const int KT = KF + (rest > 0);

  // Load t of a wave covers rows 8 (4t + wave) + lane / 8; the lane's chunk of
  // its row is the same for every t.  Offsets from the tile's first row stay
  // within 32 bits (row strides are at most 2**24, checked by the host); rows
  // past the end re-read the last.
  const int lr = 8 * wave + (lane >> 3);
  const int lc = ((lane & 7) ^ swz<CH>(lr)) * 16;
  uint32_t va[LD], vw[LD];
#pragma unroll
  for (int t = 0; t < LD; ++t) {
    va[t] = (uint32_t)(min(m0 + 32 * t + lr, p.M - 1) - m0) * (uint32_t)p.lda + lc;
    vw[t] = (uint32_t)(min(n0 + 32 * t + lr, p.N - 1) - n0) * (uint32_t)p.ldw + lc;
  }
  const uint8_t* const abase = p.a + (int64_t)m0 * p.lda;
  const uint8_t* const wbase = p.w + (int64_t)n0 * p.ldw;
  // Half a K-tile into a slot.  K-tiles past the end re-read the last one;
  // chunks past the end of K re-read the row's first chunk of the K-tile (the
  // K-steps that hold them are not multiplied).
  auto issue = [&](const uint8_t* base, const uint32_t (&v)[LD], int kt, uint8_t* slot) __attribute__((always_inline)) {
    kt = kt < KT ? kt : KT - 1;
    const uint32_t back = kt == KF && lc >= rest * 32 ? lc : 0;
    const uint8_t* b = base + (int64_t)kt * RB;
#pragma unroll
    for (int t = 0; t < LD; ++t)
      __builtin_amdgcn_global_load_lds(b + (uint64_t)(v[t] - back),
                                       (lds_void_t*)(slot + (4 * t + wave) * 1024), 16, 0, 0);
  };

  // the scales and bias this thread brings to the epilogue
  float sa[T], sw, bs = 0.f;
#pragma unroll
  for (int i = 0; i < T; ++i)
    sa[i] = *reinterpret_cast<const float*>(p.as + (int64_t)min(m0 + wm * HB + i * 32 + l32, p.M - 1) * p.ldas);
  sw = *reinterpret_cast<const float*>(p.ws + (int64_t)min(n0 + tid % TB, p.N - 1) * p.ldws);
  int my_col = -1;   // output column of this thread's weight row
  if (tid < TB && n0 + tid < p.N) my_col = p.col_map ? p.col_map[n0 + tid] : n0 + tid;
  if (my_col >= p.n_out) my_col = -1;
  if (p.bias && my_col >= 0) bs = bf16_bits_to_f32(p.bias[my_col]);

  const int swl = swz<CH>(l32);
  uint32_t a_off[KS], w_off[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const uint32_t c = ((2 * s + half) ^ swl) * 16;
    a_off[s] = (wm * HB + l32) * RB + c;
    w_off[s] = (wn * HB + l32) * RB + c;
  }
  v16i acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = v16i{};
  constexpr int NF = DEEP ? 2 * KS : 2;   // fragment buffers
  v4i fa[NF][T], fw[NF][T];
  auto read = [&](const uint8_t* A, const uint8_t* W, int s, int b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < T; ++i) {
      fw[b][i] = *reinterpret_cast<const v4i*>(W + w_off[s] + i * 32 * RB);
      fa[b][i] = *reinterpret_cast<const v4i*>(A + a_off[s] + i * 32 * RB);
    }
  };
  auto mma = [&](int b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int j = 0; j < T; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[b][j], fa[b][i], acc[i][j], 0, 0, 0);
  };
  // a K-step's T*T MFMAs with the 2T fragment reads of the next and, where
  // there are any, 2T loads
  auto interleave = [&](bool loads) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < 2 * T; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      if (T == 4) __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  };
  auto step = [&](auto slot_of, int kt) __attribute__((always_inline)) {
    constexpr int I = decltype(slot_of)::value;
    uint8_t* const A = slots[(2 * I) % 5];
    uint8_t* const W = slots[(2 * I + 1) % 5];
    uint8_t* const A1 = slots[(2 * I + 2) % 5];
    uint8_t* const W1 = slots[(2 * I + 3) % 5];
    uint8_t* const A2 = slots[(2 * I + 4) % 5];
    read(A, W, 1, 1);
    issue(abase, va, kt + 2, A2);
    mma(0);
    interleave(true);
    __builtin_amdgcn_sched_barrier(0);
    read(A, W, 2, 0);
    mma(1);
    interleave(false);
    __builtin_amdgcn_sched_barrier(0);
    read(A, W, 3, 1);
    mma(0);
    interleave(false);
    __builtin_amdgcn_sched_barrier(0);
    // every fragment of K-tile kt is read and K-tile kt+1 has landed (A of
    // K-tile kt+2 may still be in flight)
    wait_lgkmcnt0();
    wait_vmcnt<LD>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    issue(wbase, vw, kt + 2, A);   // (2I + 5) % 5: the slot that A of K-tile kt leaves
    read(A1, W1, 0, 0);
    mma(1);
    interleave(true);
    __builtin_amdgcn_sched_barrier(0);
  };

  if constexpr (DEEP) {
    uint8_t* const st[kStages] = {s0, s1, s2, s3};
    auto load = [&](int kt, uint8_t* stage) __attribute__((always_inline)) {
      issue(abase, va, kt, stage);
      issue(wbase, vw, kt, stage + kSlot);
    };
    auto read_all = [&](const uint8_t* stage, int b) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < KS; ++s) read(stage, stage + kSlot, s, b * KS + s);
    };
    // K-tile kt is in registers (buffer I % 2) and its stage is free once every
    // wave's reads of it are done; K-tile kt+1 has landed
    auto deep_step = [&](auto stage_of, int kt) __attribute__((always_inline)) {
      constexpr int I = decltype(stage_of)::value;
      wait_lgkmcnt0();
      wait_vmcnt<(kStages - 2) * 2 * LD>();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      read_all(st[(I + 1) % kStages], (I + 1) & 1);
      load(kt + kStages, st[I]);
#pragma unroll
      for (int s = 0; s < KS; ++s) mma((I & 1) * KS + s);
      __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int t = 0; t < kStages; ++t) load(t, st[t]);
    wait_vmcnt<(kStages - 1) * 2 * LD>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read_all(s0, 0);
    int kt = 0;
    for (; kt + 4 <= KF; kt += 4) {
      deep_step(std::integral_constant<int, 0>{}, kt);
      deep_step(std::integral_constant<int, 1>{}, kt + 1);
      deep_step(std::integral_constant<int, 2>{}, kt + 2);
      deep_step(std::integral_constant<int, 3>{}, kt + 3);
    }
    if (kt < KF) deep_step(std::integral_constant<int, 0>{}, kt);
    if (kt + 1 < KF) deep_step(std::integral_constant<int, 1>{}, kt + 1);
    if (kt + 2 < KF) deep_step(std::integral_constant<int, 2>{}, kt + 2);
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    __syncthreads();
    // the K-steps of a last, partial K-tile, already in registers
#pragma unroll
    for (int s = 0; s < KS - 1; ++s)
      if (s < rest) {
        if (KF & 1) mma(KS + s);
        else mma(s);
      }
  } else {
    issue(abase, va, 0, s0);
    issue(wbase, vw, 0, s1);
    issue(abase, va, 1, s2);
    issue(wbase, vw, 1, s3);
    if (KF > 0) {
      wait_vmcnt<2 * LD>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      read(s0, s1, 0, 0);
      int kt = 0;
      for (; kt + 5 <= KF; kt += 5) {
        step(std::integral_constant<int, 0>{}, kt);
        step(std::integral_constant<int, 1>{}, kt + 1);
        step(std::integral_constant<int, 2>{}, kt + 2);
        step(std::integral_constant<int, 3>{}, kt + 3);
        step(std::integral_constant<int, 4>{}, kt + 4);
      }
      if (kt < KF) step(std::integral_constant<int, 0>{}, kt);
      if (kt + 1 < KF) step(std::integral_constant<int, 1>{}, kt + 1);
      if (kt + 2 < KF) step(std::integral_constant<int, 2>{}, kt + 2);
      if (kt + 3 < KF) step(std::integral_constant<int, 3>{}, kt + 3);
    }
    wait_vmcnt<0>();
    wait_lgkmcnt0();
    __syncthreads();
    if (rest > 0) {   // the K-steps of a last, partial K-tile
      const int ia = (2 * KF) % 5, iw = (2 * KF + 1) % 5;
      const uint8_t* A = ia == 0 ? s0 : ia == 1 ? s1 : ia == 2 ? s2 : ia == 3 ? s3 : s4;
      const uint8_t* W = iw == 0 ? s0 : iw == 1 ? s1 : iw == 2 ? s2 : iw == 3 ? s3 : s4;
  #pragma unroll
      for (int s = 0; s < KS - 1; ++s)
        if (s < rest) {
          read(A, W, s, 0);
          mma(0);
        }
      __syncthreads();
    }
  }

  // Epilogue: the tile in bf16 through slots 0-3 (64 rows of 512 bytes each,
  // 16-byte chunks swizzled by the row), the columns' scales and bias in slot
  // 4; it leaves as whole rows.
  float* const col = reinterpret_cast<float*>(s4);
  if (tid < TB) {
    col[tid] = sw;
    col[TB + tid] = bs;
  }
  __syncthreads();
  constexpr int ROW = 2 * TB;   // bytes of a staged row: a slot holds 64 of them
  constexpr int SWM = TB / 8 < 16 ? TB / 8 - 1 : 15;   // chunk swizzle: the row's low bits
#pragma unroll
  for (int i = 0; i < T; ++i) {
    v16f o[1][T];
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const v4f w4 = *reinterpret_cast<const v4f*>(col + wn * HB + j * 32 + 8 * g + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[0][j][4 * g + e] = ((float)acc[i][j][4 * g + e] * sa[i]) * w4[e];
      }
    if constexpr (LR) add_lowrank<1, T>(p, o, m0 + wm * HB + i * 32, n0 + wn * HB, lane);
    // rows wm*HB + i*32 + l32 of the tile, 64 to a slot
    uint8_t* const slot = T == 1 ? s0 + wm * 32 * ROW : wm ? slots[T / 2 + i / 2] : slots[i / 2];
    uint8_t* const row = slot + ((i & 1) * 32 + l32) * ROW;
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = wn * HB + j * 32 + 8 * g + 4 * half;
        const v4f b4 = *reinterpret_cast<const v4f*>(col + TB + c);
        *reinterpret_cast<uint2*>(row + (((c >> 3) ^ (l32 & SWM)) * 16) + half * 8) =
            make_uint2(pack_bf16_rne(o[0][j][4 * g] + b4[0], o[0][j][4 * g + 1] + b4[1]),
                       pack_bf16_rne(o[0][j][4 * g + 2] + b4[2], o[0][j][4 * g + 3] + b4[3]));
      }
  }
  __syncthreads();
  if (!p.col_map && (p.ld_out & 7) == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0) {
    const int n_lim = p.N < p.n_out ? p.N : p.n_out;
    constexpr int CPR = TB / 8;   // 16-byte pieces per row
#pragma unroll
    for (int q = 0; q < T; ++q) {
#pragma unroll
      for (int t = 0; t < 64 * CPR / 256; ++t) {
        const int r = (256 / CPR) * t + tid / CPR, ch = tid % CPR, row = m0 + q * 64 + r, n = n0 + ch * 8;
        const v4u v = *reinterpret_cast<const v4u*>(slots[q] + r * ROW + ((ch ^ (r & SWM)) * 16));
        if (row >= p.M) continue;
        uint16_t* const o = p.out + (int64_t)row * p.ld_out + n;
        if (n + 8 <= n_lim) {
          __builtin_nontemporal_store(v, reinterpret_cast<v4u*>(o));
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < n_lim) o[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
    return;
  }
  // a column map, or rows that are not 16-byte aligned: one column per thread,
  // so a wave stores 64 neighbours of a row at a time
  int* const map = reinterpret_cast<int*>(col);
  __syncthreads();
  if (tid < TB) map[tid] = my_col;
  __syncthreads();
  const int c = tid % TB, mc = map[c];
  if (mc < 0) return;
#pragma unroll
  for (int q = 0; q < T; ++q) {
    const int rows = min(64, p.M - (m0 + q * 64));
#pragma unroll 8
    for (int r = tid / TB; r < rows; r += 256 / TB)
      p.out[(int64_t)(m0 + q * 64 + r) * p.ld_out + mc] =
          *reinterpret_cast<const uint16_t*>(slots[q] + r * ROW + (((c >> 3) ^ (r & SWM)) * 16) + (c & 7) * 2);
  }
}

template <int T, bool DEEP = false>
hipError_t launch_ring(GemmP p, hipStream_t s) {
  constexpr int TB = 64 * T;
  const bool grp = p.goff != nullptr;
  p.tiles_m = grp ? (int)group_tiles_bound(p.M, p.groups, TB) : (p.M + TB - 1) / TB;
  p.tiles_n = (p.N + TB - 1) / TB;
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  int gm = 1;
  while (gm * 2 <= p.tiles_m && (int64_t)gm * 2 * gm * 2 <= (tiles + 7) / 8) gm *= 2;
  const dim3 grid = grid_of(tiles);
  if (grp) gemm_i8_ring_kernel<T, false, true, DEEP><<<grid, 256, 0, s>>>(p, gm);
  else if (p.rank == 0) gemm_i8_ring_kernel<T, false, false, DEEP><<<grid, 256, 0, s>>>(p, gm);
  else if constexpr (T < 4) gemm_i8_ring_kernel<T, true, false, DEEP><<<grid, 256, 0, s>>>(p, gm);
  else return hipErrorInvalidValue;   // not launched: no registers left for the branch
  return hipGetLastError();
}

// Estimated time (us) of a product of about t tiles of 64 T x 64 T with kt
// K-tiles: the latency of one workgroup, or the rounds of the workgroups that
// fit the 256 compute units (four of T = 1, two of T = 2, one of T = 4; large
// workgroups come in whole rounds).  The constants are fits to
// 64 .. 8192 rows and columns and K = 128 .. 8192, within some 15%.
template <int T>
double cost(double t, double kt) {
  constexpr double lat0 = T == 1 ? 1.6 : T == 2 ? 4.2 : 10.0, lat1 = T == 1 ? 0.38 : T == 2 ? 0.43 : 0.94;
  constexpr double fix = T == 1 ? 2.5 : T == 2 ? 4.5 : 10.5, per = T == 1 ? 0.85 : T == 2 ? 0.97 : 1.51;
  const double slots = 256.0 * (4 / T);
  const double rounds = T == 4 ? std::ceil(t / slots) : t / slots;
  return std::max(lat0 + lat1 * kt, 2.5 + rounds * (fix + per * kt));
}

}  // namespace

hipError_t launch_gemm_i8(const GemmArgs& a, hipStream_t s) {
  const GemmP p = gemm_params(a);
  // the tile sizes trade reuse (a T = 4 tile loads a quarter of the bytes per
  // MFMA of a T = 1 tile) against how many workgroups there are to fill the
  // GPU: 8192^3 2543 / 2154 Top/s with T = 4 / 2, 4096 x 4608 x 1152 46 / 32 /
  // 42 us, 777 x 1001 x 1184 34 / 10.4 / 6.2 us with T = 4 / 2 / 1
  const double kt = (double)((a.K + BK - 1) / BK), t64 = gemm_tiles(a, 64, 64);
  // one or two workgroups of T = 1 per compute unit, operands from HBM: DEEP /
  // T = 1 / T = 2 at 512 x 2048: K = 512 4.6 / 5.0 / 7.4 us, 1152 6.6 / 8.8 / 11.8,
  // 4096 12.5 / 21.9 / 26.6; at 1024 x 2048: 6.1 / 5.7 / 7.5, 9.0 / 9.2 / 11.5, 19.8 /
  // 22.8 / 26.7; at 2048 x 2048 (four) 10.0 / 7.7 / 8.0, 13.4 / 11.5 / 11.5, 37 / 37 / 28
  if (t64 <= 256 || (t64 <= 512 && kt >= 9)) return launch_ring<1, true>(p, s);
  const double c1 = cost<1>(t64, kt), c2 = cost<2>(gemm_tiles(a, 128, 128), kt),
               c4 = cost<4>(gemm_tiles(a, 256, 256), kt);
  // T = 4 has no registers left for the low-rank branch
  if (a.rank == 0 && c4 < c2 && c4 < c1) return launch_ring<4>(p, s);
  return c2 < c1 ? launch_ring<2>(p, s) : launch_ring<1>(p, s);
}

}  // namespace mxq
