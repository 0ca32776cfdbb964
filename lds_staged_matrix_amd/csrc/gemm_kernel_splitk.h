// gemm_kernel_splitk.h -- the 64 x 64 direct-to-LDS tile with K split over KS
// groups of four waves of one workgroup, for scaled products of few tiles.
//
// A product of a few hundred 64 x 64 tiles leaves a CU one or two workgroups
// of four waves, and each walks all of K at the latency of a load, a barrier
// and a few MFMAs a step (0.45 us for 128 k).  Here KS groups of four
// waves share the tile: group g takes K tiles g, g + KS, g + 2 KS, ... through
// LDS stages of its own, by the same loads, layouts and MFMAs as
// gemm_kernel_dma.h, so that KS steps run at once; the partial tiles meet in
// LDS and are added in group order, then scaled and stored.  Steps behind the
// end of K load zeros, so every group passes the same barriers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.h"
#include "gemm_kernel_dma.h"

namespace lsm {

template <class T, int LA, int LB, int IN, int OUT, int KS, int NS>
__global__ __launch_bounds__(KS * T::NT, KS / 2) void lds_gemm_splitk_kernel(
    const uint16_t *__restrict__ A, const uint16_t *__restrict__ B, void *__restrict__ C,
    int M, int N, int K, int64_t lda, int64_t ldb, int64_t ldc, int tiles_m, int tiles_n,
    uint32_t a_bytes, uint32_t b_bytes, int c_vec, RowColScale sc) {
  static_assert(is_e4m3(IN) && T::BM == 64 && T::BN == 64 && T::NT == 256, "64 x 64 tile of four waves, E4M3");
  constexpr int KSTEPS = T::BK / InT<IN>::KSTEP;
  using OA = OperandTile<T::BM, T::BK, LA, T::NT, 1>;
  using OB = OperandTile<T::BN, T::BK, LB, T::NT, 1>;
  using F = Frags<T, IN>;
  static_assert(KSTEPS % 2 == 0, "the register double buffer alternates two k-steps");
  constexpr int STAGE = OA::BYTES + OB::BYTES;
  constexpr int TILE_BYTES = T::BM * T::BN * 4;          // one group's partial tile, fp32
  constexpr int LPT = OA::LOADS + OB::LOADS;              // loads per thread and step
  static_assert(TILE_BYTES <= NS * STAGE, "the partial tiles reuse the stages");
  static_assert((NS == 2 || NS == 4) && KS * NS * STAGE <= 160 * 1024, "stages");
  __shared__ __attribute__((aligned(1024))) char smem[KS * NS * STAGE];

  if constexpr (LSM_LDS_POISON) {   // poison build: all of LDS, before any load or write
    lds_poison(smem, KS * NS * STAGE, threadIdx.x, blockDim.x);
    __syncthreads();
  }
  const int lane = threadIdx.x & 63;
  const int gtid = threadIdx.x & (T::NT - 1);            // thread in its group
  const int wave = __builtin_amdgcn_readfirstlane(gtid >> 6);
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / T::NT);
  const int wm = wave / T::WN, wn = wave % T::WN;

  int tm, tn;
  tile_coords(xcd_logical_id(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, T::GROUP_M, tm, tn);
  const int m0 = tm * T::BM, n0 = tn * T::BN;

  const i32x4 rsA = buffer_rsrc(A, a_bytes);
  const i32x4 rsB = buffer_rsrc(B, b_bytes);
  char *mine = smem + group * NS * STAGE;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)mine;

  int a_inner, b_inner;
  const uint32_t a_voff = dma_lane_offset<OA>(gtid, m0, M, lda, a_bytes, a_inner);
  const uint32_t b_voff = dma_lane_offset<OB>(gtid, n0, N, ldb, b_bytes, b_inner);
  const uint32_t a_round = (uint32_t)(OA::ROW_STEP * lda);
  const uint32_t b_round = (uint32_t)(OB::ROW_STEP * ldb);
  const uint32_t a_kstep = (uint32_t)(LA == KC ? T::BK : T::BK * lda);
  const uint32_t b_kstep = (uint32_t)(LB == KC ? T::BK : T::BK * ldb);
  const int KT = (K + T::BK - 1) / T::BK;
  const int steps = (KT + KS - 1) / KS;

  // This group's step i into its stage.
  auto issue = [&](int i) {
    const int kt = group + i * KS, k0 = kt * T::BK;
    uint32_t av = a_voff, bv = b_voff, at = (uint32_t)kt;
    if (kt >= KT) {                      // behind the end of K: zeros
      av = bv = kOutOfRange;
      at = 0;
    } else if (k0 + T::BK > K) {         // last, partial K tile: chunks at k >= K read as zero
      if constexpr (LA == KC) av = k0 + a_inner < K ? a_voff : kOutOfRange;
      if constexpr (LB == KC) bv = k0 + b_inner < K ? b_voff : kOutOfRange;
    }
    const uint32_t st = lds0 + (uint32_t)((i & (NS - 1)) * STAGE);
    dma_tile<OA, T::NT>(rsA, st, wave, av, at * a_kstep, a_round);
    dma_tile<OB, T::NT>(rsB, st + OA::BYTES, wave, bv, at * b_kstep, b_round);
  };

  v16f32 acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; i++)
#pragma unroll
    for (int j = 0; j < T::FN; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.f;

  F cur, nxt;
  if (steps > 0) {
    const int first = steps < NS ? steps : NS;
    for (int i = 0; i < first; ++i) issue(i);
    wait_tiles<LPT>(first - 1);
    __syncthreads();                     // step 0 is in stage 0
    read_frags<T, IN, OA, OB>(cur, mine, mine + OA::BYTES, lane, wm, wn, 0);
  }
  for (int i = 0; i < steps; ++i) {
    const char *sA = mine + (i & (NS - 1)) * STAGE, *sB = sA + OA::BYTES;
#pragma unroll
    for (int kk = 0; kk + 1 < KSTEPS; kk += 2) {
      read_frags<T, IN, OA, OB>(nxt, sA, sB, lane, wm, wn, kk + 1);
      mfma_block<T, IN>(acc, cur);
      if (kk + 2 < KSTEPS) {
        read_frags<T, IN, OA, OB>(cur, sA, sB, lane, wm, wn, kk + 2);
        mfma_block<T, IN>(acc, nxt);
      }
    }
#pragma unroll
    for (int x = 0; x < T::FM; x++)
#pragma unroll
      for (int j = 0; j < T::FN; j++) pin_acc(acc[x][j]);
    if (i + 1 < steps) {
      // step i+1 landed; steps i+2 .. i+NS-1 may still be in flight
      wait_tiles<LPT>(steps - i - 2 < NS - 2 ? steps - i - 2 : NS - 2);
      __syncthreads();                   // step i+1 is in its stage; step i's is free
      const char *nA = mine + ((i + 1) & (NS - 1)) * STAGE;
      read_frags<T, IN, OA, OB>(cur, nA, nA + OA::BYTES, lane, wm, wn, 0);
      if (i + NS < steps) issue(i + NS);
    }
    mfma_block<T, IN>(acc, nxt);
  }

  // The partial tiles, row-major, the 32-column halves of every other four
  // rows exchanged: the two rows that one write of an accumulator register
  // covers are four apart and land in different banks.
  __syncthreads();                       // every wave is past its last LDS read
  if constexpr (LSM_LDS_POISON) {   // poison build: the sums' region, before its writes
    lds_poison(smem, KS * TILE_BYTES, threadIdx.x, blockDim.x);
    __syncthreads();
  }
  auto at = [](int row, int col) { return row * T::BN + (col ^ (((row >> 2) & 1) << 5)); };
  float *red = (float *)smem;
  using L = AccLayout<32>;
#pragma unroll
  for (int i = 0; i < T::FM; i++)
#pragma unroll
    for (int j = 0; j < T::FN; j++)
#pragma unroll
      for (int r = 0; r < L::R; r++)
        red[group * (TILE_BYTES / 4) + at(wm * T::TM + 32 * i + L::row(r, lane), wn * T::TN + 32 * j + L::col(lane))] =
            acc[i][j][r];
  __syncthreads();
  typedef typename OutElem<OUT>::type E;
  typedef E e4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int q = 0; q < T::BM * T::BN / 4 / (KS * T::NT); q++) {
    const int e = (int)threadIdx.x + q * KS * T::NT;     // four columns of one row
    const int row = e / (T::BN / 4), col = 4 * (e % (T::BN / 4));
    v4f32 v = *(const v4f32 *)(red + at(row, col));
#pragma unroll
    for (int g = 1; g < KS; g++) v += *(const v4f32 *)(red + g * (TILE_BYTES / 4) + at(row, col));
    const int m = m0 + row, n = n0 + col;
    if (m >= M) continue;
    e4 o;
#pragma unroll
    for (int x = 0; x < 4; x++) o[x] = (E)scale_entry(v[x], m, n + x, M, N, sc);
    E *dst = (E *)C + (int64_t)m * ldc + n;
    if (c_vec && n + 4 <= N) {
      *(e4 *)dst = o;
    } else {
#pragma unroll
      for (int x = 0; x < 4; x++)
        if (n + x < N) dst[x] = o[x];
    }
  }
}

}  // namespace lsm
