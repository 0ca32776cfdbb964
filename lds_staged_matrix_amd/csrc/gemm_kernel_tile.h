// gemm_kernel_tile.h -- smaller tiles of the grouped and of the MXFP4 products.
//
// lds_gemm_tile_kernel: WM x WN waves on one tile of BM x BN; a K tile (128
// bytes of either operand's rows, see gemm_tile.h) comes into one of NS LDS
// stages, NS - 1 of them in flight, one barrier a K tile.  With WK > 1 so many
// groups of waves take turns at the K tiles, each with stages of its own: for
// tiles too few to fill the chip, whose time is the length of the K loop.
//
// lds_gemm_stream_kernel: few rows, so that the time is that of reading B once.
// The workgroup's waves split K, slab by slab of 128 bytes, and each keeps a ring
// of LDS stages of its own: a wave waits for its own loads and no barrier stands
// in the loop.  Neighbouring waves read neighbouring slabs, whole lines of every
// row.  Each XCD starts at its own eighth of K (see rows_start in
// gemm_kernel_rows.h for what that is worth).
//
// Both add the waves' tiles, or the one tile, through LDS in wave order and store
// four consecutive columns a thread.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_tile.h"

namespace lsm {

// ------------------------------------------------------------ scales (MXFP4)
//
// The scales of `rows` rows and a K tile's 8 blocks in LDS: CH 16-byte pieces a
// block.  The first row need not stand at a multiple of 16 in the scales' rows:
// the pieces then start at the multiple before it, and one more holds the end.
template <int ROWS, bool SHIFTED>
struct ScaleTile {
  static constexpr int CH = ROWS / 16 + (SHIFTED ? 1 : 0);
  static constexpr int CHUNKS = kScaleRows * CH;
  static constexpr int INSTS = (CHUNKS + 63) / 64;                 // wave loads
  static constexpr int BYTES = INSTS > 1 ? INSTS * 1024 : CHUNKS * 16;
  uint64_t base;
  int64_t bytes;
  uint32_t ld;
  int shift;

  // `n` rows from `first` on, `blocks` blocks of k.
  __device__ __forceinline__ ScaleTile(const char *first, int64_t ld_, int n, int blocks) {
    shift = SHIFTED ? (int)((uint64_t)first & 15) : 0;
    base = (uint64_t)first - shift;
    ld = (uint32_t)ld_;
    const int width = n + shift < 16 * CH ? (n + shift + 15) & ~15 : 16 * CH;
    bytes = span_bytes(blocks, ld_, width);
  }
  // Wave load `inst` of K tile kt; only as many lanes as there are pieces.
  __device__ __forceinline__ void issue(uint32_t lds, int kt, int inst, int lane) const {
    const int64_t done = (int64_t)kt * kScaleRows * ld;
    const i32x4 rs = rest_rsrc(base + done, bytes - done);
    const int slot = 64 * inst + lane;
    const uint32_t off = (uint32_t)(slot / CH) * ld + 16 * (slot % CH);
    if (CHUNKS % 64 == 0 || slot < CHUNKS) dma16(rs, lds + (uint32_t)(1024 * inst), off, 0);
  }
  // The scale of row `row`, block kb of the K tile.
  __device__ __forceinline__ int read(const char *lds, int kb, int row) const {
    return *(const uint8_t *)(lds + kb * 16 * CH + shift + row);
  }
};

// ------------------------------------------------------------------ results

// WAVES partial tiles of BM x BN, each spread over lanes as the 16 x 16 MFMAs
// leave it, added in order and stored.  `wave` holds part `part`, rows r0.. and
// columns c0.. of the tile.  Needs PARTS * BM * BN * 4 bytes of LDS that no load
// targets any more; every thread of the workgroup calls it.
template <int BM, int BN, int PARTS, int OUT, int FM, int FN>
__device__ __forceinline__ void add_and_store(void *C, const v4f32 (&acc)[FM][FN], char *smem, const Where &w,
                                              int64_t ldc, int part, int r0, int c0, int lane, int threads) {
  // columns of a row in blocks of 16, XORed by the row so that the four rows of
  // one write lie in different banks
  auto at = [](int row, int col) { return row * BN + (col ^ (16 * ((row >> 2) & (BN >= 64 ? 3 : BN / 16 - 1)))); };
  float *red = (float *)smem;
  __syncthreads();                                       // every wave is done with the stages
  if constexpr (LSM_LDS_POISON) {   // poison build: the sums' region, before its writes
    lds_poison(smem, PARTS * BM * BN * 4, threadIdx.x, threads);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++)
#pragma unroll
      for (int r = 0; r < 4; r++)
        red[part * BM * BN + at(r0 + 16 * i + 4 * (lane >> 4) + r, c0 + 16 * j + (lane & 15))] = acc[i][j][r];
  __syncthreads();
  for (int e = threadIdx.x; e < BM * BN / 4; e += threads) {
    const int row = e / (BN / 4), col = 4 * (e % (BN / 4));
    if (row < w.skip || row >= w.rows || col >= w.cols) continue;
    v4f32 v = *(const v4f32 *)(red + at(row, col));
#pragma unroll
    for (int q = 1; q < PARTS; q++) v += *(const v4f32 *)(red + q * BM * BN + at(row, col));
    store4<OUT>(C, w.c + row * ldc + col, v, w.cols - col);
  }
}

// One k-step's products; `ga`, `gb`: the fragments' scales.
template <int IN, int FM, int FN>
__device__ __forceinline__ void tile_mfma(v4f32 (&acc)[FM][FN], const v8i16 (&a)[FM], const v8i16 (&b)[FN],
                                          const int (&ga)[FM], const int (&gb)[FN]) {
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) {
      if constexpr (IN == IN_MXFP4)
        acc[i][j] = mfma_mxfp4<0, 0>(a[i], b[j], acc[i][j], ga[i], gb[j]);
      else
        acc[i][j] = mfma_16x16x32<IN>(a[i], b[j], acc[i][j]);
    }
}

// ------------------------------------------------------------------- tiles

template <int BM_, int BN_, int WM_, int WN_, int NS_, int WK_ = 1>
struct TileShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_, WK = WK_, GROUP_M = 8;
  static constexpr int NT = 64 * WM * WN;                // of one group
  static constexpr int PER_CU = 160 * 1024 / (NS * WK * (BM + BN) * kTileBytes);     // workgroups, by their LDS
};

template <class S, int MODE, int LA, int LB, int IN, int OUT>
__global__ __launch_bounds__(S::NT * S::WK, 2) void lds_gemm_tile_kernel(const TileArgs p) {
  constexpr bool MX = IN == IN_MXFP4;
  constexpr int BM = S::BM, BN = S::BN, NS = S::NS, NT = S::NT, WK = S::WK, EB = MX ? 1 : 2;
  constexpr int TM = BM / S::WM, TN = BN / S::WN, FM = TM / 16, FN = TN / 16, KSTEPS = 2;
  using OA = TileOf<BM, LA, NT, EB>;
  using OB = TileOf<BN, LB, NT, EB>;
  using GA = ScaleTile<BM, MODE == GROUP_ROWS>;
  using GB = ScaleTile<BN, false>;
  constexpr int SA_AT = OA::BYTES + OB::BYTES, SB_AT = SA_AT + GA::BYTES;
  constexpr int STAGE = SA_AT + (MX ? (GA::BYTES + GB::BYTES + 1023) / 1024 * 1024 : 0);
  constexpr int LPT = OA::LOADS + OB::LOADS, SCALE_LOADS = MX ? GA::INSTS + GB::INSTS : 0;
  constexpr int LDS_BYTES = WK * (NS * STAGE > BM * BN * 4 ? NS * STAGE : BM * BN * 4);
  static_assert(SCALE_LOADS <= S::WM * S::WN && (NS - 2) * (LPT + 1) < 64 && LDS_BYTES <= 160 * 1024, "stages");
  __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];

  const int tid = threadIdx.x & (NT - 1), lane = tid & 63;
  if constexpr (LSM_LDS_POISON) {   // poison build: all of LDS, before any load or write
    lds_poison(smem, LDS_BYTES, threadIdx.x, NT * WK);
    __syncthreads();
  }
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wk = WK == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
  const int wm = wave / S::WN, wn = wave % S::WN;
  Where w{};
  if (!locate<BM, BN, S::GROUP_M, MODE, LA, LB, IN, 1>(p, lane, w)) return;
  const int KT = (w.K + kTileK(IN) - 1) / kTileK(IN);
  const int kbytes = MX ? w.K / 2 : 2 * w.K;
  char *stages = smem + wk * NS * STAGE;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)stages;
  const Loader<OA, NT> la(tid, w.a, p.lda, LA == KC ? w.rows : 2 * w.rows, LA == KC ? kbytes : w.K);
  const Loader<OB, NT> lb(tid, w.b, p.ldb, LB == KC ? w.cols : 2 * w.cols, LB == KC ? kbytes : w.K);
  const GA sa(w.sa, p.ldsa, w.rows, w.K / kMxBlock);
  const GB sb(w.sb, p.ldsb, w.cols, w.K / kMxBlock);

  // The group's K tile i, counted from the XCD's start, into stage `st`; behind the
  // last, zeros, so that a K tile is always as many loads.
  const int start = LA == KC ? (int)((uint32_t)(blockIdx.x & 7) * (uint32_t)KT >> 3) : 0;
  auto issue = [&](int i, int st) {
    const int at_k = i * WK + wk, on = at_k + start;
    const int kt = at_k >= KT ? KT : on < KT ? on : on - KT;
    const uint32_t at = lds0 + (uint32_t)(st * STAGE);
    const auto ra = la.at(kt, kbytes);
    const auto rb = lb.at(kt, kbytes);
#pragma unroll
    for (int d = 0; d < OA::LOADS; d++) la.issue(ra, at, wave, d);
#pragma unroll
    for (int d = 0; d < OB::LOADS; d++) lb.issue(rb, at + OA::BYTES, wave, d);
    if constexpr (MX) {
      if (wave < GA::INSTS)
        sa.issue(at + SA_AT, kt, wave, lane);
      else if (wave < SCALE_LOADS)
        sb.issue(at + SB_AT, kt, wave - GA::INSTS, lane);
    }
  };

  v4f32 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = v4f32{0.f, 0.f, 0.f, 0.f};

  if (KT > 0) {
#pragma unroll
    for (int t = 0; t < NS - 1; t++) issue(t, t);
    int st = 0, free = NS - 1;
    for (int i = 0; i * WK < KT; ++i) {
      // the group's K tile i landed (this wave's part: NS - 2 later ones may be in flight) ...
      if (wave < SCALE_LOADS)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * (LPT + 1)) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * LPT) : "memory");
      __syncthreads();                                   // ... every wave's, and the stage before it is read
      issue(i + NS - 1, free);
      const char *sA = stages + st * STAGE, *sB = sA + OA::BYTES;
#pragma unroll
      for (int kk = 0; kk < KSTEPS; kk++) {
        v8i16 fa[FM], fb[FN];
        int ga[FM], gb[FN];
#pragma unroll
        for (int q = 0; q < FM; q++) {
          fa[q] = read_tile_frag<OA>(sA, lane, wm * TM + 16 * q, kk);
          ga[q] = MX ? sa.read(sA + SA_AT, 4 * kk + (lane >> 4), wm * TM + 16 * q + (lane & 15)) : 0;
        }
#pragma unroll
        for (int q = 0; q < FN; q++) {
          fb[q] = read_tile_frag<OB>(sB, lane, wn * TN + 16 * q, kk);
          gb[q] = MX ? sb.read(sA + SB_AT, 4 * kk + (lane >> 4), wn * TN + 16 * q + (lane & 15)) : 0;
        }
        tile_mfma<IN>(acc, fa, fb, ga, gb);
      }
      st = st + 1 == NS ? 0 : st + 1;
      free = free + 1 == NS ? 0 : free + 1;
    }
    wait_dma();                                          // no load still targets the LDS
  }
  add_and_store<BM, BN, WK, OUT>(p.C, acc, smem, w, p.ldc, wk, wm * TM, wn * TN, lane, NT * WK);
}

// ------------------------------------------------------------------ streams

template <int BM_, int BN_, int WAVES_, int NS_>
struct StreamShape {
  static constexpr int BM = BM_, BN = BN_, WAVES = WAVES_, NS = NS_, GROUP_M = 8;
};

template <class S, int MODE, int LB, int IN, int OUT>
__global__ __launch_bounds__(64 * S::WAVES, 2) void lds_gemm_stream_kernel(const TileArgs p) {
  constexpr bool MX = IN == IN_MXFP4;
  constexpr int BM = S::BM, BN = S::BN, NS = S::NS, WAVES = S::WAVES, FM = BM / 16, FN = BN / 16, KSTEPS = 2;
  using OA = SlabTile<BM, KC, 64>;
  using OB = SlabTile<BN, LB, 64>;
  using GA = ScaleTile<BM, MODE == GROUP_ROWS>;
  using GB = ScaleTile<BN, false>;
  constexpr int SA_AT = OA::BYTES + OB::BYTES, SB_AT = SA_AT + GA::BYTES;
  constexpr int SLAB = SA_AT + (MX ? GA::BYTES + GB::BYTES : 0);
  constexpr int LOADS = OA::LOADS + OB::LOADS + (MX ? GA::INSTS + GB::INSTS : 0);
  constexpr int LDS_BYTES = WAVES * (NS * SLAB > BM * BN * 4 ? NS * SLAB : BM * BN * 4);
  static_assert((NS - 1) * LOADS < 64 && LDS_BYTES <= 160 * 1024, "rings");
  __shared__ __attribute__((aligned(1024))) char smem[LDS_BYTES];

  const int lane = threadIdx.x & 63;
  if constexpr (LSM_LDS_POISON) {   // poison build: all of LDS, before any load or write
    lds_poison(smem, LDS_BYTES, threadIdx.x, 64 * WAVES);
    __syncthreads();
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Where w{};
  if (!locate<BM, BN, S::GROUP_M, MODE, KC, LB, IN, 1>(p, lane, w)) return;
  const int KT = (w.K + kTileK(IN) - 1) / kTileK(IN);
  const int kbytes = MX ? w.K / 2 : 2 * w.K;
  const Loader<OA, 64> la(lane, w.a, p.lda, w.rows, kbytes);
  const Loader<OB, 64> lb(lane, w.b, p.ldb, LB == KC ? w.cols : 2 * w.cols, LB == KC ? kbytes : w.K);
  const GA sa(w.sa, p.ldsa, w.rows, w.K / kMxBlock);
  const GB sb(w.sb, p.ldsb, w.cols, w.K / kMxBlock);
  char *ring = smem + wave * NS * SLAB;
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)ring;

  // Slab i of this wave: K tile wave + WAVES * i, counted from the XCD's start.
  const int mine = KT > wave ? (KT - wave + WAVES - 1) / WAVES : 0;
  const int start = (int)((uint32_t)(blockIdx.x & 7) * (uint32_t)mine >> 3);
  auto issue = [&](int i, int st) {
    // behind the last, a tile behind K: zeros, so that a slab is always as many loads
    const int at = i + start < mine ? i + start : i + start - mine;
    const int kt = i < mine ? wave + WAVES * at : KT;
    const uint32_t to = lds + (uint32_t)(st * SLAB);
    const auto ra = la.at(kt, kbytes);
    const auto rb = lb.at(kt, kbytes);
#pragma unroll
    for (int d = 0; d < OB::LOADS; d++) lb.issue(rb, to + OA::BYTES, 0, d);
#pragma unroll
    for (int d = 0; d < OA::LOADS; d++) la.issue(ra, to, 0, d);
    if constexpr (MX) {
#pragma unroll
      for (int d = 0; d < GA::INSTS; d++) sa.issue(to + SA_AT, kt, d, lane);
#pragma unroll
      for (int d = 0; d < GB::INSTS; d++) sb.issue(to + SB_AT, kt, d, lane);
    }
  };

  v4f32 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = v4f32{0.f, 0.f, 0.f, 0.f};

  if (mine > 0) {
#pragma unroll
    for (int t = 0; t < NS; t++) issue(t, t);
    int st = 0;
    for (int i = 0; i < mine; i++) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 1) * LOADS) : "memory");      // slab i landed
      const char *sA = ring + st * SLAB, *sB = sA + OA::BYTES;
      v8i16 fa[KSTEPS][FM], fb[KSTEPS][FN];
      int ga[KSTEPS][FM], gb[KSTEPS][FN];
#pragma unroll
      for (int kk = 0; kk < KSTEPS; kk++) {
#pragma unroll
        for (int q = 0; q < FM; q++) {
          fa[kk][q] = read_tile_frag<OA>(sA, lane, 16 * q, kk);
          ga[kk][q] = MX ? sa.read(sA + SA_AT, 4 * kk + (lane >> 4), 16 * q + (lane & 15)) : 0;
        }
#pragma unroll
        for (int q = 0; q < FN; q++) {
          fb[kk][q] = read_tile_frag<OB>(sB, lane, 16 * q, kk);
          gb[kk][q] = MX ? sb.read(sA + SB_AT, 4 * kk + (lane >> 4), 16 * q + (lane & 15)) : 0;
        }
      }
      wait_lds_reads();                                  // the slab is free
      issue(i + NS, st);
#pragma unroll
      for (int kk = 0; kk < KSTEPS; kk++) tile_mfma<IN>(acc, fa[kk], fb[kk], ga[kk], gb[kk]);
      st = st + 1 == NS ? 0 : st + 1;
    }
    wait_dma();                                          // no load still targets the LDS
  }
  add_and_store<BM, BN, WAVES, OUT>(p.C, acc, smem, w, p.ldc, wave, 0, 0, lane, 64 * WAVES);
}

}  // namespace lsm
