// gemm_kernel_dma.h -- the LDS-staged GEMM kernel with direct global->LDS
// loads, for gfx950.
//
// Operand tiles move from HBM straight into LDS with
// `buffer_load_dwordx4 ... lds`: no VGPR staging and no ds_write.  This is the
// asynchronous direct-to-LDS fill of "An educational GEMM ladder for Helios
// GPUs", "Level 2: Asynchronous HBM Loads", on gfx950's LDS-DMA form of the
// buffer load.  The hardware writes lane L's 16 bytes to LDS slot L of the
// instruction's 1 KiB block (M0 holds the block address), which has two
// consequences:
//  * The XOR swizzle moves to the global side.  Lane L fills physical chunk
//    p = L mod (chunks per row) of its row, so it loads logical chunk
//    p XOR swizzle(row) from memory.  The LDS image is the same swizzled
//    layout the register-staged kernel writes, and it is read back the same
//    way.
//  * Edges cost nothing.  The buffer descriptor's record count is the
//    operand's exact footprint, so rows past the matrix read as zero.  Chunks
//    past the contiguous extent get an offset beyond the record count and
//    read as zero too.  Whole chunks only: the contiguous extents must be
//    multiples of 8 elements, and the host sends other shapes to the
//    register-staged kernel.
//
// The loads are issued with inline assembly.  The compiler's builtin form is
// tracked by its wait-count pass, which cannot tell that the in-flight loads
// target the other LDS stage and makes every ds_read_b64_tr_b16 wait for all
// of them.  Here the kernel orders the loads itself:
//   "s_waitcnt vmcnt(0)" + s_barrier publishes a stage before any wave
//   reads it, and no load targets a stage until the barrier after the last
//   read of that stage.
//
// Pipeline, two LDS stages (t = K tile, s = t & 1):
//   for each k-step kk < last: read fragments of kk+1 (stage s) while the
//                              MFMAs of kk run (register double buffer,
//                              "Level 5: Deepening the K Stride");
//   last k-step:  wait own loads, barrier (tile t+1 is in stage s^1 and
//                 stage s is free), read fragments of kk=0 from stage s^1,
//                 start the loads of tile t+2 into stage s, then run the
//                 MFMAs of the last kk from registers.
// The barrier therefore sits after the last LDS read of a stage and before
// the last MFMAs that need no LDS ("Level 8: Using Split Barriers": signal
// after the final LDS read, finish the register-only MFMAs, then continue).
// Loads of tile t+2 have one K step (64 MFMAs per wave) to land.
//
// Wave tile 128 x 128 with 4 waves, one per SIMD: each k-step of 16 reads
// 8 fragments (8 KiB) for 16 MFMAs, 2/3 of the LDS read traffic per flop of a
// 128 x 64 wave tile.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.h"

namespace lsm {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Buffer resource word 3 for gfx9-family raw buffers (32-bit data format,
// no swizzle, stride 0): byte offsets are range-checked against num_records.
constexpr uint32_t kBufferWord3 = 0x00020000u;
// An offset that is always past the record count (footprints stay below 2^31).
constexpr uint32_t kOutOfRange = 0x80000000u;

__device__ __forceinline__ i32x4 buffer_rsrc(const void *base, uint32_t bytes) {
  const uint64_t a = (uint64_t)base;
  i32x4 r;
  r[0] = (int)(uint32_t)a;
  r[1] = (int)((a >> 32) & 0xFFFFu);   // base[47:32]; stride 0
  r[2] = (int)bytes;                    // num_records
  r[3] = (int)kBufferWord3;
  return r;
}

// One 16-byte-per-lane direct-to-LDS load: lane L's bytes at
// base + voff + soff land at LDS byte address lds_block + 16*L.
// The compiler reserves M0 and warns when asm clobbers it.  In these kernels
// no compiler-generated instruction reads M0 (gfx950 LDS instructions do not
// use it), and every asm statement sets M0 right before the load that uses it.
// A scalar write of M0 needs one wait state before an LDS-DMA load reads it
// (the compiler inserts the same s_nop for its own buffer-load-to-LDS
// builtin on gfx9-family targets); its hazard check does not look inside asm.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(i32x4 rsrc, uint32_t lds_block, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :
               : "s"(lds_block), "v"(voff), "s"(rsrc), "s"(soff)
               : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ void wait_dma() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Issue this wave's loads of one operand tile.  Round i of the workgroup
// covers chunk slots [i*NT, (i+1)*NT); this wave fills the 1 KiB block at
// slot i*NT + 64*wave.
template <class OT, int NT>
__device__ __forceinline__ void dma_tile(i32x4 rs, uint32_t lds_tile, int wave, uint32_t voff,
                                         uint32_t soff, uint32_t round_step) {
#pragma unroll
  for (int i = 0; i < OT::LOADS; i++)
    dma16(rs, lds_tile + (uint32_t)((i * NT + 64 * wave) * 16), voff, soff + i * round_step);
}

// Byte offset, from the operand's base, of this thread's round-0 chunk in K
// tile 0, or kOutOfRange when the chunk lies outside the matrix.
//   K-contiguous:  row = M/N index (mn0 + row), inner = k
//   MN-contiguous: row = k index, inner = M/N index (mn0 + inner)
// `phase` = 1 gives the offset for the load rounds with OT::round_phase(d) = 1
// of a tile that takes two lane offsets (OT::LANE_OFFSETS == 2): the same row
// and slot, with the swizzle of the row OT::PHASE_ROWS rows further on.
template <class OT>
__device__ __forceinline__ uint32_t dma_lane_offset(int tid, int mn0, int mn_ext, int64_t ld,
                                                    uint32_t bytes, int &inner_out, int phase = 0) {
  const int row = loader_row(tid, OT::ROW_BYTES);
  const int pchunk = loader_chunk(tid, OT::ROW_BYTES);
  const int lchunk = pchunk ^ OT::swizzle(row + phase * OT::PHASE_ROWS);
  const int inner = OT::EPC * lchunk;                 // first element of the chunk
  inner_out = inner;
  int64_t off;
  if constexpr (OT::kcontig) {
    off = ((int64_t)(mn0 + row) * ld + inner) * OT::ES;
  } else {
    if (mn0 + inner >= mn_ext) return kOutOfRange;
    off = ((int64_t)row * ld + mn0 + inner) * OT::ES;
  }
  return off < (int64_t)bytes ? (uint32_t)off : kOutOfRange;
}

template <class T, int IN>
struct Frags {
  typename InT<IN>::frag a[T::FM], b[T::FN];
};

// Reads in the order the MFMAs (row-fragment major) consume them: a[0] with
// every b[j] first, then the remaining a[i].
template <class T, int IN, class OA, class OB>
__device__ __forceinline__ void read_frags(Frags<T, IN> &f, const char *sA, const char *sB,
                                           int lane, int wm, int wn, int kk) {
  f.a[0] = read_frag_in<OA, IN>(sA, lane, wm * T::TM, kk);
#pragma unroll
  for (int j = 0; j < T::FN; j++) f.b[j] = read_frag_in<OB, IN>(sB, lane, wn * T::TN + 32 * j, kk);
#pragma unroll
  for (int i = 1; i < T::FM; i++) f.a[i] = read_frag_in<OA, IN>(sA, lane, wm * T::TM + 32 * i, kk);
}

template <class T, int IN>
__device__ __forceinline__ void mfma_block(v16f32 (&acc)[T::FM][T::FN], const Frags<T, IN> &f) {
  if constexpr (IN == IN_E4M3_AS_BF16) {
    mfma_e4m3_as_bf16<32>(acc, f.a, f.b);
  } else {
#pragma unroll
    for (int i = 0; i < T::FM; i++)
#pragma unroll
      for (int j = 0; j < T::FN; j++) acc[i][j] = mfma_step<IN>(f.a[i], f.b[j], acc[i][j]);
  }
}

// Interleave the LDS reads of the next k-step with the MFMAs of this one:
// one MFMA, then one ds_read, until the reads run out.
template <int MFMAS, int READS>
__device__ __forceinline__ void interleave_reads_with_mfma() {
#pragma unroll
  for (int q = 0; q < MFMAS; q++) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // one MFMA
    if (q < READS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // one DS read
  }
}

// LSM_DMA_STAGES = 1 builds this kernel with a single LDS stage: every K
// tile is loaded, waited for and only then computed, with no overlap of the
// loads and the MFMAs.  It exists only for the A/B build that measures what
// the double-buffered pipeline buys; the library is built with 2.
#ifndef LSM_DMA_STAGES
#define LSM_DMA_STAGES 2
#endif

// C stores: with 16-byte aligned C rows the kernel stages C through LDS for
// the whole workgroup (epilogue_lds_rows: each store writes whole rows of the
// workgroup tile, 128-512 bytes); LSM_DMA_ROW_EPI = 0, an A/B build only,
// stages the 128 x 128 tile per wave (epilogue_lds) and stores the 64 x 64
// tile straight from the accumulators.
#ifndef LSM_DMA_ROW_EPI
#define LSM_DMA_ROW_EPI 1
#endif

// Wait until at most `n` (0..3) K tiles' loads, LPT per thread each, are
// still in flight (loads complete in issue order).
template <int LPT>
__device__ __forceinline__ void wait_tiles(int n) {
  if (n <= 0) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  else if (n == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LPT) : "memory");
  else if (n == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * LPT) : "memory");
  else asm volatile("s_waitcnt vmcnt(%0)" ::"n"(3 * LPT) : "memory");
}

// NS = number of LDS stages: 2 (double buffer), or 4 for a K loop whose
// operand panels overflow the L2 and come from further out: then the loads
// of tile kt+4 go out as soon as tile kt's stage is free, three tiles ahead
// of their use instead of one.
// SC is empty, or RowColScale for a product whose rows and columns are scaled.
template <class T, int LA, int LB, int IN, int OUT, int NS = 2, class... SC>
__global__ __launch_bounds__(T::NT, 1) void lds_gemm_dma_kernel(
    const uint16_t *__restrict__ A, const uint16_t *__restrict__ B, void *__restrict__ C,
    int M, int N, int K, int64_t lda, int64_t ldb, int64_t ldc, int tiles_m, int tiles_n,
    uint32_t a_bytes, uint32_t b_bytes, int c_vec, SC... sc) {
  constexpr int ES = InT<IN>::ES;
  constexpr int KSTEPS = T::BK / InT<IN>::KSTEP;          // MFMA k-steps per K tile
  using OA = OperandTile<T::BM, T::BK, LA, T::NT, ES>;
  using OB = OperandTile<T::BN, T::BK, LB, T::NT, ES>;
  using F = Frags<T, IN>;
  static_assert(KSTEPS % 2 == 0, "the register double buffer alternates two k-steps");
  constexpr int STAGE = OA::BYTES + OB::BYTES;
  constexpr int STAGES = LSM_DMA_STAGES == 1 ? 1 : NS;
  static_assert(STAGES == 1 || STAGES == 2 || STAGES == 4, "one, two or four LDS stages");
  constexpr int LPT = OA::LOADS + OB::LOADS;              // loads per thread and K tile
  static_assert(3 * LPT <= 63, "vmcnt counts up to 63");
  constexpr int READS = T::FM * frag_reads<OA, IN>() + T::FN * frag_reads<OB, IN>();
  __shared__ __attribute__((aligned(1024))) char smem[STAGES * STAGE];

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  if constexpr (LSM_LDS_POISON) {   // poison build: all of LDS, before any load or write
    lds_poison(smem, STAGES * STAGE, tid, blockDim.x);
    __syncthreads();
  }
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / T::WN, wn = wave % T::WN;

  int tm, tn;
  tile_coords(xcd_logical_id(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, T::GROUP_M, tm, tn);
  const int m0 = tm * T::BM, n0 = tn * T::BN;

  const i32x4 rsA = buffer_rsrc(A, a_bytes);
  const i32x4 rsB = buffer_rsrc(B, b_bytes);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem;

  int a_inner, b_inner;
  const uint32_t a_voff = dma_lane_offset<OA>(tid, m0, M, lda, a_bytes, a_inner);
  const uint32_t b_voff = dma_lane_offset<OB>(tid, n0, N, ldb, b_bytes, b_inner);
  // Advance per load round (ROW_STEP rows) and per K tile, in bytes.
  const uint32_t a_round = (uint32_t)(OA::ROW_STEP * lda * ES);
  const uint32_t b_round = (uint32_t)(OB::ROW_STEP * ldb * ES);
  const uint32_t a_kstep = (uint32_t)(LA == KC ? ES * T::BK : ES * T::BK * lda);
  const uint32_t b_kstep = (uint32_t)(LB == KC ? ES * T::BK : ES * T::BK * ldb);

  auto issue = [&](int kt) {
    const uint32_t st = lds0 + (uint32_t)((kt & (STAGES - 1)) * STAGE);
    const int k0 = kt * T::BK;
    uint32_t av = a_voff, bv = b_voff;
    if (k0 + T::BK > K) {   // last, partial K tile: chunks at k >= K read as zero
      if constexpr (LA == KC) av = k0 + a_inner < K ? a_voff : kOutOfRange;
      if constexpr (LB == KC) bv = k0 + b_inner < K ? b_voff : kOutOfRange;
    }
    dma_tile<OA, T::NT>(rsA, st, wave, av, (uint32_t)kt * a_kstep, a_round);
    dma_tile<OB, T::NT>(rsB, st + OA::BYTES, wave, bv, (uint32_t)kt * b_kstep, b_round);
  };

  v16f32 acc[T::FM][T::FN];
#pragma unroll
  for (int i = 0; i < T::FM; i++)
#pragma unroll
    for (int j = 0; j < T::FN; j++)
#pragma unroll
      for (int r = 0; r < 16; r++) acc[i][j][r] = 0.f;

  const int KT = (K + T::BK - 1) / T::BK;
  F cur, nxt;
  if constexpr (STAGES == 1) {
    // Load, wait, compute, in turn: the loads of tile kt+1 start only when
    // every wave has read tile kt.
    if (KT > 0) issue(0);
    for (int kt = 0; kt < KT; ++kt) {
      wait_dma();
      __syncthreads();                     // tile kt is in the stage
      read_frags<T, IN, OA, OB>(cur, smem, smem + OA::BYTES, lane, wm, wn, 0);
#pragma unroll
      for (int kk = 0; kk + 1 < KSTEPS; kk += 2) {
        read_frags<T, IN, OA, OB>(nxt, smem, smem + OA::BYTES, lane, wm, wn, kk + 1);
        mfma_block<T, IN>(acc, cur);
        if (kk + 2 < KSTEPS) read_frags<T, IN, OA, OB>(cur, smem, smem + OA::BYTES, lane, wm, wn, kk + 2);
        mfma_block<T, IN>(acc, nxt);
      }
      __syncthreads();                     // every wave is done with the stage
      if (kt + 1 < KT) issue(kt + 1);
    }
  } else {
  if (KT > 0) {
    if constexpr (STAGES == 2) {
      issue(0);
      wait_dma();
      __syncthreads();                     // tile 0 is in stage 0
      if (KT > 1) issue(1);                // tile 1 -> stage 1, lands during step 0
    } else {
      const int pro = KT < STAGES ? KT : STAGES;   // tiles 0 .. pro-1, one per stage
      for (int t = 0; t < pro; ++t) issue(t);
      wait_tiles<LPT>(pro - 1);            // tile 0 landed, the others may be in flight
      __syncthreads();                     // tile 0 is in stage 0
    }
    read_frags<T, IN, OA, OB>(cur, smem, smem + OA::BYTES, lane, wm, wn, 0);
  }

  for (int kt = 0; kt < KT; ++kt) {
    const char *sA = smem + (kt & (STAGES - 1)) * STAGE;
    const char *sB = sA + OA::BYTES;
#pragma unroll
    for (int kk = 0; kk + 1 < KSTEPS; kk += 2) {
      read_frags<T, IN, OA, OB>(nxt, sA, sB, lane, wm, wn, kk + 1);
      mfma_block<T, IN>(acc, cur);
      interleave_reads_with_mfma<T::FM * T::FN, READS>();
      if (kk + 2 < KSTEPS) {
        read_frags<T, IN, OA, OB>(cur, sA, sB, lane, wm, wn, kk + 2);
        mfma_block<T, IN>(acc, nxt);
        interleave_reads_with_mfma<T::FM * T::FN, READS>();
      }
    }
    // `nxt` holds the last k-step of this stage (KSTEPS is even).  The MFMAs
    // issued so far run while this wave waits for the next tile (with two
    // k-steps per tile the compiler would otherwise sink them past the wait).
    if constexpr (KSTEPS == 2) {
#pragma unroll
      for (int i = 0; i < T::FM; i++)
#pragma unroll
        for (int j = 0; j < T::FN; j++) pin_acc(acc[i][j]);
    }
    if (kt + 1 < KT) {
      if constexpr (STAGES == 2) {
        wait_dma();
      } else {
        // tile kt+1 landed; tiles kt+2 .. kt+STAGES-1 may still be in flight
        const int ahead = KT - kt - 2 < STAGES - 2 ? KT - kt - 2 : STAGES - 2;
        wait_tiles<LPT>(ahead);
      }
      __syncthreads();                     // tile kt+1 is in its stage; stage kt's is free
      const char *nA = smem + ((kt + 1) & (STAGES - 1)) * STAGE;
      read_frags<T, IN, OA, OB>(cur, nA, nA + OA::BYTES, lane, wm, wn, 0);
      if (kt + STAGES < KT) issue(kt + STAGES);
    }
    mfma_block<T, IN>(acc, nxt);
  }
  }

  if constexpr (sizeof...(SC) > 0)
    scale_acc<32>(acc, m0 + wm * T::TM, n0 + wn * T::TN, M, N, lane, sc...);
  if constexpr (LSM_DMA_ROW_EPI) {
    if (c_vec) {
      __syncthreads();                     // every wave is past its last LDS read
      epilogue_lds_rows<T, OUT, STAGES * STAGE, 32>(C, acc, smem, M, N, ldc, m0, n0, wm, wn, wave, lane);
      return;
    }
  } else if constexpr (T::TN == 64) {
    if (c_vec) {
      __syncthreads();
      epilogue_lds<T, OUT, STAGES * STAGE>(C, acc, smem, M, N, ldc, m0, n0, wm, wn, wave, lane);
      return;
    }
  }
  epilogue<T, OUT>(C, acc, M, N, ldc, m0, n0, wm, wn, lane);
}

}  // namespace lsm
