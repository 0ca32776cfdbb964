// gemm_kernel_tile256.h -- the 256 x 256 tile of the grouped and of the MXFP4
// products, on the ping-pong schedule of gemm_kernel_pingpong.h: eight waves in
// two groups, one of which reads the fragments of a K tile and loads a later
// one while the other multiplies; that file's head has the barriers, what they
// order, and who loads what.  Here
//  * a workgroup's tile and operands come from locate(): by group where there
//    are groups;
//  * 16-bit operands of which A is K-contiguous are loaded by both groups, A by
//    group 0 into two stages and B by group 1 into three; the others by group 0
//    into two stages each;
//  * an MXFP4 K tile is 256 k, the same bytes as 64 of 16 bits, and its scales (8
//    blocks by 256 rows and by 256 columns, 4 KiB) come with it, 1 KiB a loading
//    wave.  Rows are spread over the fragments (Loader's F), so that one
//    ds_read_b64 gives a lane the scales of its eight row fragments, a
//    ds_read_b32 those of its four column fragments, each a byte that the MFMA
//    picks; and a lane ends with four consecutive columns of C, stored straight
//    from the accumulators, 128 or 256 bytes a row;
//  * a tile of which the group or the matrix fills no more than 128 or 64 rows is
//    computed as one of 128 or 64 rows, and so are the halves and quarters into
//    which the last, part-filled round of tiles is cut (part_of).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_tile.h"

namespace lsm {

// Row tiles of MXFP4 groups start at multiples of 16 rows, where the scales'
// 16-byte pieces start.
template <int IN, int MODE>
constexpr int tile_align() {
  return IN == IN_MXFP4 && MODE == GROUP_ROWS ? 16 : 1;
}

// LDS bytes of a K tile's scales of one operand: 8 blocks of 256.
constexpr int kScaleBytes = kScaleRows * 256;

// Byte, in one operand's scales of a K tile, of row (column) m of block kb.  The
// XOR of the 16-byte chunks puts the four blocks that one read touches into
// four different 64-byte quarters of the bank line.
__device__ __forceinline__ int scale_chunk(int kb, int chunk) { return kb * 256 + 16 * (chunk ^ (4 * (kb & 3))); }

// Where the operands' stages lie in LDS.  256 rows: A's and B's, two each, or three
// of B where both groups load; then two of the scales.  Fewer rows leave room for
// three stages of everything, and with them a K tile more for the loads to land,
// which half or a quarter of the multiplications would not cover.
template <int LA, int LB, int IN, int FM>
struct Tile256Lds {
  static constexpr bool MX = IN == IN_MXFP4, SPLIT = !MX && LA == KC, DEEP = FM < 8;
  static constexpr int A = 32 * FM * kTileBytes, B = 256 * kTileBytes, S = MX ? 2 * kScaleBytes : 0;
  static constexpr int STAGE = A + B + S;                // of everything
  static constexpr int BYTES = DEEP ? 3 * STAGE : SPLIT ? 2 * A + 3 * B : 2 * STAGE;
  static_assert(BYTES <= 160 * 1024, "gfx950 LDS");
  __device__ static constexpr int a_at(int kt) { return DEEP ? kt % 3 * STAGE : (kt & 1) * (SPLIT ? A : A + B); }
  __device__ static constexpr int b_at(int kt) {
    return DEEP ? kt % 3 * STAGE + A : SPLIT ? 2 * A + kt % 3 * B : (kt & 1) * (A + B) + A;
  }
  __device__ static constexpr int s_at(int kt) { return DEEP ? kt % 3 * STAGE + A + B : 2 * (A + B) + (kt & 1) * S; }
};

// FM scales, one byte each.
template <int FM>
struct ScaleWord {
  typedef std::conditional_t<FM == 8, uint64_t, std::conditional_t<FM == 4, uint32_t, uint16_t>> type;
};

// The most parts of a tile: quarters, or halves where A is MN-contiguous, whose
// fragments want 128 of its rows in LDS.
constexpr int tile256_parts(int la) { return la == KC ? 4 : 2; }

// The tile at `w`, or the first 32 FM of its rows.
template <int MODE, int LA, int LB, int IN, int OUT, int FM>
__device__ __forceinline__ void tile256(const TileArgs &p, const Where &w, char *smem, int tid, int wave) {
  using T = Tile<32 * FM, 256, 64, 2, 4, 8>;
  constexpr bool MX = IN == IN_MXFP4;
  constexpr int NT = 256;                                // threads of a loading group
  constexpr int FN = T::TN / 16, KSTEPS = 2;
  constexpr int EB = MX ? 1 : 2;                         // what OperandTile counts: bytes, or 16-bit elements
  using OA = OperandTile<T::BM, kTileBytes / EB, LA, NT, EB, 1>;
  using OB = OperandTile<T::BN, kTileBytes / EB, LB, NT, EB, 1>;
  using L = Tile256Lds<LA, LB, IN, FM>;
  constexpr bool SPLIT = L::SPLIT, DEEP = L::DEEP;
  constexpr int LEAD = DEEP ? 2 : 1;                     // K tiles that group 0 loads ahead
  constexpr int LOADS = OA::LOADS + OB::LOADS + (MX ? 1 : 0);   // of a lone loading wave and K tile
  constexpr int FRAGS = KSTEPS * (FM + FN);
  const int lane = tid & 63;
  const int group = wave >> 2, lwave = wave & 3;
  const int wm = group, wn = lwave;

  const int KT = (w.K + kTileK(IN) - 1) / kTileK(IN);
  const int kbytes = MX ? w.K / 2 : 2 * w.K;             // of a K-contiguous row
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)smem;

  const Loader<OA, NT, MX ? FM : 0> la(tid & (NT - 1), w.a, p.lda, LA == KC ? w.rows : 2 * w.rows, LA == KC ? kbytes : w.K);
  const Loader<OB, NT, MX ? FN : 0> lb(tid & (NT - 1), w.b, p.ldb, LB == KC ? w.cols : 2 * w.cols, LB == KC ? kbytes : w.K);
  // Both operands K-contiguous: one memory phase whose operand each group picks
  // (a copy of the phase for each would take more registers than there are).
  constexpr bool SELECT = SPLIT && LB == KC && FM == 8;
  static_assert(!SELECT || OA::LOADS == OB::LOADS, "as many load rounds for either operand");
  const auto own = [&] {
    if constexpr (SELECT)
      return group == 1 ? lb : la;
    else
      return la;
  }();
  auto a_stage = [&](int kt) { return (uint32_t)L::a_at(kt); };
  auto b_stage = [&](int kt) { return (uint32_t)L::b_at(kt); };
  auto scales = [&](int kt) { return (uint32_t)L::s_at(kt); };

  // MXFP4: this wave's kilobyte of the scales of K tile kt, four blocks of A
  // (waves 0, 1) or of B.  Blocks behind K read as zero, by the record count.
  const int blocks = w.K / kMxBlock;
  auto issue_scales = [&](int kt) {
    const bool b = lwave >= 2;
    const int64_t ld = b ? p.ldsb : p.ldsa, done = (int64_t)kt * kScaleRows * ld;
    const int n = b ? w.cols : w.rows, width = n < 256 ? (n + 15) & ~15 : 256;
    const i32x4 rs = rest_rsrc((uint64_t)(b ? w.sb : w.sa) + done, span_bytes(blocks, ld, width) - done);
    const int kb = 4 * (lwave & 1) + (lane >> 4), chunk = (lane & 15) ^ (4 * (kb & 3));
    dma16(rs, lds0 + scales(kt) + (uint32_t)(1024 * lwave), (uint32_t)kb * (uint32_t)ld + 16 * chunk, 0);
  };

  v4f32 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; i++)
#pragma unroll
    for (int j = 0; j < FN; j++) acc[i][j] = v4f32{0.f, 0.f, 0.f, 0.f};

  if (KT > 0) {
    // tiles 0 and 1
    if (SPLIT || group == 0) {
      if constexpr (SELECT) {
#pragma unroll
        for (int t = 0; t < 2; t++)
          if (t < KT) {
            const auto r = own.at(t, kbytes);
#pragma unroll
            for (int d = 0; d < OA::LOADS; d++) own.issue(r, lds0 + (group == 1 ? b_stage(t) : a_stage(t)), lwave, d);
          }
      } else if (SPLIT && group == 1) {
#pragma unroll
        for (int t = 0; t < 2; t++)
          if (t < KT) {
            const auto r = lb.at(t, kbytes);
#pragma unroll
            for (int d = 0; d < OB::LOADS; d++) lb.issue(r, lds0 + b_stage(t), lwave, d);
          }
      } else {
#pragma unroll
        for (int t = 0; t < 2; t++)
          if (t < KT) {
            const auto r = la.at(t, kbytes);
#pragma unroll
            for (int d = 0; d < OA::LOADS; d++) la.issue(r, lds0 + a_stage(t), lwave, d);
            if constexpr (!SPLIT) {
              const auto q = lb.at(t, kbytes);
#pragma unroll
              for (int d = 0; d < OB::LOADS; d++) lb.issue(q, lds0 + b_stage(t), lwave, d);
              if constexpr (MX) issue_scales(t);
            }
          }
      }
      if (KT > 1 && SPLIT && group == 0)                 // tile 0 landed
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(OA::LOADS) : "memory");
      else if (KT > 1)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(SPLIT ? OB::LOADS : LOADS) : "memory");
      else
        wait_dma();
    }
    wg_barrier();
    if (group == 1) wg_barrier();                        // group 1 runs one phase behind

    v8i16 fa[KSTEPS][FM], fb[KSTEPS][FN];
    typename ScaleWord<FM>::type ga[KSTEPS];             // scales: a byte for each row fragment
    int gb[KSTEPS];                                      // and for each column fragment
    for (int kt = 0; kt < KT; ++kt) {
      const char *sA = smem + a_stage(kt), *sB = smem + b_stage(kt);
      // LOAD: 0 none, 1 all of tile kt + LEAD (group 0 alone), 2 the group's own of 3 and 4, 3 A of
      // tile kt + LEAD, 4 B of tile kt + 2
      auto m_phase = [&](auto load_kind) {
        constexpr int LOAD = decltype(load_kind)::value;
        constexpr int NL = LOAD == 1 ? LOADS : LOAD == 4 ? OB::LOADS : OA::LOADS;
        const int lt = kt + (LOAD == 4 || (LOAD == 2 && group == 1) ? 2 : LEAD);
        const auto ra = LOAD == 2 ? own.at(lt, kbytes) : la.at(lt, kbytes);
        const auto rb = lb.at(lt, kbytes);
        if constexpr (MX) {
          const char *s = smem + scales(kt);
#pragma unroll
          for (int kk = 0; kk < KSTEPS; kk++) {
            const int kb = 4 * kk + (lane >> 4), c = lane & 15;
            const int row = wm * T::TM + FM * c;
            ga[kk] = *(const typename ScaleWord<FM>::type *)(s + scale_chunk(kb, row / 16) + row % 16);
            gb[kk] = *(const int *)(s + kScaleBytes + scale_chunk(kb, wn * 4 + c / 4) + 4 * (c & 3));
          }
        }
#pragma unroll
        for (int kk = 0; kk < KSTEPS; ++kk) {
#pragma unroll
          for (int i = 0; i < FM + FN; i++) {
            if (i < FM)
              fa[kk][i] = read_frag16<OA>(sA, lane, wm * T::TM + 16 * i, kk);
            else
              fb[kk][i - FM] = read_frag16<OB>(sB, lane, wn * T::TN + 16 * (i - FM), kk);
            const int q = kk * (FM + FN) + i;            // the loads, spread over the reads
#pragma unroll
            for (int d = q * NL / FRAGS; LOAD != 0 && d < (q + 1) * NL / FRAGS; d++) {
              // of a lone loader's: A's, B's, the scales'
              if constexpr (LOAD == 2)
                own.issue(ra, lds0 + (group == 1 ? b_stage(lt) : a_stage(lt)), lwave, d);
              else if ((LOAD == 1 && d < OA::LOADS) || LOAD == 3)
                la.issue(ra, lds0 + a_stage(lt), lwave, d);
              else if (LOAD == 4 || d < OA::LOADS + OB::LOADS)
                lb.issue(rb, lds0 + b_stage(lt), lwave, LOAD == 4 ? d : d - OA::LOADS);
              else if constexpr (MX)
                issue_scales(lt);
            }
          }
        }
      };
      using None = std::integral_constant<int, 0>;
      // tile 1 came with the start
      const bool load0 = DEEP ? kt + 2 < KT : kt >= 1 && kt + 1 < KT;
      if constexpr (SPLIT) {
        const bool load = group == 1 ? kt + 2 < KT : load0;
        if (SELECT && load)
          m_phase(std::integral_constant<int, SELECT ? 2 : 0>{});
        else if (load && group == 0)
          m_phase(std::integral_constant<int, 3>{});
        else if (load)
          m_phase(std::integral_constant<int, 4>{});
        else
          m_phase(None{});
        if (group == 1) {                                // B of tile kt + 1
          if (load)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(OB::LOADS) : "memory");
          else
            wait_dma();
        }
      } else {
        if (group == 0 && load0)
          m_phase(std::integral_constant<int, 1>{});
        else
          m_phase(None{});
      }
      wait_lds_reads();
      wg_barrier();                                      // end of the memory phase

      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        each<FM>([&](auto ic) {
          constexpr int i = decltype(ic)::value;
          each<FN>([&](auto jc) {
            constexpr int j = decltype(jc)::value;
            if constexpr (MX)
              acc[i][j] = mfma_mxfp4<i & 3, j>(fa[kk][i], fb[kk][j], acc[i][j], (int)((uint64_t)ga[kk] >> (32 * (i >> 2))),
                                             gb[kk]);
            else
              acc[i][j] = mfma_16x16x32<IN>(fa[kk][i], fb[kk][j], acc[i][j]);
          });
        });
      }
#pragma unroll
      for (int i = 0; i < FM; i++)
#pragma unroll
        for (int j = 0; j < FN; j++) pin_acc(acc[i][j]);
      __builtin_amdgcn_s_setprio(0);
      if (group == 0) {
        if (DEEP && load0)                               // what group 0 loads of tile kt + 1 landed
          asm volatile("s_waitcnt vmcnt(%0)" ::"n"(SPLIT ? OA::LOADS : LOADS) : "memory");
        else
          wait_dma();
        wg_barrier();                                    // end of the compute phase
      } else if (kt + 1 < KT) {
        wg_barrier();
      }
    }
  }

  typedef typename OutElem<OUT>::type E;
  if constexpr (MX) {
    // register r of fragment (i, j): row 8 (4 g + r) + i of the wave tile, column 4 c + j
    const int c = lane & 15, g = lane >> 4;
    const int col = wn * T::TN + 4 * c;
#pragma unroll
    for (int r = 0; r < 4; r++)
#pragma unroll
      for (int i = 0; i < FM; i++) {
        const int row = wm * T::TM + FM * (4 * g + r) + i;
        if (row >= w.skip && row < w.rows)
          store4<OUT>(p.C, w.c + row * p.ldc + col, v4f32{acc[i][0][r], acc[i][1][r], acc[i][2][r], acc[i][3][r]},
                      w.cols - col);
      }
  } else {
    E *C = (E *)p.C + w.c;
    if (p.c_vec) {
      __syncthreads();                                   // the LDS is free
      epilogue_lds_rows<T, OUT, (L::BYTES < 128 * 1024 ? 64 : 128) * 1024, 16>(C, acc, smem, w.rows, w.cols, p.ldc, 0, 0, wm, wn, wave, lane);
    } else {
      epilogue<T, OUT, 16>(C, acc, w.rows, w.cols, p.ldc, 0, 0, wm, wn, lane);
    }
  }
}

template <int MODE, int LA, int LB, int IN, int OUT>
__global__ __launch_bounds__(512, 1) void lds_gemm_tile256_kernel(const TileArgs p) {
  constexpr int HALF = Tile256Lds<LA, LB, IN, 4>::BYTES, WHOLE = Tile256Lds<LA, LB, IN, 8>::BYTES;
  constexpr int BYTES = HALF > WHOLE ? HALF : WHOLE;
  __shared__ __attribute__((aligned(1024))) char smem[BYTES];
  const int tid = threadIdx.x;
  if constexpr (LSM_LDS_POISON) {   // poison build: all of LDS, before any load or write
    lds_poison(smem, BYTES, tid, blockDim.x);
    __syncthreads();
  }
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Where w{};
  if (!locate<256, 256, 8, MODE, LA, LB, IN, tile_align<IN, MODE>(), tile256_parts(LA)>(p, tid & 63, w)) return;
  const int rows = w.rows < w.height ? w.rows : w.height;
  if (rows > 128)
    tile256<MODE, LA, LB, IN, OUT, 8>(p, w, smem, tid, wave);
  else if (rows > 64 || LA == MNC)
    tile256<MODE, LA, LB, IN, OUT, 4>(p, w, smem, tid, wave);
  else if constexpr (LA == KC)
    tile256<MODE, LA, LB, IN, OUT, 2>(p, w, smem, tid, wave);
}

}  // namespace lsm
