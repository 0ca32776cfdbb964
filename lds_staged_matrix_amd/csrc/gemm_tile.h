// gemm_tile.h -- what the kernels of the grouped and of the MXFP4 products
// share: their arguments, where a workgroup's tile lies, the loads of an
// operand's tile and the stores of C.
//
// Every operand is addressed from its tile's first element in 64 bits, and the
// buffer descriptor of a K tile starts at that tile: offsets inside it stay below
// 2^31 however long the operand is.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "gemm_common.h"
#include "gemm_groups.h"
#include "gemm_kernel_pingpong.h"
#include "gemm_mxfp4.h"

namespace lsm {

enum { IN_MXFP4 = 4 };            // beside the IN_ types of gemm_common.h; K-contiguous operands only

// A row's 128 bytes of K are a K tile's: 64 elements of 16 bits, 256 of 4.  A
// fragment of the 16 x 16 MFMAs is 16 bytes of it (frag16_kc_offset), two k-steps
// a K tile: 32 elements of 16 bits a k-step, 128 of 4.
constexpr int kTileK(int in) { return in == IN_MXFP4 ? 256 : 64; }
constexpr int kTileBytes = 128;
constexpr int kScaleRows = kTileK(IN_MXFP4) / kMxBlock;      // blocks of k in a K tile

struct TileArgs {
  const char *A, *B;
  void *C;
  const char *SA, *SB;                      // MXFP4: the operands' scales
  const int32_t *ends;                      // groups
  int G;
  int M, N, K;                              // GROUP_ROWS: M, GROUP_SUMS: K counts the rows of all groups
  int64_t lda, ldb, strideb;                // bytes
  int64_t ldc, stridec;                     // elements
  int64_t ldsa, ldsb, stridesb;             // bytes
  int tiles_m, tiles_n;                     // of one product or group (GROUP_ROWS: tiles_n alone)
  int c_vec;                                // 16-byte stores to C's rows are aligned
  int by_size;                              // GROUP_SUMS: groups with more rows first
};

// A workgroup's tile, or its part of one.  Pointers are to the first row and
// column (of A and B: at k = 0), `rows` and `cols` count from there to the end of
// the matrix or group, and may be more than the tile's or part's `height` and width.
struct Where {
  const char *a, *b, *sa, *sb;
  int64_t c;            // element of C
  int rows, cols, K;
  int skip;             // rows at the start that belong to the group before
  int height;
};

// The tile of this workgroup, or one of up to PARTS parts of it; false if there is
// none for it.  ALIGN: row tiles of GROUP_ROWS start at multiples of it.
template <int BM, int BN, int GROUP_M, int MODE, int LA, int LB, int IN, int ALIGN, int PARTS = 1>
__device__ __forceinline__ bool locate(const TileArgs &p, int lane, Where &w) {
  constexpr int ES2 = IN == IN_MXFP4 ? 1 : 4;          // half bytes of an element
  int tm, tn;
  Part part;
  if constexpr (MODE == GROUP_ROWS) {
    static_assert(LA == KC, "grouped rows are K-contiguous");
    Group at;
    if (!find_row_tile<BM, ALIGN, PARTS>(p.ends, p.G, p.M, p.tiles_n, GROUP_M, (int)blockIdx.x, lane, at, part, tm, tn))
      return false;
    w.height = BM / part.parts;
    const int m0 = at.first - early_rows<ALIGN>(at.first) + tm * BM + part.sub * w.height, n0 = tn * BN;
    if (m0 >= at.last) return false;
    w.a = p.A + m0 * p.lda;
    w.b = p.B + at.g * p.strideb + (LB == KC ? n0 * p.ldb : (int64_t)n0 * ES2 / 2);
    w.c = m0 * p.ldc + n0;
    w.rows = at.last - m0, w.cols = p.N - n0, w.K = p.K;
    w.skip = at.first > m0 ? at.first - m0 : 0;
    if constexpr (IN == IN_MXFP4) w.sa = p.SA + m0, w.sb = p.SB + at.g * p.stridesb + n0;
    return true;
  }
  const int tiles = p.tiles_m * p.tiles_n;
  if (!part_of<PARTS>((int)blockIdx.x, tiles * (MODE == GROUP_SUMS ? p.G : 1), part)) return false;
  // Group after group, each spread over all the XCDs: with whole groups to an
  // XCD the one with the most rows keeps the others waiting (16384 rows in eight
  // uneven groups, 4096 x 4096 fp32: 784 us; so 476, as with even groups).  Where not all
  // tiles run at once the groups with the most rows come first: a long one that
  // starts last is waited for (16384 rows in eight groups, 1024 x 4096: 157 us, so 131);
  // in one round the search only takes time (0.1 us for eight groups).
  const int g = MODE == GROUP_SUMS ? part.tile / tiles : 0;
  tile_coords(xcd_logical_id(part.tile - g * tiles, tiles), p.tiles_m, p.tiles_n, GROUP_M, tm, tn);
  w.height = BM / part.parts;
  const int m0 = tm * BM + part.sub * w.height, n0 = tn * BN;
  if (m0 >= p.M) return false;
  w.a = p.A + (LA == KC ? m0 * p.lda : (int64_t)m0 * ES2 / 2);
  w.b = p.B + (LB == KC ? n0 * p.ldb : (int64_t)n0 * ES2 / 2);
  w.c = m0 * p.ldc + n0;
  w.rows = p.M - m0, w.cols = p.N - n0, w.K = p.K, w.skip = 0;
  if constexpr (IN == IN_MXFP4) w.sa = p.SA + m0, w.sb = p.SB + n0;
  if constexpr (MODE == GROUP_SUMS) {
    const Group at = p.by_size ? find_group<true>(p.ends, p.G, p.K, g, lane)
                               : find_group<false>(p.ends, p.G, p.K, g, lane);
    w.a += at.first * p.lda, w.b += at.first * p.ldb, w.c += at.g * p.stridec;
    w.K = at.last - at.first;
  }
  return true;
}

// ------------------------------------------------- MN-contiguous rows of 64
//
// An MN-contiguous tile 64 elements wide has k-rows of 128 bytes, two to a bank
// line.  One 32-lane phase of the transposed read takes k-rows k..k+3 and
// k+8..k+11, 32 bytes each (mn16_swizzle in lds_layout.h); four of the eight lie in
// either half of the line, rows 2 and 8 apart, and the XOR below puts them into its
// four 32-byte quarters.
__host__ __device__ constexpr int narrow_swizzle(int k) { return 2 * (((k >> 1) & 1) | ((k >> 2) & 2)); }

// The LDS tile of MN rows or columns of an operand, loaded by NT threads: as
// OperandTile, for the geometries that it does not take (one wave's loads, of 8
// rows of 128 bytes or 4 of 256; k-rows of 128 bytes).
template <int MN, int LAYOUT, int NT>
struct SlabTile {
  static constexpr bool kcontig = LAYOUT == KC, mf16 = !kcontig, narrow = !kcontig && MN == 64;
  static constexpr int ROWS = kcontig ? MN : 64, ROW_BYTES = kcontig ? kTileBytes : 2 * MN;
  static constexpr int BYTES = ROWS * ROW_BYTES, LOADS = BYTES / (16 * NT), ROW_STEP = 16 * NT / ROW_BYTES;
  static constexpr int PHASE_ROWS = 8, LANE_OFFSETS = ROW_STEP % 16 == 0 ? 1 : 2;
  static_assert(kcontig || ROW_BYTES == 256 || ROW_BYTES == 128, "rows of 128 or 256 bytes");
  static_assert(LOADS >= 1 && (ROW_STEP % 16 == 0 || PHASE_ROWS % ROW_STEP == 0), "one or two swizzle phases");
  __host__ __device__ static constexpr int round_phase(int d) {
    return LANE_OFFSETS == 1 ? 0 : d * ROW_STEP / PHASE_ROWS & 1;
  }
  __host__ __device__ static constexpr int swizzle(int row) {
    return kcontig ? kc_swizzle(row, ROW_BYTES) : narrow ? narrow_swizzle(row) : mn16_swizzle(row, ROW_BYTES);
  }
};
template <int MN, int LAYOUT, int NT, int EB>
using TileOf = std::conditional_t<LAYOUT == MNC && MN == 64, SlabTile<MN, LAYOUT, NT>,
                                  OperandTile<MN, kTileBytes / EB, LAYOUT, NT, EB, 1>>;

// A 16 x 16 fragment of either (see read_frag16).
template <class OT>
__device__ __forceinline__ v8i16 read_tile_frag(const char *lds, int lane, int base, int kk) {
  if constexpr (!OT::kcontig && OT::ROW_BYTES == 128) {
    const int k0 = 8 * (lane >> 4) + ((lane >> 2) & 3);          // the k-row, less 32 * kk + 4 * half
    const char *a = lds + (k0 + 32 * kk) * 128 + 32 * ((base >> 4) ^ (narrow_swizzle(k0) >> 1)) + 16 * ((lane & 3) >> 1) +
                    8 * (lane & 1);
    const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)a);
    const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16 *)(a + 4 * 128));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  } else {
    return read_frag16<OT>(lds, lane, base, kk);
  }
}

// ------------------------------------------------------------------- loads

// Bytes of `inner` bytes a row from the first of `outer` rows to the last.
__device__ __forceinline__ int64_t span_bytes(int outer, int64_t ld, int64_t inner) { return (outer - 1) * ld + inner; }

// A buffer descriptor of the `left` bytes from `first` on, 2^31 - 1 at most.  In
// 32-bit comparisons, which stay in scalar registers.
__device__ __forceinline__ i32x4 rest_rsrc(uint64_t first, int64_t left) {
  const int high = (int)(left >> 32);
  uint32_t n = (uint32_t)left;
  if (high > 0 || n > 0x7FFFFFFFu) n = 0x7FFFFFFFu;
  return buffer_rsrc((const void *)first, high < 0 ? 0u : n);
}

// An operand's tile, loaded by NT threads 16 bytes at a time (OT: an OperandTile
// of NT threads).  F > 0 spreads the rows over the fragments: fragment i of a
// wave tile of F fragments holds its rows F * r + i, r = 0..15, so that a lane's
// F scales, or F columns of C, stand side by side.
template <class OT, int NT, int F = 0>
struct Loader {
  static constexpr int TM = 16 * F;
  uint64_t base;
  int64_t bytes;             // from base to the operand's end
  uint32_t ld, kstep, v0, v1;
  int inner0, inner1;        // K-contiguous: first byte of the chunk in its row

  // The row, less the lane's own, of load d.
  static constexpr int round_row(int d) {
    const int p = d * OT::ROW_STEP;
    return F == 0 ? p : TM * (p / (F ? TM : 1)) + (p % (F ? TM : 1)) / 16;
  }
  // `ext`: rows (K-contiguous), or bytes of a row.  `kbytes`: bytes (K-contiguous), or rows, of K.
  __device__ __forceinline__ Loader(int tid, const char *first, int64_t ld_, int ext, int kbytes) {
    static_assert(F == 0 || (OT::ROW_STEP == 32 && OT::kcontig && OT::ROW_BYTES == 128), "spread rows");
    base = (uint64_t)first;
    ld = (uint32_t)ld_;
    bytes = OT::kcontig ? span_bytes(ext < OT::ROWS ? ext : OT::ROWS, ld_, kbytes) : span_bytes(kbytes, ld_, ext);
    kstep = OT::kcontig ? OT::ROW_BYTES : OT::ROWS * ld;
    v0 = v1 = lane_offset(tid, ext, 0, inner0);
    inner1 = inner0;
    if constexpr (OT::LANE_OFFSETS == 2) v1 = lane_offset(tid, ext, 1, inner1);
  }
  __device__ __forceinline__ uint32_t lane_offset(int tid, int ext, int phase, int &inner) {
    const int row = loader_row(tid, OT::ROW_BYTES);
    const int chunk = loader_chunk(tid, OT::ROW_BYTES) ^ OT::swizzle(row + phase * OT::PHASE_ROWS);
    inner = 16 * chunk;
    if (!OT::kcontig && inner >= ext) return kOutOfRange;
    const int at = F == 0 ? row : F * (row & 15) + (row >> 4);
    const int64_t off = (int64_t)at * ld + inner;
    return off < bytes ? (uint32_t)off : kOutOfRange;
  }
  // The descriptor of K tile kt, and its lane offsets: in the last, cut tile,
  // chunks behind K (`kbytes` bytes of it) read as zero.
  struct At {
    i32x4 rs;
    uint32_t v0, v1;
  };
  __device__ __forceinline__ At at(int kt, int kbytes) const {
    const int64_t done = (int64_t)kt * kstep;
    At a{rest_rsrc(base + done, bytes - done), v0, v1};
    if constexpr (OT::kcontig)
      if ((kt + 1) * OT::ROW_BYTES > kbytes) {
        a.v0 = kt * OT::ROW_BYTES + inner0 < kbytes ? v0 : kOutOfRange;
        a.v1 = OT::LANE_OFFSETS == 1 ? a.v0 : kt * OT::ROW_BYTES + inner1 < kbytes ? v1 : kOutOfRange;
      }
    return a;
  }
  // Load d of a K tile, by wave `wave` of the NT threads, into the LDS tile.
  __device__ __forceinline__ void issue(const At &a, uint32_t lds_tile, int wave, int d) const {
    dma16(a.rs, lds_tile + (uint32_t)((d * NT + 64 * wave) * 16), OT::round_phase(d) ? a.v1 : a.v0,
          (uint32_t)round_row(d) * ld);
  }
};

// ------------------------------------------------------------------ stores

// Four consecutive entries of C, of which those from `cols` on do not exist.
template <int OUT>
__device__ __forceinline__ void store4(void *C, int64_t at, v4f32 v, int cols) {
  typedef typename OutElem<OUT>::type E;
  E *c = (E *)C + at;
  if (cols >= 4) {
    typedef unsigned int u32xn __attribute__((ext_vector_type(sizeof(E)), aligned(sizeof(E))));
    E e[4];
#pragma unroll
    for (int i = 0; i < 4; i++) e[i] = (E)v[i];
    __builtin_nontemporal_store(__builtin_bit_cast(u32xn, e), (u32xn *)c);
  } else {
#pragma unroll
    for (int i = 0; i < 3; i++)
      if (i < cols) __builtin_nontemporal_store((E)v[i], c + i);
  }
}

// f(std::integral_constant<int, 0>) ... f(std::integral_constant<int, N - 1>)
template <class F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void each(F f) {
  each_of(f, std::make_integer_sequence<int, N>{});
}

}  // namespace lsm
