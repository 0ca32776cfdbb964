// gemm_grouped.hip -- gemm_grouped_run: the rows of each group (expert) times the
// group's own matrix, and gemm_grouped_wgrad_run: the gradient of those matrices.
//
//   C[t][n]    = sum_k A[t][k] * B[g][k][n]         for t in group g
//   C[g][m][n] = sum over t in group g of A[t][m] * B[t][n]
//
// The gradient of the rows is the first of them with B's other layout.  The
// kernels are those of gemm_kernel_tile256.h and gemm_kernel_tile.h.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_tile_launch.h"

namespace lsm {

// Tiles: rows x columns, waves, LDS stages, groups of waves that share K.  Streams:
// rows x columns, waves, stages a wave.
using Tile128 = TileShape<128, 128, 2, 2, 2>;
using Tile128Alone = TileShape<128, 128, 2, 4, 3>;
using Tile64 = TileShape<64, 128, 2, 2, 2>;
using Tile64SplitK = TileShape<64, 128, 2, 2, 3, 2>;
using SmallSplitK = TileShape<64, 64, 2, 2, 3, 2>;
using SmallSplitKMN = TileShape<32, 128, 1, 4, 3, 2>;
using Stream16 = StreamShape<16, 64, 4, 2>;
using Stream32 = StreamShape<32, 64, 4, 2>;
using Stream16MN = StreamShape<16, 128, 2, 3>;
using Stream32MN = StreamShape<32, 128, 2, 2>;

// By the mean number of rows a group, and by how many tiles are to be expected
// against the 256 CUs.  Times of uneven groups in bf16, B K- and MN-contiguous
// (rows, groups, N, K):
//  * streams up to 32 rows (64, 16, 4096, 4096: 84 and 94 us; 240, 8, 4096, 4096: 58
//    and 69, as 128 x 128 tiles 69 and 62);
//  * the 256 x 256 tile and its halves and quarters from 192 rows on (2048, 8, 4096,
//    4096: 95 and 88 us, as 128 x 128 tiles 125; 16384, 8, 4096, 4096: 435 and 429, 590;
//    but 1024, 8, 4096, 4096: 84 and 78, 74 and 78);
//  * few tiles share K out over two groups of waves: 64 x 128 (1500, 8, 896, 1152: 11.9
//    and 11.7 us; with one group 14.2), fewer still 64 x 64 or 32 x 128 (700, 8, 1152,
//    896: 8.7 and 8.8; as 64 x 128 10.3);
//  * tiles of 128 x 128 that are about as many as the CUs stand alone on one, with
//    three stages (300, 8, 4096, 4096: 50 and 49 us, as 64 x 128 72); more of them go two
//    to a CU (1024, 8, 4096, 4096: 74 and 78, alone 84 and 83), and those of up to 96
//    rows are 64 x 128 (2048, 32, 1152, 896: 20.5 and 20.0, as 128 x 128 23.0 and 22.6).
template <int LB, int IN, int OUT>
static Plan plan_rows(const TileArgs &p) {
  const int64_t mean = ceil_div(p.M, p.G);
  if (mean <= 16) return plan_stream<std::conditional_t<LB == KC, Stream16, Stream16MN>, GROUP_ROWS, LB, IN, OUT>();
  if (mean <= 32) return plan_stream<std::conditional_t<LB == KC, Stream32, Stream32MN>, GROUP_ROWS, LB, IN, OUT>();
  if (mean >= 192 && expected_tiles(p, 256, 256) >= 128) return plan_tile256<GROUP_ROWS, KC, LB, IN, OUT>();
  if (expected_tiles(p, 64, 128) < 160)
    return plan_tile<std::conditional_t<LB == KC, SmallSplitK, SmallSplitKMN>, GROUP_ROWS, KC, LB, IN, OUT>();
  const int64_t tiles = expected_tiles(p, 128, 128);
  if (tiles < 192) return plan_tile<Tile64SplitK, GROUP_ROWS, KC, LB, IN, OUT>();
  if (tiles <= 264) return plan_tile<Tile128Alone, GROUP_ROWS, KC, LB, IN, OUT>();
  if (mean <= 96) return plan_tile<Tile64, GROUP_ROWS, KC, LB, IN, OUT>();
  return plan_tile<Tile128, GROUP_ROWS, KC, LB, IN, OUT>();
}

// The 256 x 256 tile where it fills the CUs and its sums are 512 rows long or more
// in the mean (bf16 to fp32; rows, groups, M, N: 16384, 8, 4096, 4096: 485 us, as 128 x
// 128 tiles 597; 4096, 8, 2048, 2048: 54 and 57; but 1000, 8, 4096, 4096: 131 and 112).
// 128 x 128 tiles of which a CU has one or none have three stages (16384, 4, 1024,
// 1024: 72 us, with two 102), few of them two groups of waves that share the sum out
// (8192, 2, 512, 512: 47 us; 54 without).
using Tile128Sums = TileShape<128, 128, 2, 4, 2>;
using Tile128SplitK = TileShape<128, 128, 2, 2, 2, 2>;

template <int IN, int OUT>
static Plan plan_sums(const TileArgs &p) {
  if (ceil_div(p.K, p.G) >= 512 && workgroups<GROUP_SUMS>(p, 256, 256) >= 256)
    return plan_tile256<GROUP_SUMS, MNC, MNC, IN, OUT>();
  const int64_t tiles = workgroups<GROUP_SUMS>(p, 128, 128);
  if (tiles <= 128) return plan_tile<Tile128SplitK, GROUP_SUMS, MNC, MNC, IN, OUT>();
  if (tiles <= 256) return plan_tile<Tile128Alone, GROUP_SUMS, MNC, MNC, IN, OUT>();
  return plan_tile<Tile128Sums, GROUP_SUMS, MNC, MNC, IN, OUT>();
}

template <class F>
static Plan with_types(int dtype, F call) {
  constexpr std::integral_constant<int, IN_BF16> bf16{};
  constexpr std::integral_constant<int, IN_F16> f16{};
  constexpr std::integral_constant<int, OUT_F32> f32{};
  switch (dtype) {
    case GEMM_BF16_F32: return call(bf16, f32);
    case GEMM_BF16_BF16: return call(bf16, std::integral_constant<int, OUT_BF16>{});
    case GEMM_F16_F16: return call(f16, std::integral_constant<int, OUT_F16>{});
    default: return call(f16, f32);
  }
}

}  // namespace lsm

extern "C" int gemm_grouped_run(gemm_handle_t h, const void *A, const void *B, void *C, const int32_t *ends, int64_t G,
                                int64_t T, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t strideb,
                                int64_t ldc, int layoutB, int dtype, hipStream_t stream) {
  using namespace lsm;
  if (!h || G < 0 || T < 0 || N < 0 || K < 0 || dtype < GEMM_BF16_F32 || dtype > GEMM_F16_F32) return GEMM_ERR_INVALID_ARG;
  if (layoutB != GEMM_K_CONTIG && layoutB != GEMM_MN_CONTIG) return GEMM_ERR_INVALID_ARG;
  if (G == 0 || T == 0 || N == 0) return GEMM_OK;
  const bool kc = layoutB == GEMM_K_CONTIG;
  if (!C || !ends || (K > 0 && (!A || !B))) return GEMM_ERR_INVALID_ARG;
  if (ldc < N || (K > 0 && (lda < K || ldb < (kc ? K : N) || strideb < 0))) return GEMM_ERR_INVALID_ARG;

  const bool out_f32 = dtype == GEMM_BF16_F32 || dtype == GEMM_F16_F32;
  if (G > kMaxGroups || T >= kTileMaxDim || N >= kTileMaxDim || K >= kTileMaxDim || ldc >= kTileMaxLd)
    return GEMM_ERR_UNSUPPORTED;
  if (((uintptr_t)C & (out_f32 ? 3 : 1)) || ((uintptr_t)ends & 3)) return GEMM_ERR_UNSUPPORTED;
  if (K > 0) {
    if (2 * lda >= kTileMaxPitch || ldb >= kTileMaxPitch / 2 || strideb >= kTileMaxLd) return GEMM_ERR_UNSUPPORTED;
    if (((uintptr_t)A & 15) || ((uintptr_t)B & 15) || lda % 8 || ldb % 8 || strideb % 8) return GEMM_ERR_UNSUPPORTED;
    if (K % 8 || (!kc && N % 8)) return GEMM_ERR_UNSUPPORTED;
  }
  const int64_t c_bytes = footprint_bytes(T, ldc, N, out_f32 ? 4 : 2);
  const int64_t a_bytes = K > 0 ? footprint_bytes(T, lda, K, 2) : 0;
  const int64_t b_bytes = K > 0 ? stacked_bytes(G, 2 * strideb, kc ? footprint_bytes(N, ldb, K, 2) : footprint_bytes(K, ldb, N, 2)) : 0;
  if (c_bytes < 0 || a_bytes < 0 || b_bytes < 0) return GEMM_ERR_UNSUPPORTED;
  if (overlaps_any({C, c_bytes}, {{A, a_bytes}, {B, b_bytes}, {ends, 4 * G}})) return GEMM_ERR_INVALID_ARG;

  TileArgs p{};
  p.A = (const char *)A, p.B = (const char *)B, p.C = C, p.ends = ends, p.G = (int)G;
  p.M = (int)T, p.N = (int)N, p.K = (int)K;
  p.lda = 2 * lda, p.ldb = 2 * ldb, p.strideb = 2 * strideb, p.ldc = ldc;
  p.c_vec = (uintptr_t)C % 16 == 0 && ldc * (out_f32 ? 4 : 2) % 16 == 0;
  const Plan plan = with_types(dtype, [&](auto in, auto out) {
    constexpr int IN = decltype(in)::value, OUT = decltype(out)::value;
    return kc ? plan_rows<KC, IN, OUT>(p) : plan_rows<MNC, IN, OUT>(p);
  });
  return run_plan(h, plan, p, stream);
}

extern "C" int gemm_grouped_wgrad_run(gemm_handle_t h, const void *A, const void *B, void *C, const int32_t *ends,
                                      int64_t G, int64_t T, int64_t M, int64_t N, int64_t lda, int64_t ldb, int64_t ldc,
                                      int64_t stridec, int dtype, hipStream_t stream) {
  using namespace lsm;
  if (!h || G < 0 || T < 0 || M < 0 || N < 0 || dtype < GEMM_BF16_F32 || dtype > GEMM_F16_F32) return GEMM_ERR_INVALID_ARG;
  if (G == 0 || M == 0 || N == 0) return GEMM_OK;
  if (!C || !ends || (T > 0 && (!A || !B))) return GEMM_ERR_INVALID_ARG;
  if (ldc < N || (T > 0 && (lda < M || ldb < N))) return GEMM_ERR_INVALID_ARG;

  const bool out_f32 = dtype == GEMM_BF16_F32 || dtype == GEMM_F16_F32;
  const int64_t size = out_f32 ? 4 : 2;
  if (G > kMaxGroups || T >= kTileMaxDim || M >= kTileMaxDim || N >= kTileMaxDim || ldc >= kTileMaxLd)
    return GEMM_ERR_UNSUPPORTED;
  if (((uintptr_t)C & (uintptr_t)(size - 1)) || ((uintptr_t)ends & 3)) return GEMM_ERR_UNSUPPORTED;
  if (T > 0) {
    if (2 * lda >= kTileMaxPitch || 2 * ldb >= kTileMaxPitch) return GEMM_ERR_UNSUPPORTED;
    if (((uintptr_t)A & 15) || ((uintptr_t)B & 15) || lda % 8 || ldb % 8 || M % 8 || N % 8) return GEMM_ERR_UNSUPPORTED;
  }
  const int64_t one = footprint_bytes(M, ldc, N, size);
  if (one < 0) return GEMM_ERR_UNSUPPORTED;
  // the groups' results are disjoint
  if (G > 1 && (stridec < 0 || stridec < one / size)) return GEMM_ERR_INVALID_ARG;
  if (G > 1 && stridec >= ((int64_t)1 << 60)) return GEMM_ERR_UNSUPPORTED;
  const int64_t c_bytes = stacked_bytes(G, G > 1 ? size * stridec : 0, one);
  const int64_t a_bytes = T > 0 ? footprint_bytes(T, lda, M, 2) : 0, b_bytes = T > 0 ? footprint_bytes(T, ldb, N, 2) : 0;
  if (c_bytes < 0 || a_bytes < 0 || b_bytes < 0) return GEMM_ERR_UNSUPPORTED;
  if (overlaps_any({C, c_bytes}, {{A, a_bytes}, {B, b_bytes}, {ends, 4 * G}})) return GEMM_ERR_INVALID_ARG;

  TileArgs p{};
  p.A = (const char *)A, p.B = (const char *)B, p.C = C, p.ends = ends, p.G = (int)G;
  p.M = (int)M, p.N = (int)N, p.K = (int)T;
  p.lda = 2 * lda, p.ldb = 2 * ldb, p.ldc = ldc, p.stridec = G > 1 ? stridec : 0;
  p.c_vec = (uintptr_t)C % 16 == 0 && ldc * size % 16 == 0 && p.stridec * size % 16 == 0;
  const Plan plan = with_types(dtype, [&](auto in, auto out) {
    return plan_sums<decltype(in)::value, decltype(out)::value>(p);
  });
  return run_plan(h, plan, p, stream);
}
