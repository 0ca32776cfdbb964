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
using Tile128 = TileShape<128, 128, 2, 4, 2>;
using Tile128Alone = TileShape<128, 128, 2, 4, 3>;
using Tile64 = TileShape<64, 128, 2, 2, 2>;
using Tile64SplitK = TileShape<64, 128, 2, 2, 3, 2>;
using Tile64x64 = TileShape<64, 64, 2, 2, 2>;
using Tile64x64SplitK = TileShape<64, 64, 2, 2, 3, 2>;
using Tile32SplitK = TileShape<32, 64, 1, 2, 3, 2>;

// Up to 32 rows a group in the mean: the columns of a stream by how many workgroups
// there are to be (bf16, B K-contiguous; rows, groups, N, K: 1, 1, 2048, 4096: 7.4 us in
// 16 columns, 8.8 in 32, 10.1 in 64; 2, 2, 4096, 4096: 15.7, 15.5, 18.4; 4, 4, 4096, 4096: 21.2,
// 21.3, 19.9; 64, 16, 4096, 4096: 88 in 32, 84 in 64; B MN-contiguous, 1, 1, 352, 2344: 8.3 in
// 64, 15.3 in 128; 32, 8, 4096, 4096: 57 in 64, 50 in 128 of four waves, 52 of two with three
// stages).
template <int BM, int LB, int IN, int OUT>
static Plan plan_few_rows(const TileArgs &p) {
  const int64_t used = p.G < p.M ? p.G : p.M;
  const auto columns = [&](int bn) { return used * ceil_div(p.N, bn); };
  if constexpr (LB == KC) {
    if (columns(16) <= 256) return plan_stream<StreamShape<BM, 16, 8, 2>, GROUP_ROWS, KC, IN, OUT>();
    if (columns(32) < 512) return plan_stream<StreamShape<BM, 32, 4, 2>, GROUP_ROWS, KC, IN, OUT>();
    return plan_stream<StreamShape<BM, 64, 4, 2>, GROUP_ROWS, KC, IN, OUT>();
  } else {
    if (columns(64) < 256) return plan_stream<StreamShape<BM, 64, 4, 2>, GROUP_ROWS, MNC, IN, OUT>();
    return plan_stream<StreamShape<BM, 128, BM == 16 ? 4 : 2, 2>, GROUP_ROWS, MNC, IN, OUT>();
  }
}

// More rows: the shape that takes the least (uneven groups in bf16; rows, groups, N, K:
// 300, 8, 4096, 4096: 49 us in 128 x 128 alone on a CU, 67 in 64 x 128; 1500, 4, 4096, 1152: 23
// in 256 x 256, 28 in 128 x 128; 6000, 16, 1152, 2048: 43 in 128 x 128, 53 in 256 x 256; 2048, 32,
// 1152, 896: 20.6 in 64 x 128, 24.8 in 128 x 128; 1500, 8, 896, 1152: 12.1 in 64 x 128 with K
// shared out, 14.2 without; 767, 1, 448, 1856: 9.6 in 32 x 64, 11.9 in 64 x 64; 1500, 8, 512, 2560:
// 14.8 in 64 x 64, 16.4 in 32 x 64).  128 x 128 takes eight waves: four take 5% longer at 256 k
// and as long at 4096.
template <int LB, int IN, int OUT>
static Plan plan_rows(const TileArgs &p) {
  const int64_t mean = ceil_div(p.M, p.G);
  if (mean <= 16) return plan_few_rows<16, LB, IN, OUT>(p);
  if (mean <= 32) return plan_few_rows<32, LB, IN, OUT>(p);
  const auto tiles = [&](int bm, int bn) { return expected_tiles(p, bm, bn); };
  const float k = k_tiles(p, IN);
  Cheapest c{plan_tile256<GROUP_ROWS, KC, LB, IN, OUT>(),
             tile256_time({5.4f, 1.35f, 0.79f, 0.57f}, tiles(256, 256), k, tile256_parts(KC))};
  c.offer(plan_tile<Tile128, GROUP_ROWS, KC, LB, IN, OUT>(), tiles_time({512, 3.7f, 1.22f, 0.77f}, tiles(128, 128), k));
  c.offer(plan_tile<Tile128Alone, GROUP_ROWS, KC, LB, IN, OUT>(), tiles_time({256, 3.5f, 0.58f, 0.49f}, tiles(128, 128), k));
  c.offer(plan_tile<Tile64, GROUP_ROWS, KC, LB, IN, OUT>(), tiles_time({768, 2.6f, 1.33f, 0.65f}, tiles(64, 128), k));
  c.offer(plan_tile<Tile64SplitK, GROUP_ROWS, KC, LB, IN, OUT>(), tiles_time({256, 2.7f, 0.44f, 0.37f}, tiles(64, 128), k));
  c.offer(plan_tile<Tile64x64SplitK, GROUP_ROWS, KC, LB, IN, OUT>(), tiles_time({256, 2.f, 0.25f, 0.22f}, tiles(64, 64), k));
  c.offer(plan_tile<Tile32SplitK, GROUP_ROWS, KC, LB, IN, OUT>(), tiles_time({512, 2.1f, 0.4f, 0.2f}, tiles(32, 64), k));
  return c.plan;
}

// The gradient of the matrices: the shape that takes the least for groups of the
// mean number of rows, C's bytes included in `fixed` (bf16 to fp32; rows, groups, M, N:
// 16384, 8, 4096, 4096: 470-482 us in 256 x 256, 625 in 128 x 128; 1500, 8, 1152, 896: 11.9 in 128 x
// 128, 19.7 in 256 x 256; 8192, 1, 768, 4096: 81 in 128 x 128 alone on a CU, 107 two to a CU; 59, 7,
// 1280, 1016: 12.9 in 64 x 64, 16.3 in 128 x 128; with the rows shared out, 9826, 1, 512, 512: 37 in
// 64 x 64, 55 in 64 x 128; 1500, 1, 1536, 1152: 14.3 in 64 x 128, 17.4 in 64 x 64).
template <int IN, int OUT>
static Plan plan_sums(const TileArgs &p) {
  const auto tiles = [&](int bm, int bn) { return (float)workgroups<GROUP_SUMS>(p, bm, bn); };
  const float k = (float)p.K / (float)p.G / (float)kTileK(IN);
  constexpr float C = OUT == OUT_F32 ? 1.f : 0.5f;             // C's bytes, in fp32's
  Cheapest c{plan_tile256<GROUP_SUMS, MNC, MNC, IN, OUT>(),
             tile256_time({6.7f + 3.2f * C, 1.7f, 0.86f, 0.86f}, tiles(256, 256), k, tile256_parts(MNC))};
  c.offer(plan_tile<Tile128, GROUP_SUMS, MNC, MNC, IN, OUT>(), tiles_time({512, 2.9f + 1.9f * C, 1.09f, 0.65f}, tiles(128, 128), k));
  c.offer(plan_tile<Tile128Alone, GROUP_SUMS, MNC, MNC, IN, OUT>(), tiles_time({256, 3.7f + 0.4f * C, 0.6f, 0.57f}, tiles(128, 128), k));
  c.offer(plan_tile<Tile64SplitK, GROUP_SUMS, MNC, MNC, IN, OUT>(), tiles_time({256, 2.8f + C, 0.4f, 0.32f}, tiles(64, 128), k));
  c.offer(plan_tile<Tile64x64, GROUP_SUMS, MNC, MNC, IN, OUT>(), tiles_time({1280, 2.5f + 0.8f * C, 1.27f, 0.59f}, tiles(64, 64), k));
  c.offer(plan_tile<Tile64x64SplitK, GROUP_SUMS, MNC, MNC, IN, OUT>(), tiles_time({256, 2.6f + 1.3f * C, 0.22f, 0.21f}, tiles(64, 64), k));
  return c.plan;
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
