// gemm_mxfp4.hip -- gemm_mxfp4_run: the product of two MXFP4 matrices, and
// gemm_grouped_mxfp4_run: the same by groups of rows, each with its own matrix.
//
//   C[m][n] = sum_k qa(m,k) 2^(SA[k/32][m] - 127) * qb(n,k) 2^(SB[k/32][n] - 127)
//
// The scales enter the matrix instruction beside the elements, one byte for each
// lane's block of 32 (gemm_mxfp4.h); the kernels are those of
// gemm_kernel_tile256.h and gemm_kernel_tile.h.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_tile_launch.h"

namespace lsm {

// Shapes as in gemm_grouped.hip.
using MxTile128 = TileShape<128, 128, 2, 4, 2>;
using MxTile128Alone = TileShape<128, 128, 2, 4, 3>;
using MxTile64 = TileShape<64, 128, 2, 2, 2>;
using MxTile64SplitK = TileShape<64, 128, 2, 2, 3, 2>;
using MxTile64x64 = TileShape<64, 64, 2, 2, 2>;
using MxTile64x64SplitK = TileShape<64, 64, 2, 2, 3, 2>;
using MxTile32SplitK = TileShape<32, 64, 1, 2, 3, 2>;
using MxStream16x16 = StreamShape<16, 16, 4, 2>;
using MxStream16x32 = StreamShape<16, 32, 4, 2>;
using MxStream16 = StreamShape<16, 64, 2, 2>;
using MxStream16x128 = StreamShape<16, 128, 2, 2>;
using MxStream32x32 = StreamShape<32, 32, 4, 2>;
using MxStream32 = StreamShape<32, 64, 2, 2>;

// Streams up to 32 rows, of the widest tiles that give every CU one (1 x 16384 x
// 8192: 16.1 us in 64 columns, 18.0 in 16; 1 x 4096 x 4096: 5.6 in 16, 6.1 in 32; uneven
// groups, rows, groups, N, K: 64, 16, 4096, 4096: 27.1 in 128 columns, 30.5 in 64, 37.5 in 16;
// 240, 8, 4096, 4096: 20.7, as 128 x 128 tiles 24).  128 columns as long as all run at once,
// two workgroups to a CU (8, 8, 14336, 4096: 39.7, in 64 columns 34.4).
template <int MODE, int OUT>
static Plan plan_mx_stream(const TileArgs &p, int64_t rows, int64_t groups) {
  const int64_t wide = groups * ceil_div(p.N, 64), half = groups * ceil_div(p.N, 32);
  if (rows > 16)
    return wide >= 256 ? plan_stream<MxStream32, MODE, KC, IN_MXFP4, OUT>()
                       : plan_stream<MxStream32x32, MODE, KC, IN_MXFP4, OUT>();
  const int64_t wider = groups * ceil_div(p.N, 128);
  if (wider >= 256 && wider <= 512) return plan_stream<MxStream16x128, MODE, KC, IN_MXFP4, OUT>();
  if (wide >= 256) return plan_stream<MxStream16, MODE, KC, IN_MXFP4, OUT>();
  if (half >= 256) return plan_stream<MxStream16x32, MODE, KC, IN_MXFP4, OUT>();
  return plan_stream<MxStream16x16, MODE, KC, IN_MXFP4, OUT>();
}

// More rows: the shape that takes the least (8192 x 8192 x 8192 235-247 us in 256 x 256; 1024 x
// 8192 x 8192 45 us, as 128 x 128 tiles 51; 2048 x 2048 x 16384 55 in 128 x 128 alone on a CU, 63 in
// 128 x 128 two to a CU; 256 x 8192 x 8192 20.6 in 64 x 128 with K shared out, 32.4 without; 2399
// x 832 x 4512 17.3 in 64 x 64, 19.4 in 64 x 128; 1500 x 512 x 8192 14.9 in 64 x 64 with K shared
// out, 21.3 without; 128 x 4096 x 4096 8.4 in 32 x 64, 9.8 in 64 x 64; uneven groups, rows, groups, N,
// K: 2048, 32, 1152, 896: 10.0 in 64 x 128, 12.3 in 128 x 128; 6000, 16, 1152, 2560: 21 in 128 x 128,
// 27 in 256 x 256; 2048, 8, 4096, 4096: 38 in 256 x 256, 47 in 128 x 128; 1225, 4, 733, 352: 6.2 in 64
// x 64, 6.9 with K shared out).
template <int MODE, int OUT, class Tiles>
static Plan plan_mx_tiles(const TileArgs &p, Tiles tiles) {
  const float k = k_tiles(p, IN_MXFP4);
  Cheapest c{plan_tile256<MODE, KC, KC, IN_MXFP4, OUT>(),
             tile256_time({3.6f, 2.f, 1.26f, 0.82f}, tiles(256, 256), k, tile256_parts(KC))};
  c.offer(plan_tile<MxTile128, MODE, KC, KC, IN_MXFP4, OUT>(), tiles_time({512, 3.2f, 1.65f, 0.88f}, tiles(128, 128), k));
  c.offer(plan_tile<MxTile128Alone, MODE, KC, KC, IN_MXFP4, OUT>(), tiles_time({256, 3.3f, 0.79f, 0.76f}, tiles(128, 128), k));
  c.offer(plan_tile<MxTile64, MODE, KC, KC, IN_MXFP4, OUT>(), tiles_time({768, 2.f, 1.5f, 0.76f}, tiles(64, 128), k));
  c.offer(plan_tile<MxTile64SplitK, MODE, KC, KC, IN_MXFP4, OUT>(), tiles_time({256, 3.1f, 0.53f, 0.47f}, tiles(64, 128), k));
  c.offer(plan_tile<MxTile64x64, MODE, KC, KC, IN_MXFP4, OUT>(), tiles_time({1280, 1.7f, 1.83f, 0.64f}, tiles(64, 64), k));
  c.offer(plan_tile<MxTile64x64SplitK, MODE, KC, KC, IN_MXFP4, OUT>(), tiles_time({256, 2.7f, 0.32f, 0.26f}, tiles(64, 64), k));
  c.offer(plan_tile<MxTile32SplitK, MODE, KC, KC, IN_MXFP4, OUT>(), tiles_time({512, 2.4f, 0.5f, 0.27f}, tiles(32, 64), k));
  return c.plan;
}

// One product; up to 64 rows of few columns are streamed (64 x 4096 x 4096 6.7 us, in
// 32 x 64 tiles 8.3).
template <int OUT>
static Plan plan_mx_one(const TileArgs &p) {
  const auto tiles = [&](int bm, int bn) { return (float)(ceil_div(p.M, bm) * ceil_div(p.N, bn)); };
  if (p.M <= 32 || (p.M <= 64 && tiles(32, 32) <= 256)) return plan_mx_stream<GROUP_NONE, OUT>(p, p.M, 1);
  return plan_mx_tiles<GROUP_NONE, OUT>(p, tiles);
}

// Groups, by their mean number of rows.
template <int OUT>
static Plan plan_mx_groups(const TileArgs &p) {
  const int64_t mean = ceil_div(p.M, p.G);
  if (mean <= 32) return plan_mx_stream<GROUP_ROWS, OUT>(p, mean, p.G < p.M ? p.G : p.M);
  return plan_mx_tiles<GROUP_ROWS, OUT>(p, [&](int bm, int bn) { return expected_tiles(p, bm, bn); });
}

template <int MODE, int OUT>
static Plan plan_mx(const TileArgs &p) {
  if constexpr (MODE == GROUP_ROWS)
    return plan_mx_groups<OUT>(p);
  else
    return plan_mx_one<OUT>(p);
}

// What both products check; `G`: groups, or 0 for the one product.
static int check_mx(const void *A, const void *B, void *C, const void *SA, const void *SB, const int32_t *ends,
                    int64_t G, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t strideb, int64_t ldc,
                    int64_t ldsa, int64_t ldsb, int64_t stridesb, int dtype, TileArgs &p) {
  const int64_t n = G > 0 ? G : 1;
  if (!C || (K > 0 && (!A || !B || !SA || !SB)) || (G > 0 && !ends)) return GEMM_ERR_INVALID_ARG;
  if (ldc < N || (K > 0 && (lda < K || ldb < K || ldsa < M || ldsb < N || strideb < 0 || stridesb < 0)))
    return GEMM_ERR_INVALID_ARG;
  const int64_t size = mxfp4_out(dtype) == OUT_F32 ? 4 : 2;
  if (G > kMaxGroups || M >= kTileMaxDim || N >= kTileMaxDim || K >= kTileMaxDim || ldc >= kTileMaxLd)
    return GEMM_ERR_UNSUPPORTED;
  if (((uintptr_t)C & (uintptr_t)(size - 1)) || ((uintptr_t)ends & 3)) return GEMM_ERR_UNSUPPORTED;
  if (K > 0) {
    if (lda / 2 >= kTileMaxPitch || ldb / 2 >= kTileMaxPitch || ldsa >= kScaleMaxPitch || ldsb >= kScaleMaxPitch ||
        strideb >= kTileMaxLd || stridesb >= kTileMaxLd)
      return GEMM_ERR_UNSUPPORTED;
    if (((uintptr_t)A & 15) || ((uintptr_t)B & 15) || ((uintptr_t)SA & 15) || ((uintptr_t)SB & 15) || K % kMxBlock ||
        lda % kMxBlock || ldb % kMxBlock || strideb % kMxBlock || ldsa % 16 || ldsb % 16 || stridesb % 16)
      return GEMM_ERR_UNSUPPORTED;
  }
  const int64_t blocks = K / kMxBlock;
  const int64_t c_bytes = footprint_bytes(M, ldc, N, size);
  const int64_t a_bytes = K > 0 ? footprint_bytes(M, lda / 2, K / 2, 1) : 0;
  const int64_t b_bytes = K > 0 ? stacked_bytes(n, strideb / 2, footprint_bytes(N, ldb / 2, K / 2, 1)) : 0;
  const int64_t sa_bytes = K > 0 ? footprint_bytes(blocks, ldsa, (M + 15) & ~(int64_t)15, 1) : 0;
  const int64_t sb_bytes = K > 0 ? stacked_bytes(n, stridesb, footprint_bytes(blocks, ldsb, (N + 15) & ~(int64_t)15, 1)) : 0;
  if (c_bytes < 0 || a_bytes < 0 || b_bytes < 0 || sa_bytes < 0 || sb_bytes < 0) return GEMM_ERR_UNSUPPORTED;
  if (overlaps_any({C, c_bytes}, {{A, a_bytes}, {B, b_bytes}, {SA, sa_bytes}, {SB, sb_bytes}, {ends, 4 * G}}))
    return GEMM_ERR_INVALID_ARG;
  p = TileArgs{};
  p.A = (const char *)A, p.B = (const char *)B, p.C = C, p.SA = (const char *)SA, p.SB = (const char *)SB;
  p.ends = ends, p.G = (int)G, p.M = (int)M, p.N = (int)N, p.K = (int)K;
  p.lda = lda / 2, p.ldb = ldb / 2, p.strideb = strideb / 2, p.ldc = ldc;
  p.ldsa = ldsa, p.ldsb = ldsb, p.stridesb = stridesb;
  return GEMM_OK;
}

template <int MODE>
static int run_mx(gemm_handle_t h, const TileArgs &p, int dtype, hipStream_t stream) {
  const Plan plan = with_out(mxfp4_out(dtype), [&](auto out) { return plan_mx<MODE, decltype(out)::value>(p); });
  return run_plan(h, plan, p, stream);
}

}  // namespace lsm

extern "C" int gemm_mxfp4_run(gemm_handle_t h, const void *A, const void *B, void *C, const void *SA, const void *SB,
                              int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int64_t ldsa,
                              int64_t ldsb, int dtype, hipStream_t stream) {
  using namespace lsm;
  if (!h || M < 0 || N < 0 || K < 0 || dtype < GEMM_MXFP4_BF16 || dtype > GEMM_MXFP4_F32) return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  TileArgs p;
  const int st = check_mx(A, B, C, SA, SB, nullptr, 0, M, N, K, lda, ldb, 0, ldc, ldsa, ldsb, 0, dtype, p);
  return st != GEMM_OK ? st : run_mx<GROUP_NONE>(h, p, dtype, stream);
}

extern "C" int gemm_grouped_mxfp4_run(gemm_handle_t h, const void *A, const void *B, void *C, const void *SA,
                                      const void *SB, const int32_t *ends, int64_t G, int64_t T, int64_t N, int64_t K,
                                      int64_t lda, int64_t ldb, int64_t strideb, int64_t ldc, int64_t ldsa, int64_t ldsb,
                                      int64_t stridesb, int dtype, hipStream_t stream) {
  using namespace lsm;
  if (!h || G < 0 || T < 0 || N < 0 || K < 0 || dtype < GEMM_MXFP4_BF16 || dtype > GEMM_MXFP4_F32) return GEMM_ERR_INVALID_ARG;
  if (G == 0 || T == 0 || N == 0) return GEMM_OK;
  TileArgs p;
  const int st = check_mx(A, B, C, SA, SB, ends, G, T, N, K, lda, ldb, strideb, ldc, ldsa, ldsb, stridesb, dtype, p);
  return st != GEMM_OK ? st : run_mx<GROUP_ROWS>(h, p, dtype, stream);
}
