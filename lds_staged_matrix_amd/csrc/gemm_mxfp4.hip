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

using MxTile64 = TileShape<64, 64, 2, 2, 4>;
using MxTile128 = TileShape<128, 128, 2, 2, 2>;
using MxStream16x16 = StreamShape<16, 16, 8, 3>;
using MxStream16 = StreamShape<16, 32, 8, 2>;
using MxStream32 = StreamShape<32, 32, 8, 2>;

template <int MODE, int OUT>
static hipError_t dispatch_mx(const TileArgs &p, hipStream_t s) {
  const int64_t rows = MODE == GROUP_ROWS ? ceil_div(p.M, p.G) : p.M;
  const int64_t groups = MODE == GROUP_ROWS ? p.G : 1;
  if (rows <= 16) {
    if (groups * ceil_div(p.N, 32) < 256) return launch_stream<MxStream16x16, MODE, KC, IN_MXFP4, OUT>(p, s);
    return launch_stream<MxStream16, MODE, KC, IN_MXFP4, OUT>(p, s);
  }
  if (rows <= 32) return launch_stream<MxStream32, MODE, KC, IN_MXFP4, OUT>(p, s);
  if (rows >= 192 && workgroups<MODE>(p, 256, 256, 16) >= 256) return launch_tile256<MODE, KC, KC, IN_MXFP4, OUT>(p, s);
  if (workgroups<MODE>(p, 128, 128) >= 256) return launch_tile<MxTile128, MODE, KC, KC, IN_MXFP4, OUT>(p, s);
  return launch_tile<MxTile64, MODE, KC, KC, IN_MXFP4, OUT>(p, s);
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
  if (G >= kTileMaxDim || M >= kTileMaxDim || N >= kTileMaxDim || K >= kTileMaxDim || ldc >= kTileMaxLd)
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
  // the smallest tiles, 16 x 16, must fit a launch of fewer than 2^32 threads of 512 each
  int64_t tiles;
  if (__builtin_mul_overflow(G > 0 ? most_row_tiles(M, G, 16, 1) : ceil_div(M, 16), ceil_div(N, 16), &tiles) ||
      tiles >= (int64_t)1 << 23)
    return GEMM_ERR_UNSUPPORTED;
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
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != h->device) return GEMM_ERR_DEVICE;
  const hipError_t e = with_out(mxfp4_out(dtype), [&](auto out) { return dispatch_mx<MODE, decltype(out)::value>(p, stream); });
  return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
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
