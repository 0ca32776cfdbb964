// gemm_scaled.hip -- gemm_scaled_run: the E4M3 product whose rows and columns
// carry fp32 scales.  The kernels are gemm_run's, with the scales applied to
// the fp32 sums before they are rounded (scale_acc in gemm_common.h), and the
// few-rows kernel of gemm_kernel_rows.h.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_kernel_rows.h"
#include "gemm_launch.h"

namespace lsm {

// An fp32 output multiplies its operands as bf16, whose MFMAs sum in fp32
// throughout (see e4m3_part_as_bf16); 16-bit outputs, rounded to 2^-8 or 2^-11,
// take the fp8 MFMAs at twice the rate -- except where HBM is the bound anyway
// (few rows, IN16).
template <class T, int KIND, int IN16 = IN_E4M3>
static hipError_t launch_scaled(const Args &a, int la, int lb, int dtype, hipStream_t s, const RowColScale &sc) {
  switch (dtype) {
    case GEMM_E4M3_F32: return launch_layout<T, KIND, IN_E4M3_AS_BF16, OUT_F32, RowColScale>(a, la, lb, s, sc);
    case GEMM_E4M3_BF16: return launch_layout<T, KIND, IN16, OUT_BF16, RowColScale>(a, la, lb, s, sc);
    default: return launch_layout<T, KIND, IN16, OUT_F16, RowColScale>(a, la, lb, s, sc);
  }
}

// Waves of a workgroup: as many as K has blocks for, up to eight.
template <int AR, int NT, int OUT>
static hipError_t launch_rows(const Args &a, hipStream_t stream, RowColScale sc) {
  using T = RowsE4M3<AR, NT>;
  int waves = 1;
  while (2 * waves <= kRowsMaxWaves && 2 * waves * kRowsBlockK <= a.K) waves *= 2;
  const char *A = (const char *)a.A, *B = (const char *)a.B;
  void *C = a.C;
  int M = a.M, N = a.N, K = a.K;
  uint32_t lda = (uint32_t)a.lda, ldb = (uint32_t)a.ldb;
  int64_t ldc = a.ldc;
  int tiles_m = (int)ceil_div(a.M, 16 * T::RB);
  const int64_t tiles = tiles_m * ceil_div(a.N, 16 * NT);
  void *params[] = {&A, &B, &C, &M, &N, &K, &lda, &ldb, &ldc, &tiles_m, &sc};
  return hipLaunchKernel((const void *)lds_gemm_rows_e4m3_kernel<AR, NT, OUT>, dim3((unsigned)tiles),
                         dim3(64u * waves), params,
                         (size_t)waves * (T::SLICE > 1024 * T::RB * NT ? T::SLICE : 1024 * T::RB * NT), stream);
}

template <int AR, int NT>
static hipError_t launch_rows_out(const Args &a, int dtype, hipStream_t s, const RowColScale &sc) {
  switch (dtype) {
    case GEMM_E4M3_F32: return launch_rows<AR, NT, OUT_F32>(a, s, sc);
    case GEMM_E4M3_BF16: return launch_rows<AR, NT, OUT_BF16>(a, s, sc);
    default: return launch_rows<AR, NT, OUT_F16>(a, s, sc);
  }
}

// Column blocks by M and N: two if that still makes a workgroup for every CU;
// one where at most 8 rows make the activations' share small (1 x 16384 x 8192:
// 23.6 us with one, 25.7 with two).
template <int AR>
static hipError_t dispatch_rows(const Args &a, int dtype, hipStream_t s, const RowColScale &sc) {
  if (AR > 8 && ceil_div(a.M, AR < 16 ? 16 : AR) * ceil_div(a.N, 32) >= 256)
    return launch_rows_out<AR, 2>(a, dtype, s, sc);
  return launch_rows_out<AR, 1>(a, dtype, s, sc);
}

// With both operands K-contiguous the few-rows kernel takes M <= 48, and up to
// 192 rows while 64 x 64 tiles would fill no more than half of the CUs, each
// walking all of K.  bf16 output, the few-rows kernel against the 64 x 64 tiles:
// 33 x 16384 x 8192 31 and 35 us, 64 x 8192 x 8192 17 and 30, 128 x 4096 x 4096 11
// and 17, 192 x 1152 x 896 5.0 and 5.4; but 64 x 16384 x 8192 43 and 36,
// 128 x 8192 x 8192 36 and 32, 256 x 4096 x 4096 20 and 18.
static bool few_rows(const Args &a, int la, int lb) {
  return la == KC && lb == KC &&
         (a.M <= 48 || (a.M <= 192 && ceil_div(a.M, 64) * ceil_div(a.N, 64) <= 128));
}

// Otherwise the shape classes of gemm_run's E4M3 products.
static hipError_t dispatch_scaled(const Args &a, int la, int lb, int dtype, hipStream_t s, const RowColScale &sc) {
  if (few_rows(a, la, lb)) {
    if (a.M <= 8) return dispatch_rows<8>(a, dtype, s, sc);
    if (a.M <= 16) return dispatch_rows<16>(a, dtype, s, sc);
    if (a.M <= 32) return dispatch_rows<32>(a, dtype, s, sc);
    return a.M <= 48 ? dispatch_rows<48>(a, dtype, s, sc) : dispatch_rows<64>(a, dtype, s, sc);
  }
  if (a.M <= 32) return launch_scaled<SkinnyStream8, SKINNY, IN_E4M3_AS_BF16>(a, la, lb, dtype, s, sc);
  if (ceil_div(a.M, 256) * ceil_div(a.N, 256) >= 256)
    return launch_scaled<PingPong8, PINGPONG>(a, la, lb, dtype, s, sc);
  if (ceil_div(a.M, 128) * ceil_div(a.N, 128) >= 256)
    return launch_scaled<DmaMid8, DMA>(a, la, lb, dtype, s, sc);
  if (small_tile_four_stages(a, 1)) return launch_scaled<DmaSmall8, DMA4>(a, la, lb, dtype, s, sc);
  return launch_scaled<DmaSmall8, DMA>(a, la, lb, dtype, s, sc);
}

}  // namespace lsm

extern "C" int gemm_scaled_run(gemm_handle_t h, const void *A, const void *B, void *C, const float *SA,
                               const float *SB, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                               int64_t ldc, int incA, int incB, int layoutA, int layoutB, int dtype,
                               hipStream_t stream) {
  using namespace lsm;
  if (!h || M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (dtype != GEMM_E4M3_F32 && dtype != GEMM_E4M3_BF16 && dtype != GEMM_E4M3_F16) return GEMM_ERR_INVALID_ARG;
  if ((incA != 0 && incA != 1) || (incB != 0 && incB != 1)) return GEMM_ERR_INVALID_ARG;
  const int64_t out_size = dtype == GEMM_E4M3_F32 ? 4 : 2;
  Args args;
  const int st = check_product(A, B, C, M, N, K, lda, ldb, ldc, layoutA, layoutB, 1, out_size, args);
  if (st != GEMM_OK || M == 0 || N == 0) return st;
  if (!SA || !SB) return GEMM_ERR_INVALID_ARG;
  if (((uintptr_t)SA & 3) || ((uintptr_t)SB & 3)) return GEMM_ERR_UNSUPPORTED;
  const int64_t c_bytes = footprint_bytes(M, ldc, N, out_size);
  if (ranges_overlap(C, c_bytes, SA, incA ? 4 * M : 4) || ranges_overlap(C, c_bytes, SB, incB ? 4 * N : 4))
    return GEMM_ERR_INVALID_ARG;
  if (!dma_ok(args, layoutA, layoutB, 1)) return GEMM_ERR_UNSUPPORTED;

  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != h->device) return GEMM_ERR_DEVICE;
  if (dispatch_scaled(args, layoutA, layoutB, dtype, stream, RowColScale{SA, SB, incA, incB}) != hipSuccess)
    return GEMM_ERR_LAUNCH;
  return GEMM_OK;
}
