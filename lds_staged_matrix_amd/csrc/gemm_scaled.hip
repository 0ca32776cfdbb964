// gemm_scaled.hip -- gemm_scaled_run: the E4M3 product whose rows and columns
// carry fp32 scales.  The kernels are gemm_run's, with the scales applied to
// the fp32 sums before they are rounded (scale_acc in gemm_common.h), the
// few-rows kernel of gemm_kernel_rows.h and the split-K tile of
// gemm_kernel_splitk.h.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gemm_kernel_rows.h"
#include "gemm_kernel_splitk.h"
#include "gemm_launch.h"

namespace lsm {

// What is asked for: the output's type, and whether the sums are to be exact.
// An fp32 output multiplies its operands as bf16, whose MFMAs sum in fp32
// throughout (see e4m3_part_as_bf16).  A 16-bit output, whose rounding is off by
// up to 2^-8 or 2^-11, takes the fp8 MFMAs at twice the rate, unless the caller
// asks for exact sums (GEMM_EXACT_SUMS) or HBM is the bound anyway (few rows).
struct Wanted {
  int out;
  bool exact;
};

// call(IN, OUT) with the element types as constants; IN16: of 16-bit outputs
// that need no exact sums.
template <int IN16, class F>
static hipError_t with_types(const Wanted &w, F call) {
  constexpr std::integral_constant<int, IN_E4M3_AS_BF16> exact{};
  constexpr std::integral_constant<int, IN16> fast{};
  constexpr std::integral_constant<int, OUT_F32> f32{};
  constexpr std::integral_constant<int, OUT_BF16> bf16{};
  constexpr std::integral_constant<int, OUT_F16> f16{};
  if (w.out == OUT_F32) return call(exact, f32);
  if (w.out == OUT_BF16) return w.exact ? call(exact, bf16) : call(fast, bf16);
  return w.exact ? call(exact, f16) : call(fast, f16);
}

template <class T, int KIND, int IN16 = IN_E4M3>
static hipError_t launch_scaled(const Args &a, int la, int lb, const Wanted &w, hipStream_t s, const RowColScale &sc) {
  return with_types<IN16>(w, [&](auto in, auto out) {
    return launch_layout<T, KIND, decltype(in)::value, decltype(out)::value, RowColScale>(a, la, lb, s, sc);
  });
}

template <int LA, int LB, int IN, int OUT, int KS, int NS>
static hipError_t launch_splitk(const Args &a, hipStream_t stream, RowColScale sc) {
  using T = DmaSmall8;
  int tiles_m = (int)ceil_div(a.M, T::BM), tiles_n = (int)ceil_div(a.N, T::BN);
  const uint16_t *A = a.A, *B = a.B;
  void *C = a.C;
  int M = a.M, N = a.N, K = a.K;
  int64_t lda = a.lda, ldb = a.ldb, ldc = a.ldc;
  uint32_t ab = a.a_bytes, bb = a.b_bytes;
  constexpr int64_t esz = OUT == OUT_F32 ? 4 : 2;
  int c_vec = ((uintptr_t)C % 16 == 0) && ((ldc * esz) % 16 == 0);
  void *params[] = {&A, &B, &C, &M, &N, &K, &lda, &ldb, &ldc, &tiles_m, &tiles_n, &ab, &bb, &c_vec, &sc};
  return hipLaunchKernel((const void *)lds_gemm_splitk_kernel<T, LA, LB, IN, OUT, KS, NS>,
                         dim3((unsigned)(tiles_m * tiles_n)), dim3(KS * T::NT), params, 0, stream);
}

template <int KS, int NS, int IN, int OUT>
static hipError_t launch_splitk_layout(const Args &a, int la, int lb, hipStream_t s, const RowColScale &sc) {
  if (la == KC && lb == KC) return launch_splitk<KC, KC, IN, OUT, KS, NS>(a, s, sc);
  if (la == KC && lb == MNC) return launch_splitk<KC, MNC, IN, OUT, KS, NS>(a, s, sc);
  if (la == MNC && lb == KC) return launch_splitk<MNC, KC, IN, OUT, KS, NS>(a, s, sc);
  return launch_splitk<MNC, MNC, IN, OUT, KS, NS>(a, s, sc);
}

// Other products of at most 256 tiles of 64 x 64 (one for a CU) share each tile's K
// out over groups of waves once it is 1024 long: two groups with four LDS
// stages, or four with two for exact sums, whose conversions want the waves.
// Up to 1024 tiles and from K = 4096 on, two groups with two stages, so that
// two workgroups fit a CU.  Kernel times against the kernels without the split:
//   bf16 output  256 x 4096 x 4096 12.2 and 18.2 us, 256 x 2048 x 8192 16.9 and
//   32.1, 128 x 8192 x 8192 18.1 and 29.9, 512 x 8192 x 8192 55 and 67, 1024 x
//   4096 x 4096 31 and 35; but 1500 x 1152 x 896 8.3 and 6.8, 2048 x 4096 x 4096
//   65 and 47.
//   fp32 output  256 x 4096 x 4096 14.1 and 18.7 us, 256 x 2048 x 8192 20.2 and
//   32.4, 512 x 8192 x 8192 77 and 89.
// Returns false where the split does not pay.
static bool dispatch_splitk(const Args &a, int la, int lb, const Wanted &w, hipStream_t s, const RowColScale &sc,
                            hipError_t &e) {
  const int64_t tiles = ceil_div(a.M, 64) * ceil_div(a.N, 64);
  const bool few = tiles <= 256 && a.K >= 1024, more = tiles > 256 && tiles <= 1024 && a.K >= 4096;
  if (!few && !more) return false;
  e = with_types<IN_E4M3>(w, [&](auto in, auto out) {
    constexpr int IN = decltype(in)::value, OUT = decltype(out)::value;
    if (more) return launch_splitk_layout<2, 2, IN, OUT>(a, la, lb, s, sc);
    if constexpr (IN == IN_E4M3)
      return launch_splitk_layout<2, 4, IN, OUT>(a, la, lb, s, sc);
    else
      return launch_splitk_layout<4, 2, IN, OUT>(a, la, lb, s, sc);
  });
  return true;
}

// Waves of a workgroup: as many as K has blocks for, up to eight.
template <int AR, int NT, int IN, int OUT>
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
  return hipLaunchKernel((const void *)lds_gemm_rows_e4m3_kernel<AR, NT, IN, OUT>, dim3((unsigned)tiles),
                         dim3(64u * waves), params,
                         (size_t)rows_lds_bytes(waves, T::SLICE, T::RB * NT), stream);
}

// From 33 rows on 16-bit outputs take the fp8 MFMA (128 x 4096 x 4096 9.7 and
// 8.7 us, 192 x 2048 x 8192 14.5 and 12.0); with fewer HBM is the bound and the
// exact form costs nothing.
template <int AR, int NT>
static hipError_t launch_rows_out(const Args &a, const Wanted &w, hipStream_t s, const RowColScale &sc) {
  return with_types<(AR > 32 ? IN_E4M3 : IN_E4M3_AS_BF16)>(w, [&](auto in, auto out) {
    return launch_rows<AR, NT, decltype(in)::value, decltype(out)::value>(a, s, sc);
  });
}

// Column blocks: two if tiles of one would be more than the 256 CUs (measured
// with one and two: 48 x 4608 x 4096 9.8 and 8.4 us, 16 x 4608 x 4096 6.5 and
// 6.0; but 64 x 4096 x 4096 7.9 and 9.6); one where at most 8 rows make the
// activations' share small (4 x 8192 x 8192: 12.5 us with one, 13.0 with two).
template <int AR>
static hipError_t dispatch_rows(const Args &a, const Wanted &w, hipStream_t s, const RowColScale &sc) {
  if (AR > 8 && ceil_div(a.M, AR < 16 ? 16 : AR) * ceil_div(a.N, 16) > 256)
    return launch_rows_out<AR, 2>(a, w, s, sc);
  return launch_rows_out<AR, 1>(a, w, s, sc);
}

// With both operands K-contiguous the few-rows kernel takes M <= 32, and more
// rows while its 64-row tiles, of one block of columns or of two, are at most
// the 256 CUs: up to 64 tiles of 64 x 64, or up to 128 and K long enough for its
// waves.  bf16 output, the few-rows kernel against the tiled ones: 64 x 4096 x
// 4096 7.7 and 10.0 us, 1024 x 256 x 4096 7.1 and 9.7, 128 x 4096 x 4096 8.8 and
// 9.9, 64 x 8192 x 8192 19.2 and 23.3 (fp32 output 19.8 and 30.5); but 128 x
// 4096 x 896 6.2 and 5.6, 48 x 12288 x 4096 12.6 and 11.0, 128 x 8192 x 8192 33
// and 23 (fp32 output 33 and 30).
static bool few_rows(const Args &a, int la, int lb) {
  const int64_t tiles = ceil_div(a.M, 64) * ceil_div(a.N, 64);
  return la == KC && lb == KC && (a.M <= 32 || tiles <= 64 || (tiles <= 128 && a.K >= 1536));
}

// Otherwise the split-K tiles where they pay, and the shape classes of
// gemm_run's E4M3 products.
static hipError_t dispatch_scaled(const Args &a, int la, int lb, const Wanted &w, hipStream_t s, const RowColScale &sc) {
  if (few_rows(a, la, lb)) {
    if (a.M <= 8) return dispatch_rows<8>(a, w, s, sc);
    if (a.M <= 16) return dispatch_rows<16>(a, w, s, sc);
    if (a.M <= 32) return dispatch_rows<32>(a, w, s, sc);
    // tiles of 48 rows where they pad M less than 64 (96 x 4096 x 8192 11.0 and 12.5 us)
    return ceil_div(a.M, 48) * 48 < ceil_div(a.M, 64) * 64 ? dispatch_rows<48>(a, w, s, sc)
                                                           : dispatch_rows<64>(a, w, s, sc);
  }
  if (a.M <= 32) return launch_scaled<SkinnyStream8, SKINNY, IN_E4M3_AS_BF16>(a, la, lb, w, s, sc);
  hipError_t e;
  if (dispatch_splitk(a, la, lb, w, s, sc, e)) return e;
  // The 256 x 256 tile also wins with fewer workgroups than CUs where it
  // replaces more than two rounds of 128 x 128 tiles.  bf16 output, ping-pong
  // against 128 x 128: 1100 x 8192 x 8192 79 and 141 us, 2048 x 5000 x 3200 42 and
  // 61, 1500 x 6000 x 1024 19.5 and 25.7; at two rounds 2048 x 4096 x 4096 47 and
  // 46, 1024 x 8192 x 8192 97 and 89 (fp32 output 86 and 79, 164 and 165).
  const int64_t t128 = ceil_div(a.M, 128) * ceil_div(a.N, 128);
  if (ceil_div(a.M, 256) * ceil_div(a.N, 256) >= 256 || t128 > 512)
    return launch_scaled<PingPong8, PINGPONG>(a, la, lb, w, s, sc);
  if (t128 >= 256)
    return launch_scaled<DmaMid8, DMA>(a, la, lb, w, s, sc);
  if (small_tile_four_stages(a, 1)) return launch_scaled<DmaSmall8, DMA4>(a, la, lb, w, s, sc);
  return launch_scaled<DmaSmall8, DMA>(a, la, lb, w, s, sc);
}

}  // namespace lsm

extern "C" int gemm_scaled_run(gemm_handle_t h, const void *A, const void *B, void *C, const float *SA,
                               const float *SB, int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb,
                               int64_t ldc, int incA, int incB, int layoutA, int layoutB, int dtype,
                               hipStream_t stream) {
  using namespace lsm;
  if (!h || M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  const bool exact = dtype >= 0 && (dtype & GEMM_EXACT_SUMS);
  if (exact) dtype -= GEMM_EXACT_SUMS;
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
  const Wanted w{dtype == GEMM_E4M3_F32 ? OUT_F32 : dtype == GEMM_E4M3_BF16 ? OUT_BF16 : OUT_F16, exact};
  if (dispatch_scaled(args, layoutA, layoutB, w, stream, RowColScale{SA, SB, incA, incB}) != hipSuccess)
    return GEMM_ERR_LAUNCH;
  return GEMM_OK;
}
