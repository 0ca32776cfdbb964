// gemm_w4.hip -- gemm_w4_run: the product of a few 16-bit rows with 4-bit
// weights (kernel in gemm_kernel_rows.h).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_kernel_rows.h"
#include "gemm_launch.h"

namespace lsm {

// Rows of a tile, of which so many are loaded: from 17 on 32 or 48, whichever
// pads M less (128 x 8192 x 8192 39.4 us with 32 and 50.6 with 48; 192 rows, a tie,
// 57.5 and 52.3).
static int w4_rows(int64_t M) {
  if (M <= 16) return M <= 4 ? 4 : 16;
  return ceil_div(M, 48) * 48 <= ceil_div(M, 32) * 32 ? 48 : 32;
}
// Waves of a workgroup: as many as K has blocks for, up to eight (sixteen halve
// the registers, and took 16.2 us for 1 x 16384 x 8192 where eight took 14.1).
static int w4_waves(int64_t K) {
  int waves = 1;
  while (2 * waves <= kRowsMaxWaves && 2 * waves * kRowsBlockK <= K) waves *= 2;
  return waves;
}
static int64_t w4_row_tiles(int64_t M) {
  const int rows = w4_rows(M);
  return ceil_div(M, rows < 16 ? 16 : rows);
}
// Column blocks of 16: two if tiles of one would be more than the 256 CUs, and
// from 17 rows on four if tiles of two would.  Measured with one and two: 48 x
// 4608 x 4096 14.6 and 9.8 us, 16 x 4608 x 4096 7.0 and 6.2, one row of it 6.2 and
// 5.8; but 48 x 4096 x 4096 8.8 and 10.5, 16 x 4096 x 4096 5.8 and 6.5.  With two
// and four: 48 x 8256 x 8192 31.5 and 26.3, 48 x 16384 x 8192 40.2 and 32.3
// (groups of 64), 32 x 16384 x 8192 29.0 and 24.4.
static int w4_column_blocks(int64_t M, int64_t N) {
  if (w4_row_tiles(M) * ceil_div(N, 16) <= 256) return 1;
  return M > 16 && w4_row_tiles(M) * ceil_div(N, 32) > 256 ? 4 : 2;
}

template <int IN, int AR, int NT, int GS>
static hipError_t launch_w4(const W4Args &p, int waves, hipStream_t stream) {
  using T = RowsW4<AR, NT>;
  W4Args a = p;
  a.tiles_m = (int)ceil_div(p.M, 16 * T::RB);
  const int64_t tiles = a.tiles_m * ceil_div(p.N, 16 * NT);
  void *params[] = {&a};
  return hipLaunchKernel((const void *)lds_gemm_w4_kernel<IN, AR, NT, GS>, dim3((unsigned)tiles), dim3(64u * waves),
                         params, (size_t)rows_lds_bytes(waves, T::SLICE, T::RB * NT), stream);
}

template <int IN, int AR, int NT>
static hipError_t launch_w4_group(const W4Args &p, hipStream_t s) {
  const int waves = w4_waves(p.K);
  if (p.gshift == 5) return launch_w4<IN, AR, NT, 1>(p, waves, s);
  if (p.gshift == 6) return launch_w4<IN, AR, NT, 2>(p, waves, s);
  return launch_w4<IN, AR, NT, 4>(p, waves, s);
}

template <int IN, int AR>
static hipError_t launch_w4_columns(const W4Args &p, hipStream_t s) {
  const int blocks = w4_column_blocks(p.M, p.N);
  if constexpr (AR > 16)
    if (blocks == 4) return launch_w4_group<IN, AR, 4>(p, s);
  if (blocks == 2) return launch_w4_group<IN, AR, 2>(p, s);
  return launch_w4_group<IN, AR, 1>(p, s);
}

template <int IN>
static hipError_t dispatch_w4(const W4Args &p, hipStream_t s) {
  switch (w4_rows(p.M)) {
    case 4: return launch_w4_columns<IN, 4>(p, s);
    case 16: return launch_w4_columns<IN, 16>(p, s);
    case 32: return launch_w4_columns<IN, 32>(p, s);
    default: return launch_w4_columns<IN, 48>(p, s);
  }
}

}  // namespace lsm

extern "C" int gemm_w4_run(gemm_handle_t h, const void *A, const void *B, const void *S, const void *Z, void *C,
                           int64_t M, int64_t N, int64_t K, int64_t group, int64_t lda, int64_t ldb, int64_t lds,
                           int64_t ldz, int64_t ldc, int dtype, hipStream_t stream) {
  using namespace lsm;
  if (!h || M < 0 || N < 0 || K < 0 || group < 1) return GEMM_ERR_INVALID_ARG;
  if (dtype < GEMM_BF16_F32 || dtype > GEMM_F16_F32) return GEMM_ERR_INVALID_ARG;
  const bool out_f32 = dtype == GEMM_BF16_F32 || dtype == GEMM_F16_F32;
  if (M == 0 || N == 0) return GEMM_OK;
  if (!C || (K > 0 && (!A || !B || !S))) return GEMM_ERR_INVALID_ARG;
  if (ldc < N || (K > 0 && (lda < K || ldb < K || lds < N || (Z && ldz < N)))) return GEMM_ERR_INVALID_ARG;

  const int64_t kMaxDim = (int64_t)1 << 30, kMaxLd = (int64_t)1 << 40;
  if (M >= kMaxDim || N >= kMaxDim || K >= kMaxDim) return GEMM_ERR_UNSUPPORTED;
  if (lda >= kMaxLd || ldb >= kMaxLd || lds >= kMaxLd || (Z && ldz >= kMaxLd) || ldc >= kMaxLd)
    return GEMM_ERR_UNSUPPORTED;
  // 32-bit offsets inside a tile of 48 rows and 64 columns
  if (K > 0 && (lda >= ((int64_t)1 << 24) || ldb >= ((int64_t)1 << 25))) return GEMM_ERR_UNSUPPORTED;
  // groups of a power of two of at least 32, and whole 32s of K
  if (group < 32 || (group & (group - 1)) || group > kMaxDim || K % 32) return GEMM_ERR_UNSUPPORTED;
  // a launch holds fewer than 2^32 threads
  if (w4_row_tiles(M) * ceil_div(N, 16 * w4_column_blocks(M, N)) * 64 * w4_waves(K) >= ((int64_t)1 << 32))
    return GEMM_ERR_UNSUPPORTED;
  if ((uintptr_t)C & (out_f32 ? 3 : 1)) return GEMM_ERR_UNSUPPORTED;
  if (K > 0 && (((uintptr_t)A & 15) || ((uintptr_t)B & 15) || ((uintptr_t)S & 1) || lda % 8 || ldb % 32))
    return GEMM_ERR_UNSUPPORTED;

  const int64_t G = ceil_div(K, group);
  const int64_t c_bytes = footprint_bytes(M, ldc, N, out_f32 ? 4 : 2);
  const int64_t a_bytes = K > 0 ? footprint_bytes(M, lda, K, 2) : 0;
  const int64_t b_bytes = K > 0 ? footprint_bytes(N, ldb / 2, K / 2, 1) : 0;
  const int64_t s_bytes = K > 0 ? footprint_bytes(G, lds, N, 2) : 0;
  const int64_t z_bytes = K > 0 && Z ? footprint_bytes(G, ldz, N, 1) : 0;
  if (c_bytes < 0 || a_bytes < 0 || b_bytes < 0 || s_bytes < 0 || z_bytes < 0) return GEMM_ERR_UNSUPPORTED;
  if (K > 0 && (ranges_overlap(C, c_bytes, A, a_bytes) || ranges_overlap(C, c_bytes, B, b_bytes) ||
                ranges_overlap(C, c_bytes, S, s_bytes) || (Z && ranges_overlap(C, c_bytes, Z, z_bytes))))
    return GEMM_ERR_INVALID_ARG;

  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != h->device) return GEMM_ERR_DEVICE;
  // Without zero points the kernel reads S's first row in their place and counts 8.
  const W4Args p{(const uint16_t *)A, (const uint8_t *)B, (const uint16_t *)S, (const uint8_t *)(Z ? Z : S), C,
                 (int)M, (int)N, (int)K, (int)G, __builtin_ctzll((unsigned long long)group),
                 lda, ldb / 2, lds, Z ? ldz : 0, ldc, 1, out_f32 ? 1 : 0, Z ? 255u : 0u, Z ? 0u : 8u};
  const bool bf16 = dtype == GEMM_BF16_F32 || dtype == GEMM_BF16_BF16;
  const hipError_t e = bf16 ? dispatch_w4<IN_BF16>(p, stream) : dispatch_w4<IN_F16>(p, stream);
  return e == hipSuccess ? GEMM_OK : GEMM_ERR_LAUNCH;
}
