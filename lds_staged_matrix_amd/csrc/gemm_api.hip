// gemm_api.hip -- the C ABI declared in include/lds_gemm.h: argument
// validation, choice of kernel and tile shape, and the launch on the
// caller's stream.  The kernels: the ping-pong kernel (gemm_kernel_pingpong.h,
// shapes with at least 256 tiles of 256 x 256), the direct-to-LDS kernel
// (gemm_kernel_dma.h, 128 and 64 tiles), the split-K ring kernel
// (gemm_kernel_skinny.h, M <= 32) and the register-staged kernel
// (gemm_kernel.h, shapes the 16-byte direct-to-LDS loads cannot take).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <new>

#include "gemm_launch.h"

namespace lsm {

// Shape classes.  M <= 32 takes the split-K ring kernel (HBM-bound).
// Otherwise the big tile when it still gives every CU at least one
// workgroup, else the 128 tile when that does, else the 64 tile (a short,
// latency-bound K loop per workgroup; more workgroups hide more of it),
// with four LDS stages when its operand panels overflow the L2.
// Shapes whose contiguous extents are not whole 16-byte chunks (dma_ok()
// false) take the register-staged kernel of the same class.
// 8-bit inputs run on the direct-to-LDS kernels only (gemm_run rejects fp8
// shapes those cannot take).
static hipError_t dispatch(const Args &a, int la, int lb, int dtype, hipStream_t s) {
  const int64_t t256 = ceil_div(a.M, 256) * ceil_div(a.N, 256);
  const int64_t t128 = ceil_div(a.M, 128) * ceil_div(a.N, 128);
  if (is_fp8(dtype)) {
    if (a.M <= 32) return launch_fp8<SkinnyStream8, SKINNY>(a, la, lb, dtype, s);
    if (t256 >= 256) return launch_fp8<PingPong8, PINGPONG>(a, la, lb, dtype, s);
    if (t128 >= 256) return launch_fp8<DmaMid8, DMA>(a, la, lb, dtype, s);
    if (small_tile_four_stages(a, 1)) return launch_fp8<DmaSmall8, DMA4>(a, la, lb, dtype, s);
    return launch_fp8<DmaSmall8, DMA>(a, la, lb, dtype, s);
  }
  const bool dma = dma_ok(a, la, lb, 2);
  if (dma) {
    if (a.M <= 32) return launch_dtype<SkinnyStream, SKINNY>(a, la, lb, dtype, s);
    if (t256 >= 256) return launch_dtype<PingPong, PINGPONG>(a, la, lb, dtype, s);
    if (t128 >= 256) return launch_dtype<DmaMid, DMA>(a, la, lb, dtype, s);
    if (small_tile_four_stages(a, 2)) return launch_dtype<DmaSmall, DMA4>(a, la, lb, dtype, s);
    return launch_dtype<DmaSmall, DMA>(a, la, lb, dtype, s);
  }
  if (a.M <= 32) return launch_dtype<Skinny>(a, la, lb, dtype, s);
  if (t256 >= 256) return launch_dtype<Big>(a, la, lb, dtype, s);
  if (t128 >= 64) return launch_dtype<Mid>(a, la, lb, dtype, s);
  return launch_dtype<Small>(a, la, lb, dtype, s);
}

}  // namespace lsm

extern "C" {

#if LSM_PP_TIMELINE
// Measurement builds only: install (or, with NULL, remove) the buffer the
// ping-pong kernel writes its per-wave phase cycles to, 64 counts per
// workgroup of the launch.  0 on success, -1 on a HIP error.
int lsm_pp_timeline_set(void *buf) {
  return hipMemcpyToSymbol(HIP_SYMBOL(lsm::pp_timeline_buf), &buf, sizeof(buf)) == hipSuccess ? 0 : -1;
}
#endif

int gemm_create(gemm_handle_t *out) {
  if (!out) return GEMM_ERR_INVALID_ARG;
  *out = nullptr;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess) return GEMM_ERR_DEVICE;
  hipDeviceProp_t prop;
  if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GEMM_ERR_DEVICE;
  if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) return GEMM_ERR_DEVICE;
  gemm_ctx *h = new (std::nothrow) gemm_ctx{dev};
  if (!h) return GEMM_ERR_DEVICE;
  *out = h;
  return GEMM_OK;
}

int gemm_destroy(gemm_handle_t h) {
  delete h;
  return GEMM_OK;
}

const char *gemm_status_str(int status) {
  switch (status) {
    case GEMM_OK: return "success";
    case GEMM_ERR_INVALID_ARG: return "invalid argument";
    case GEMM_ERR_UNSUPPORTED: return "unsupported argument (alignment or size)";
    case GEMM_ERR_DEVICE: return "device is not a usable gfx950 device";
    case GEMM_ERR_LAUNCH: return "kernel launch failed";
    default: return "unknown status";
  }
}

int gemm_run(gemm_handle_t h, const void *A, const void *B, void *C, int64_t M, int64_t N,
             int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int layoutA, int layoutB,
             int dtype, hipStream_t stream) {
  using namespace lsm;
  if (!h) return GEMM_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0) return GEMM_ERR_INVALID_ARG;
  if (dtype < GEMM_BF16_F32 || dtype > GEMM_E4M3_BF16) return GEMM_ERR_INVALID_ARG;
  const int64_t out_size =
      (dtype == GEMM_BF16_F32 || dtype == GEMM_F16_F32 || dtype == GEMM_E4M3_F32) ? 4 : 2;
  const int64_t es = is_fp8(dtype) ? 1 : 2;             // input element bytes
  Args args;
  const int st = check_product(A, B, C, M, N, K, lda, ldb, ldc, layoutA, layoutB, es, out_size, args);
  if (st != GEMM_OK || M == 0 || N == 0) return st;
  // 8-bit inputs need the direct-to-LDS kernels: whole 16-element chunks
  // along both contiguous extents and 32-bit buffer offsets.
  if (is_fp8(dtype) && !dma_ok(args, layoutA, layoutB, 1)) return GEMM_ERR_UNSUPPORTED;

  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != h->device) return GEMM_ERR_DEVICE;
  if (dispatch(args, layoutA, layoutB, dtype, stream) != hipSuccess) return GEMM_ERR_LAUNCH;
  return GEMM_OK;
}

}  // extern "C"
