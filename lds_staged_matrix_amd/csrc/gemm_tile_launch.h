// gemm_tile_launch.h -- host side shared by the grouped and the MXFP4 products:
// launches of the kernels of gemm_kernel_tile.h and gemm_kernel_tile256.h, and
// argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "gemm_kernel_tile.h"
#include "gemm_kernel_tile256.h"
#include "gemm_launch.h"

namespace lsm {

// Workgroups of tiles of bm x bn.
template <int MODE>
static int64_t workgroups(const TileArgs &p, int bm, int bn, int align = 1) {
  const int64_t tn = ceil_div(p.N, bn);
  if (MODE == GROUP_ROWS) return most_row_tiles(p.M, p.G, bm, align) * tn;
  return ceil_div(p.M, bm) * tn * (MODE == GROUP_SUMS ? p.G : 1);
}

// Tiles that groups of rows have, as far as the host can tell: a group of the mean
// number of rows ends in half a tile, and one of fewer rows has a tile all the same.
static int64_t expected_tiles(const TileArgs &p, int bm, int bn) {
  const int64_t used = p.G < p.M ? p.G : p.M;
  const int64_t halves = 2 * (int64_t)p.M / bm + used;
  return (halves > 2 * used ? halves / 2 : used) * ceil_div(p.N, bn);
}

// The launch that a product takes.
struct Plan {
  const void *kernel;
  int mode, bm, bn, threads, align, parts;
};

template <int MODE, int LA, int LB, int IN, int OUT>
static Plan plan_tile256() {
  return {(const void *)lds_gemm_tile256_kernel<MODE, LA, LB, IN, OUT>, MODE, 256, 256, 512, tile_align<IN, MODE>(),
          tile256_parts(LA)};
}
template <class S, int MODE, int LA, int LB, int IN, int OUT>
static Plan plan_tile() {
  return {(const void *)lds_gemm_tile_kernel<S, MODE, LA, LB, IN, OUT>, MODE, S::BM, S::BN, S::NT * S::WK, 1, 1};
}
template <class S, int MODE, int LB, int IN, int OUT>
static Plan plan_stream() {
  return {(const void *)lds_gemm_stream_kernel<S, MODE, LB, IN, OUT>, MODE, S::BM, S::BN, 64 * S::WAVES, 1, 1};
}

static int64_t plan_workgroups(const Plan &l, const TileArgs &p) {
  const int64_t n = l.mode == GROUP_ROWS   ? workgroups<GROUP_ROWS>(p, l.bm, l.bn, l.align)
                    : l.mode == GROUP_SUMS ? workgroups<GROUP_SUMS>(p, l.bm, l.bn)
                                           : workgroups<GROUP_NONE>(p, l.bm, l.bn);
  return workgroups_in_parts(n, l.parts, l.mode != GROUP_ROWS);
}
// A launch holds fewer than 2^32 threads.
static bool plan_fits(const Plan &l, const TileArgs &p) { return plan_workgroups(l, p) < ((int64_t)1 << 32) / l.threads; }

// Enqueue the plan on the handle's device; a gemm_status.
static int run_plan(gemm_handle_t h, const Plan &l, TileArgs p, hipStream_t stream) {
  if (!plan_fits(l, p)) return GEMM_ERR_UNSUPPORTED;
  int dev = -1;
  if (hipGetDevice(&dev) != hipSuccess || dev != h->device) return GEMM_ERR_DEVICE;
  p.tiles_m = l.mode == GROUP_ROWS ? 0 : (int)ceil_div(p.M, l.bm);
  p.tiles_n = (int)ceil_div(p.N, l.bn);
  void *params[] = {&p};
  return hipLaunchKernel(l.kernel, dim3((unsigned)plan_workgroups(l, p)), dim3((unsigned)l.threads), params, 0, stream) ==
                 hipSuccess
             ? GEMM_OK
             : GEMM_ERR_LAUNCH;
}

// call(OUT) with the output type as a constant.
template <class F>
static Plan with_out(int out, F call) {
  if (out == OUT_BF16) return call(std::integral_constant<int, OUT_BF16>{});
  if (out == OUT_F16) return call(std::integral_constant<int, OUT_F16>{});
  return call(std::integral_constant<int, OUT_F32>{});
}

// Groups: a workgroup reads all their ends.
constexpr int64_t kMaxGroups = (int64_t)1 << 16;
constexpr int64_t kTileMaxDim = (int64_t)1 << 30, kTileMaxLd = (int64_t)1 << 40;
// Bytes of an operand's leading dimension: 256 rows of it stay within 2^30.
constexpr int64_t kTileMaxPitch = (int64_t)1 << 22;
// Of a scales' row: 8 of them stay within 2^30.
constexpr int64_t kScaleMaxPitch = (int64_t)1 << 27;

// A span of memory that an argument stands for.
struct Span {
  const void *p;
  int64_t bytes;
};
static bool overlaps_any(const Span &out, std::initializer_list<Span> in) {
  for (const Span &s : in)
    if (s.p && s.bytes > 0 && ranges_overlap(out.p, out.bytes, s.p, s.bytes)) return true;
  return false;
}

// Bytes from the first of `n` matrices of `one` bytes to the end of the last, -1
// beyond 63 bits.
static int64_t stacked_bytes(int64_t n, int64_t stride, int64_t one) {
  int64_t r;
  if (one < 0 || __builtin_mul_overflow(n - 1, stride, &r) || __builtin_add_overflow(r, one, &r)) return -1;
  return r;
}

}  // namespace lsm
