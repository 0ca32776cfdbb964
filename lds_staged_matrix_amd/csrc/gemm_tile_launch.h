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

template <int MODE>
static hipError_t launch_tiles(const void *kernel, TileArgs p, int bm, int bn, int threads, hipStream_t s, int align = 1,
                               int parts = 1) {
  p.tiles_m = MODE == GROUP_ROWS ? 0 : (int)ceil_div(p.M, bm);
  p.tiles_n = (int)ceil_div(p.N, bn);
  void *params[] = {&p};
  const int64_t grid = workgroups_in_parts(workgroups<MODE>(p, bm, bn, align), parts, MODE != GROUP_ROWS);
  return hipLaunchKernel(kernel, dim3((unsigned)grid), dim3((unsigned)threads), params, 0, s);
}

template <int MODE, int LA, int LB, int IN, int OUT>
static hipError_t launch_tile256(const TileArgs &p, hipStream_t s) {
  return launch_tiles<MODE>((const void *)lds_gemm_tile256_kernel<MODE, LA, LB, IN, OUT>, p, 256, 256, 512, s,
                            tile_align<IN, MODE>(), tile256_parts(LA));
}
template <class S, int MODE, int LA, int LB, int IN, int OUT>
static hipError_t launch_tile(const TileArgs &p, hipStream_t s) {
  return launch_tiles<MODE>((const void *)lds_gemm_tile_kernel<S, MODE, LA, LB, IN, OUT>, p, S::BM, S::BN, S::NT * S::WK, s);
}
template <class S, int MODE, int LB, int IN, int OUT>
static hipError_t launch_stream(const TileArgs &p, hipStream_t s) {
  return launch_tiles<MODE>((const void *)lds_gemm_stream_kernel<S, MODE, LB, IN, OUT>, p, S::BM, S::BN, 64 * S::WAVES, s);
}

// call(OUT) with the output type of an enum gemm_mxfp4_dtype as a constant.
template <class F>
static hipError_t with_out(int out, F call) {
  if (out == OUT_BF16) return call(std::integral_constant<int, OUT_BF16>{});
  if (out == OUT_F16) return call(std::integral_constant<int, OUT_F16>{});
  return call(std::integral_constant<int, OUT_F32>{});
}

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
