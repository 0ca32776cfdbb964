// gemm_tile_launch.h -- host side shared by the grouped and the MXFP4 products:
// launches of the kernels of gemm_kernel_tile.h and gemm_kernel_tile256.h, and
// argument checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
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
// number of rows ends in half a tile, and one of few rows has a tile all the same.
static float expected_tiles(const TileArgs &p, int bm, int bn) {
  const int used = p.G < p.M ? p.G : p.M;
  if (used == 1) return (float)(ceil_div(p.M, bm) * ceil_div(p.N, bn));
  const float rows = (float)p.M / (float)bm + 0.5f * (float)used;
  return (rows > (float)used ? rows : (float)used) * (float)ceil_div(p.N, bn);
}

// What a shape of tiles takes, in microseconds, the launch left out: `fixed` for a
// round of `slots` workgroups, and for each K tile `full` where the round fills all
// slots and `half` where it fills half or fewer.  The figures were fitted to times
// measured on MI355X, every shape at 3800 sizes: N and K (M and N of the sums) from 256
// to 8192, one to 32 groups, mostly uneven, of up to 16384 rows in all.  The shape
// chosen is slower than the fastest by 1.9% in the mean (16 bits), 1.5% (MXFP4) and
// 2.6% (sums).
struct Cost {
  int slots;
  float fixed, full, half;
};
// K tiles.  Where groups are so short (up to 512 rows in the mean) that their
// matrices come from HBM, each takes a fifth longer.
static float k_tiles(const TileArgs &p, int in) {
  const float k = (float)ceil_div(p.K, kTileK(in));
  return p.G > 1 && ceil_div(p.M, p.G) <= 512 ? 1.2f * k : k;
}
static float round_time(const Cost &c, float share, float ktiles) {
  return c.fixed + ktiles * (c.half + (c.full - c.half) * (share > 0.5f ? 2 * share - 1 : 0.f));
}
static float tiles_time(const Cost &c, float tiles, float ktiles) {
  const float rounds = tiles / (float)c.slots, whole = floorf(rounds), rest = rounds - whole;
  return whole * round_time(c, 1.f, ktiles) + (rest > 0.f ? round_time(c, rest, ktiles) : 0.f);
}
// The 256 x 256 tile, whose last round is cut into parts: `half` and `quarter` are a
// K tile of so much of a tile.
struct Cost256 {
  float fixed, full, half, quarter;
};
static float tile256_time(const Cost256 &c, float tiles, float ktiles, int most) {
  const float whole = floorf(tiles / kCUs), rest = tiles - whole * kCUs;
  const int parts = rest_parts((int)ceilf(rest), most);
  const float last = parts == 4 ? c.quarter : parts == 2 ? c.half : c.full;
  return whole * (c.fixed + ktiles * c.full) + (rest > 0.f ? c.fixed + ktiles * last : 0.f);
}

// The launch that a product takes.
struct Plan {
  const void *kernel;
  int mode, bm, bn, threads, align, parts, slots;       // `slots`: workgroups at once
};

template <int MODE, int LA, int LB, int IN, int OUT>
static Plan plan_tile256() {
  return {(const void *)lds_gemm_tile256_kernel<MODE, LA, LB, IN, OUT>, MODE, 256, 256, 512, tile_align<IN, MODE>(),
          tile256_parts(LA), kCUs};
}
template <class S, int MODE, int LA, int LB, int IN, int OUT>
static Plan plan_tile() {
  return {(const void *)lds_gemm_tile_kernel<S, MODE, LA, LB, IN, OUT>, MODE, S::BM, S::BN, S::NT * S::WK, 1, 1,
          kCUs * S::PER_CU};
}
template <class S, int MODE, int LB, int IN, int OUT>
static Plan plan_stream() {
  return {(const void *)lds_gemm_stream_kernel<S, MODE, LB, IN, OUT>, MODE, S::BM, S::BN, 64 * S::WAVES, 1, 1, 0};
}

// The cheaper of the plans so far and of a shape's.
struct Cheapest {
  Plan plan;
  float time;
  void offer(const Plan &l, float t) {
    if (t < time) plan = l, time = t;
  }
};

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
  p.by_size = l.mode == GROUP_SUMS && p.G > 1 && plan_workgroups(l, p) > l.slots;
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
