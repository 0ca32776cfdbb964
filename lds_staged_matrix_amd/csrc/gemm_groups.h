// gemm_groups.h -- where a workgroup of a grouped product works.
//
// The rows of A are sorted by group (expert); ends[g], on the device, is the row
// behind group g's last, and group g starts where the groups before it end.  No
// host ever reads the ends, so a launch holds as many workgroups as any ends
// could ask for, and each finds its own tile in them: every wave reads all the
// ends, 64 at a time, and scans them in registers.  A workgroup past the last
// tile leaves at once.
//
// Whatever the ends hold, the groups found are disjoint, in order and inside the
// T rows: an end counts as no less than the ends before it and no more than T.
// Ends that change while the work runs may leave waves with different tiles, and
// so with wrong results; each wave still stays inside the T rows and ends.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemm_common.h"

namespace lsm {

// How a product's work is divided among groups.
enum { GROUP_NONE = 0, GROUP_ROWS = 1, GROUP_SUMS = 2 };   // one product; rows of A and C by group; the summed rows by group

struct Group {
  int g;                // its number
  int first, last;      // its rows
  int before;           // row tiles of the groups before it
  int tiles;            // its own
};

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or_zero(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xF, false);
}

// Inclusive scans over the 64 lanes, of numbers whose neutral element is zero:
// shifts by 1, 2, 4 and 8 inside rows of 16 lanes, then lane 15 of rows 0 and 2
// to the rows after them, and lane 31 to the upper half.
template <class Op>
__device__ __forceinline__ uint32_t wave_scan(uint32_t x, Op op) {
  x = op(x, dpp_or_zero<0x111, 0xF>(x));
  x = op(x, dpp_or_zero<0x112, 0xF>(x));
  x = op(x, dpp_or_zero<0x114, 0xF>(x));
  x = op(x, dpp_or_zero<0x118, 0xF>(x));
  x = op(x, dpp_or_zero<0x142, 0xA>(x));
  x = op(x, dpp_or_zero<0x143, 0xC>(x));
  return x;
}

// Rows that a group's first tile starts early, so that tiles start at a
// multiple of ALIGN (the rows of other groups in it are not stored).
template <int ALIGN>
__device__ __forceinline__ int early_rows(int first) { return first & (ALIGN - 1); }

// The groups 64 c .. 64 c + 63, one a lane; `end` and `tiles` carry from chunk
// to chunk.
template <int BM, int ALIGN>
struct GroupChunk {
  int first, last, tiles, through;     // `through`: row tiles up to and with this group
  __device__ __forceinline__ GroupChunk(const int32_t *ends, int G, int T, int c, int lane, uint32_t &end,
                                        uint32_t &count) {
    const int g = 64 * c + lane;
    int e = g < G ? ends[g] : 0;
    e = e < 0 ? 0 : e > T ? T : e;
    uint32_t m = wave_scan((uint32_t)e, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
    m = m > end ? m : end;
    const uint32_t prev = (uint32_t)__shfl_up((int)m, 1);
    first = (int)(lane == 0 ? end : prev);
    last = (int)m;
    tiles = last > first ? (last - first + early_rows<ALIGN>(first) + BM - 1) / BM : 0;
    through = (int)(wave_scan((uint32_t)tiles, [](uint32_t a, uint32_t b) { return a + b; }) + count);
    end = (uint32_t)__builtin_amdgcn_readlane((int)m, 63);
    count = (uint32_t)__builtin_amdgcn_readlane(through, 63);
  }
  // Lane l's group.
  __device__ __forceinline__ Group at(int c, int l) const {
    const int n = __builtin_amdgcn_readlane(tiles, l);
    return {64 * c + l, __builtin_amdgcn_readlane(first, l), __builtin_amdgcn_readlane(last, l),
            __builtin_amdgcn_readlane(through, l) - n, n};
  }
};

// A workgroup's part of the work: a tile, or one of `parts` equal shares of its
// rows.
struct Part {
  int tile, sub, parts;
};

// The last `rest` tiles that do not fill the 256 CUs once more are cut into up to
// MOST parts each, as many as still fit one round: a large tile takes long, and a
// round of few of them as long as a full one (256 x 256 tiles: one group of 1500 bf16
// rows, 4096 x 4096 77 us, in parts 62; four uneven ones, 4096 x 1152 27 and 23; one MXFP4
// product of 1024 x 8192 x 8192 58 and 45).  With many rounds it hardly shows (16384 bf16
// rows, eight groups of 4096 x 4096: 442 and 440), and where HBM sets the pace it costs (2048
// rows, the same matrices: 95 and 100).
constexpr int kCUs = 256;
__host__ __device__ constexpr int rest_parts(int rest, int most) {
  return most >= 4 && 4 * rest <= kCUs ? 4 : most >= 2 && 2 * rest <= kCUs ? 2 : 1;
}
template <int MOST>
__device__ __forceinline__ bool part_of(int bid, int total, Part &w) {
  w = {bid, 0, 1};
  if constexpr (MOST == 1) return bid < total;
  const int rest = total % kCUs, full = total - rest;
  if (bid < full) return true;
  w.parts = rest_parts(rest, MOST);
  const int j = bid - full;
  if (j >= rest * w.parts) return false;
  w.sub = j / rest, w.tile = full + j - w.sub * rest;
  return true;
}
// Workgroups of `total` tiles, or of no more than that many.
constexpr int64_t workgroups_in_parts(int64_t total, int most, bool exact) {
  if (most == 1) return total;
  if (!exact) return total + kCUs * 3 / 4;             // 64 tiles in four parts, 128 in two
  const int64_t rest = total % kCUs;
  return total - rest + rest * rest_parts((int)rest, most);
}

// Workgroup `bid`'s group and its tile there, of BM rows by one of `tiles_n`
// columns; false past the last tile.  Tiles are numbered group by group, and
// each XCD has one contiguous range of the numbers.
template <int BM, int ALIGN, int MOST>
__device__ __forceinline__ bool find_row_tile(const int32_t *ends, int G, int T, int tiles_n, int group_m, int bid,
                                              int lane, Group &at, Part &part, int &tm, int &tn) {
  const int chunks = (G + 63) / 64;
  uint32_t end = 0, count = 0;
  GroupChunk<BM, ALIGN> s(ends, G, T, 0, lane, end, count);
  for (int c = 1; c < chunks; c++) GroupChunk<BM, ALIGN>(ends, G, T, c, lane, end, count);
  const int total = (int)count * tiles_n;
  if (!part_of<MOST>(bid, total, part)) return false;
  const int id = xcd_logical_id(part.tile, total), q = id / tiles_n;
  end = count = 0;
  for (int c = 0; c < chunks; c++) {
    if (chunks > 1) s = GroupChunk<BM, ALIGN>(ends, G, T, c, lane, end, count);
    const uint64_t past = __ballot(s.through > q);
    if (past) {
      at = s.at(c, __builtin_ctzll(past));
      tile_coords(id - at.before * tiles_n, at.tiles, tiles_n, group_m, tm, tn);
      return true;
    }
  }
  return false;             // the ends have changed since the first pass
}

// Group `at`, or the group at place `at` of an order in which, among each 64, those
// with more rows (in 16s) come first.
template <bool BY_SIZE>
__device__ __forceinline__ Group find_group(const int32_t *ends, int G, int T, int at, int lane) {
  uint32_t end = 0, count = 0;
  const int chunk = at / 64;
  for (int c = 0; c < chunk; c++) GroupChunk<64, 1>(ends, G, T, c, lane, end, count);
  const GroupChunk<64, 1> s(ends, G, T, chunk, lane, end, count);
  if (!BY_SIZE) return s.at(chunk, at & 63);
  // rows are fewer than 2^30; the lane makes all keys differ, and lanes without a
  // group come last
  const uint32_t key = (uint32_t)(s.last - s.first) >> 4 << 6 | (uint32_t)(63 - lane);
  const int n = G - 64 * chunk < 64 ? G - 64 * chunk : 64;
  int place = 0;
  for (int l = 0; l < n; l++) place += (uint32_t)__builtin_amdgcn_readlane((int)key, l) > key;
  return s.at(chunk, __builtin_ctzll(__ballot(place == (at & 63))));
}

// The most row tiles that any ends give: a group of r rows has at most
// (r + ALIGN - 1 + BM - 1) / BM, and at most T groups have rows.
static inline int64_t most_row_tiles(int64_t T, int64_t G, int BM, int align) {
  const int64_t used = G < T ? G : T;
  return (T + used * (BM + align - 2)) / BM;
}

}  // namespace lsm
