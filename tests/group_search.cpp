// group_search.cpp -- gemm_groups.h on the CPU: 64 coroutines are the lanes of one wave, and a cross-lane operation
// of the header is a value that each lane leaves before all of them go on.  Built with a copy of the header
// beside stand-ins for its includes (test_group_search.py).
//
//   group_search rows  MOST BM ALIGN G T tiles_n group_m first last OLD.. [NEW..]
//       find_row_tile for workgroups first .. last - 1: "g first last before tiles tile sub parts tm tn"
//       or "none".  A second set of ends takes the first one's place between the two passes over them.
//   group_search sums  BY_SIZE G T ENDS..
//       find_group for every place: "g first last".
#include <ucontext.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <functional>
#include <vector>

#include "gemm_groups.h"

namespace wave {
ucontext_t lanes[64], scheduler;
bool ended[64];
int lane;                           // the one that runs
int value[2][64], turn[64];         // two sets, so that a lane may leave its next value before all have read the last
std::function<void(int)> body;

// f(all lanes' x).
template <class F>
static auto exchange(int x, F f) {
  const int l = lane, t = turn[l]++ & 1;
  value[t][l] = x;
  swapcontext(&lanes[l], &scheduler);
  return f(value[t]);
}

static void start() {
  const int l = lane;
  body(l);
  ended[l] = true;
  swapcontext(&lanes[l], &scheduler);
}
static void run(std::function<void(int)> f) {
  static std::vector<char> stacks(64 << 16);
  body = f;
  for (int l = 0; l < 64; l++) {
    getcontext(&lanes[l]);
    lanes[l].uc_stack.ss_sp = &stacks[l << 16], lanes[l].uc_stack.ss_size = 1 << 16, lanes[l].uc_link = &scheduler;
    makecontext(&lanes[l], start, 0);
    ended[l] = false, turn[l] = 0;
  }
  for (bool left = true; left;) {
    left = false;
    for (lane = 0; lane < 64; lane++)
      if (!ended[lane]) swapcontext(&scheduler, &lanes[lane]), left = true;
  }
}
}  // namespace wave

int lane_shfl_up(int x, int n) {
  return wave::exchange(x, [&](const int *v) { return wave::lane < n ? x : v[wave::lane - n]; });
}
int lane_readlane(int x, int l) {
  return wave::exchange(x, [&](const int *v) { return v[l]; });
}
uint64_t lane_ballot(bool p) {
  return wave::exchange(p, [&](const int *v) {
    uint64_t m = 0;
    for (int l = 0; l < 64; l++) m |= (uint64_t)(v[l] != 0) << l;
    return m;
  });
}
// row_shr:n (0x110 + n), row_bcast:15 (0x142), row_bcast:31 (0x143); lanes without a source, or in rows that
// the mask leaves out, keep `old`.
int lane_update_dpp(int old, int x, int ctrl, int rows, int, bool) {
  return wave::exchange(x, [&](const int *v) {
    const int l = wave::lane, row = l / 16;
    if (!(rows >> row & 1)) return old;
    int from = -1;
    if (ctrl == 0x142 && row > 0) from = 16 * row - 1;
    else if (ctrl == 0x143 && row >= 2) from = 31;
    else if (ctrl > 0x110 && ctrl < 0x120 && l % 16 >= ctrl - 0x110) from = l - (ctrl - 0x110);
    return from < 0 ? old : v[from];
  });
}

static std::vector<int32_t> ends, next;
// Between the passes (xcd_logical_id is called there): the new ends, by lane 0 alone.
void between_passes() {
  wave::exchange(0, [](const int *) { return 0; });
  if (wave::lane == 0 && !next.empty()) ends = next;
  wave::exchange(0, [](const int *) { return 0; });
}

template <int BM, int ALIGN, int MOST>
static void rows(int G, int T, int tiles_n, int group_m, int from, int to, const std::vector<int32_t> &old) {
  for (int bid = from; bid < to; bid++) {
    ends = old;
    wave::run([=](int l) {
      lsm::Group at{};
      lsm::Part p{};
      int tm = -1, tn = -1;
      const bool found = lsm::find_row_tile<BM, ALIGN, MOST>(ends.data(), G, T, tiles_n, group_m, bid, l, at, p, tm, tn);
      if (l != 0) return;
      if (found)
        std::printf("%d %d %d %d %d %d %d %d %d %d\n", at.g, at.first, at.last, at.before, at.tiles, p.tile, p.sub, p.parts,
                    tm, tn);
      else
        std::printf("none\n");
    });
  }
}

int main(int n, char **a) {
  auto num = [&](int i) { return i < n ? std::atoi(a[i]) : 0; };
  auto list = [&](int i, int count) {
    std::vector<int32_t> v;
    for (int j = 0; j < count && i + j < n; j++) v.push_back(std::atoi(a[i + j]));
    return v;
  };
  if (!std::strcmp(a[1], "rows")) {
    const int most = num(2), bm = num(3), align = num(4), G = num(5), T = num(6);
    const auto old = list(11, G);
    next = list(11 + G, G);
    auto go = most == 4 && align == 16 ? rows<256, 16, 4> : most == 4 ? rows<256, 1, 4> : bm == 16 ? rows<16, 1, 1> : rows<128, 1, 1>;
    go(G, T, num(7), num(8), num(9), num(10), old);
    return 0;
  }
  const int by_size = num(2), G = num(3), T = num(4);
  ends = list(5, G);
  wave::run([=](int l) {
    for (int at = 0; at < G; at++) {
      const lsm::Group g = by_size ? lsm::find_group<true>(ends.data(), G, T, at, l) : lsm::find_group<false>(ends.data(), G, T, at, l);
      if (l == 0) std::printf("%d %d %d\n", g.g, g.first, g.last);
    }
  });
  return 0;
}
