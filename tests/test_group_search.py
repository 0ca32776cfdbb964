"""The search of a workgroup's tile in the groups' ends (gemm_groups.h) on the CPU: the header itself, its wave
of 64 lanes as 64 coroutines (group_search.cpp).  Every tile of every group is found once, whatever the ends hold;
and the search ends, and stays inside the groups, if the ends change between its two passes."""
import os
import shutil
import subprocess

import numpy as np
import pytest

import grouped_reference as G

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "lds_staged_matrix_amd", "csrc")
STAND_INS = {"hip/hip_runtime.h": "#define __device__\n#define __host__\n#define __forceinline__ inline\n",
             "gemm_common.h": """#pragma once
#include <stdint.h>
#include "lds_layout.h"
int lane_shfl_up(int x, int n);
int lane_readlane(int x, int l);
uint64_t lane_ballot(bool p);
int lane_update_dpp(int old, int x, int ctrl, int rows, int banks, bool bound);
void between_passes();
namespace lsm {
inline int found_id(int bid, int n) { between_passes(); return xcd_logical_id(bid, n); }
}
#define xcd_logical_id found_id
#define __shfl_up lane_shfl_up
#define __ballot lane_ballot
#define __builtin_amdgcn_readlane lane_readlane
#define __builtin_amdgcn_update_dpp lane_update_dpp
"""}


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("group_search")
    for name, text in STAND_INS.items():
        path = d / name
        path.parent.mkdir(exist_ok=True)
        path.write_text(text)
    shutil.copy(os.path.join(CSRC, "gemm_groups.h"), d)
    shutil.copy(os.path.join(CSRC, "lds_layout.h"), d)
    shutil.copy(os.path.join(HERE, "group_search.cpp"), d)
    exe = str(d / "group_search")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", str(d), str(d / "group_search.cpp"), "-o", exe], check=True)

    def run(*args, timeout=60):
        out = subprocess.run([exe, *map(str, args)], check=True, capture_output=True, text=True, timeout=timeout).stdout
        return [None if l == "none" else tuple(map(int, l.split())) for l in out.splitlines()]
    return run


def ends_of(rng, groups, T, how):
    if how == "none":
        return [0] * groups
    if how == "wild":
        return [int(e) for e in rng.integers(-T, 2 * T, groups)]
    return [int(e) for e in np.sort(rng.integers(0, T + 1, groups))]


@pytest.mark.parametrize("groups,T", [(1, 700), (5, 900), (63, 1500), (64, 1500), (65, 1500), (130, 2000)])
@pytest.mark.parametrize("how", ["sorted", "wild", "none"])
@pytest.mark.parametrize("most,bm,align", [(1, 128, 1), (4, 256, 1), (4, 256, 16)])
def test_every_row_tile_once(search, groups, T, how, most, bm, align):
    rng = np.random.default_rng([groups, T, most, align, len(how)])
    ends, tiles_n = ends_of(rng, groups, T, how), 2
    # as many workgroups as the host launches for these groups, or a sample of them
    bound = (T + min(groups, T) * (bm + align - 2)) // bm * tiles_n + (192 if most > 1 else 0)
    spans = G.bounds(ends, T)
    per = [-(-(l - f + f % align) // bm) if l > f else 0 for f, l in spans]
    total = sum(per) * tiles_n
    rest = total % 256
    parts = 4 if most == 4 and 4 * rest <= 256 else 2 if most == 4 and 2 * rest <= 256 else 1
    work = total - rest + rest * parts
    assert work <= bound
    # (group, row tile, column, part) of every workgroup that has work, and none behind
    got = search("rows", most, bm, align, groups, T, tiles_n, 8, 0, min(work + 2, bound), *ends)
    assert got[work:] == [None] * (min(work + 2, bound) - work) and None not in got[:work]
    seen = set()
    for g, first, last, before, tiles, tile, sub, n, tm, tn in got[:work]:
        assert (first, last) == spans[g] and tiles == per[g] and before == sum(per[:g])
        assert 0 <= tm < tiles and 0 <= tn < tiles_n and n == (parts if tile >= total - rest else 1) and 0 <= sub < n
        seen.add((g, tm, tn, sub))
    assert len(seen) == work


@pytest.mark.parametrize("groups", [1, 7, 64, 65, 150])
@pytest.mark.parametrize("by_size", [0, 1])
def test_every_group_once(search, groups, by_size):
    rng = np.random.default_rng([groups, by_size])
    ends = ends_of(rng, groups, 5000, "wild" if groups == 7 else "sorted")
    spans = G.bounds(ends, 5000)
    got = search("sums", by_size, groups, 5000, *ends)
    assert sorted(got) == [(g, *s) for g, s in enumerate(spans)]
    if by_size:
        for c in range(0, groups, 64):
            sizes = [(l - f) // 16 for _, f, l in got[c:c + 64]]
            assert sizes == sorted(sizes, reverse=True)


@pytest.mark.parametrize("groups,old,new", [(70, [1000] * 70, [0] * 70), (130, [10 * i for i in range(130)], [0] * 130),
                                            (130, [1300] * 130, [10] * 130), (40, [1000] * 40, [0] * 40),
                                            (70, [0] * 69 + [1300], [1300] * 70)])
def test_ends_that_change_meanwhile(search, groups, old, new):
    """The caller must not write the ends while the work runs; if it does, the search ends all the same and what it
    finds lies in one of the two sets of groups."""
    T = 1300
    got = search("rows", 1, 128, 1, groups, T, 1, 8, 0, 8, *old, *new, timeout=20)
    spans = set(enumerate(G.bounds(old, T))) | set(enumerate(G.bounds(new, T)))
    for r in got:
        if r is not None:
            g, first, last, _, tiles, _, _, _, tm, tn = r
            assert (g, (first, last)) in spans and 0 <= tm < tiles and tn == 0
