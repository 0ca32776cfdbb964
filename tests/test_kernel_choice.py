"""Which kernel the host chooses for the sizes of the GPU tests of the grouped and of the MXFP4 products, recorded on
the CPU (launches.py), so that another choice of shapes cannot leave a kernel, or a form of one, without its tests:
a size that moves shows here, and its test gets another size that reaches the kernel."""
import collections

import pytest

import grouped_reference as G
import launches as L
import lds_staged_matrix_amd as lsm
import test_gpu_grouped as grouped
import test_gpu_long_k as long_k
import test_gpu_mxfp4 as mxfp4
import test_gpu_mxfp4_range as mx_range
import test_gpu_tile256 as tile256
from tile_checks import ends_of, rows_in_all, uneven

A = [(i + 1) << 44 for i in range(6)]          # made-up addresses


def rows(T, groups, N, K, layout="K"):
    ldb, b = (K, N * K) if layout == "K" else (G.up(N, 8), G.up(N, 8) * K)
    return ("gemm_grouped_run", (A[0], A[1], A[2], A[3], groups, T, N, K, K, ldb, b, N, int(layout == "MN"), lsm.GEMM_BF16_F32))


def sums(T, groups, M, N, out="f32"):
    return ("gemm_grouped_wgrad_run", (A[0], A[1], A[2], A[3], groups, T, M, N, M, N, N, M * N,
                                       lsm.GEMM_BF16_F32 if out == "f32" else lsm.GEMM_BF16_BF16))


def product(M, N, K):
    return ("gemm_mxfp4_run", (A[0], A[1], A[2], A[3], A[4], M, N, K, K, K, N, G.up(M, 16), G.up(N, 16), lsm.GEMM_MXFP4_F32))


def mx_rows(T, groups, N, K):
    n = G.up(N, 16)
    return ("gemm_grouped_mxfp4_run", (*A, groups, T, N, K, K, K, N * K, N, G.up(T, 16), n, n * K // 32, lsm.GEMM_MXFP4_F32))


def shapes(calls):
    return [L.shape(name) for name, _, _ in L.launches(calls)]


# ------------------------------------------------- the sizes that name a kernel

def cases_256():
    """(call, K tiles (of the longest group), [(rows of a tile's form, parts)] of the launch)"""
    out = []
    for name, (n, N, Ks) in tile256.GROUPS.items():
        spans, T = G.bounds(ends_of(n), sum(n)), rows_in_all(n)
        for K in Ks:
            out += [(rows(T, len(n), N, K, l), L.cdiv(K, 64), L.tiles_of_rows(spans, N, 1)) for l in ("K", "MN")]
        out += [(mx_rows(T, len(n), N, K), L.cdiv(K, 256), L.tiles_of_rows(spans, N, 16)) for K in tile256.MX_K]
    for name, (M, N, Ks) in tile256.PRODUCTS.items():
        out += [(product(M, N, K), L.cdiv(K, 256), L.tiles_of_rows([(0, M)], N, 1)) for K in Ks]
    out += [(product(16384, 8192, K), L.cdiv(K, 256), L.tiles_of_rows([(0, 16384)], 8192, 1)) for K in (0, 64)]
    for name, (n, M, N, types) in tile256.SUMS.items():
        out += [(sums(rows_in_all(n), len(n), M, N, t), max(L.cdiv(r, 64) for r in n), L.tiles_of_sums(len(n), M, N)) for t in types]
    n, N, _ = tile256.GROUPS["whole"]
    out += [(rows(sum(n) + 2, len(n), N, 0, l), 0, []) for l in ("K", "MN")]
    n, M, N, _ = tile256.SUMS["more than a round, halves"]
    return out + [(sums(sum(n), len(n), M, N), 0, [])]


def test_sizes_of_the_256_tile():
    cases = cases_256()
    for (call, _, tiles), (name, grid, block) in zip(cases, L.launches([c for c, _, _ in cases])):
        assert L.shape(name) == "256x256" and block == 512, (call, name)
        assert grid >= len(tiles), (call, grid, len(tiles))


def test_forms_of_the_256_tile():
    """In every kernel of its kind: tiles of 256, 128 and 64 rows, alone and as halves and quarters, each over one K tile,
    as many as come with the start, and enough for the stages to come round twice; the gradient also by size in more
    than one round, halves among them."""
    seen = collections.defaultdict(set)
    for (entry, args), k_tiles, tiles in cases_256():
        kind = entry if entry != "gemm_grouped_run" else entry + str(args[-2])
        for form in set(tiles):
            seen[kind, form].add(k_tiles)
    for kind in ("gemm_grouped_run0", "gemm_grouped_run1", "gemm_grouped_mxfp4_run", "gemm_mxfp4_run"):
        for rows_ in (256, 64):
            assert seen[kind, (rows_, 1)] >= {1, 2} and max(seen[kind, (rows_, 1)]) >= 7, (kind, rows_, seen[kind, (rows_, 1)])
        for form in ((128, 2), (64, 4)):
            assert min(seen[kind, form]) <= 4 and max(seen[kind, form]) >= 7, (kind, form, seen[kind, form])
    for kind in ("gemm_grouped_run0", "gemm_grouped_run1", "gemm_grouped_mxfp4_run"):
        assert max(seen[kind, (128, 1)]) >= 7 and max(seen[kind, (64, 2)]) >= 7, kind
    for form in ((256, 1), (128, 1), (128, 2)):
        assert max(seen["gemm_grouped_wgrad_run", form]) >= 7
    n, M, N, types = tile256.SUMS["more than a round, halves"]
    tiles = L.tiles_of_sums(len(n), M, N)
    assert len(tiles) > 256 and {f for f, _ in tiles} == {256, 128} and {p for _, p in tiles} == {1, 2}


@pytest.mark.parametrize("cases,call", [(long_k.ROWS_K, rows), (long_k.ROWS_MN, lambda *c: rows(*c, "MN")),
                                        (long_k.SUMS, lambda *c: sums(*c[:4])), (long_k.SUMS, lambda *c: sums(*c[:4], "16")),
                                        (long_k.PRODUCTS, product), (long_k.MX_ROWS, mx_rows)],
                         ids=["rows K", "rows MN", "sums f32", "sums 16", "product", "mx rows"])
def test_sizes_over_many_k_tiles(cases, call):
    """Each case takes the kernel that it names, with K tiles for its stages to come round twice in every wave group."""
    assert dict(zip(cases, shapes([call(*c) for c in cases.values()]))) == {k: k for k in cases}
    for kernel, c in cases.items():
        k_tiles = max(L.cdiv(n, 64) for n in uneven(*c[:2])) if cases is long_k.SUMS else \
            L.cdiv(c[-1], 256 if cases in (long_k.PRODUCTS, long_k.MX_ROWS) else 64)
        f = kernel.split()
        stages, sharing = (2, int(f[-1])) if f[0] == "stream" else (int(f[2]), int(f[-1]) if "by" in f else 1)
        assert k_tiles > 2 * stages * sharing, (kernel, k_tiles)


# ------------------------------------- the sizes of the tests by group patterns

S16, S32, S64, S128 = "stream 16x16", "stream 16x32", "stream 16x64", "stream 16x128"
T128, T128A, T64, T64K = "tile 128x128, 2 stages", "tile 128x128, 3 stages", "tile 64x128, 2 stages", "tile 64x128, 3 stages, K by 2"
Q64, Q64K, T32K = "tile 64x64, 2 stages", "tile 64x64, 3 stages, K by 2", "tile 32x64, 3 stages, K by 2"
CHOSEN = {
    "rows K": [S16 + " of 8"] * 2 + [S32 + " of 4"] * 2 + ["stream 32x16 of 8"] * 2 + [T32K, T64K] + [T64] * 3 + ["256x256"] * 2 +
              [S64 + " of 4", "stream 32x64 of 4", "stream 32x32 of 4", T32K, S64 + " of 4", "stream 32x64 of 4", Q64K, T128A, T128A,
               T128, T128],
    "rows MN": [S64 + " of 4"] * 4 + ["stream 32x64 of 4"] * 2 + [T32K, T64K] + [T64] * 3 + ["256x256"] * 2 +
               [S128 + " of 4", "stream 32x128 of 2", "stream 32x64 of 4", T32K, S128 + " of 4", "stream 32x128 of 2", Q64K, T128A,
                T128A, T128, T128],
    "sums f32": [Q64] * 4 + [Q64K, T128, Q64, T128, T128, Q64, "256x256", Q64, Q64, T64K, T128A],
    "sums 16": [Q64] * 4 + [Q64K, T128, Q64, T128, T128, Q64, "256x256", Q64, Q64, T64K, Q64],
    "mx rows": [S16 + " of 4"] * 3 + [S32 + " of 4"] + ["stream 32x32 of 4"] * 2 + [S64 + " of 2", "stream 32x64 of 2", T32K, Q64, Q64,
                Q64, T64, "256x256", T64, T32K, T128, Q64K, T128A, T64K, S128 + " of 2"],
    "products": [S16 + " of 4"] * 4 + [S32 + " of 4"] * 2 + [S64 + " of 2"] + ["stream 32x32 of 4"] * 2 + ["stream 32x64 of 2"] +
                ["stream 32x32 of 4", Q64, "stream 32x32 of 4", T32K, Q64, Q64, T64, T64, T64, "256x256", "256x256", T128, Q64K, Q64,
                 T64K, T128A, S128 + " of 2"],
}


@pytest.mark.parametrize("name,sizes,call", [("rows K", grouped.ROWS, rows), ("rows MN", grouped.ROWS, lambda *c: rows(*c, "MN")),
                                             ("sums f32", grouped.WGRAD, sums), ("sums 16", grouped.WGRAD, lambda *c: sums(*c, "16")),
                                             ("mx rows", grouped.MX, mx_rows), ("products", mxfp4.PRODUCTS, product)],
                         ids=lambda x: x if isinstance(x, str) else "")
def test_chosen_kernels(name, sizes, call):
    assert list(zip(sizes, shapes([call(*s) for s in sizes]))) == list(zip(sizes, CHOSEN[name]))
    assert len(CHOSEN[name]) == len(sizes)


def test_chosen_kernels_over_the_scales_range():
    calls = [product(*s) for s in mx_range.SIZES] + [mx_rows(M, 1, N, K) for M, N, K in mx_range.SIZES]
    assert [s.split()[0] for s in shapes(calls)] == ["stream", "stream", "tile", "256x256"] * 2
