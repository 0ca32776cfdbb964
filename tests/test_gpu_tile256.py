"""The 256 x 256 kernel of the grouped and of the MXFP4 products (gemm_kernel_tile256.h) in each of its forms: tiles of
256, 128 and 64 rows, whole, halved and quartered, of one K tile to 18, the last one cut or not; gradients of groups
without rows and with many, in one round of tiles and in more, the groups in order and by size.  test_kernel_choice.py
holds that these sizes take this kernel and which forms they reach (test_gpu_grouped.py's test_rows_256_tiles_by_k is
served by 64 x 128 and 128 x 128 tiles).  Each case on the library and on the poison
build, against fp64: bit for bit on integers, and within the bounds of the sums on real values."""
import pytest
import torch

import grouped_reference as G
import lds_staged_matrix_amd as lsm
from test_gpu_grouped import TYPE
from test_gpu_mxfp4 import DTYPE, LAYOUT
from tile_checks import (Data, Mx, build, check_mx_rows, check_product, check_rows, check_sums, compare, ends_of,  # noqa: F401
                         matmul, ok)

pytestmark = pytest.mark.gpu

KINDS = sorted(TYPE)

ROWS_K = [8, 64, 128, 200, 328, 520, 1096]                   # 1, 1, 2, 4, 6, 9 and 18 K tiles
MX_K = [32, 256, 480, 800, 1312, 2048, 4320]                 # 1, 1, 2, 4, 6, 8 and 17
# Rows of the groups, columns, and the K of ROWS_K that take this kernel: whole tiles, tiles of which the last round is
# cut into quarters, and into halves.
GROUPS = {"whole": ([700, 260, 33, 500], 8192, ROWS_K), "quarters": ([700, 300, 100, 770], 8184, ROWS_K[2:]),
          "halves": ([700, 300, 100, 0, 1201], 8192, ROWS_K[1:])}
# M, N, and the K of MX_K that take this kernel
PRODUCTS = {"whole": (2100, 6199, MX_K), "quarters": (2100, 8192, MX_K), "halves": (1172, 5380, MX_K[3:])}
# Rows of the groups, M, N, and the types of C that take this kernel
SUMS = {"halves, one group": ([2000], 4096, 1920, ("f32", "16")),
        "halves, two groups": ([1, 2899], 2048, 2048, ("f32", "16")),
        "tiles of 56 rows, short groups": ([0, 1, 64, 65, 130, 8, 100, 52], 1848, 1008, ("f32",)),
        "more than a round": ([300, 64, 1600], 2056, 4104, ("f32", "16")),
        "more than a round, halves": ([900, 2500, 64, 4000], 1800, 2560, ("f32", "16"))}


# --------------------------------------------------------------------- rows

@pytest.mark.parametrize("name,K", [(n, K) for n in GROUPS for K in GROUPS[n][2]])
@pytest.mark.parametrize("layout", ["K", "MN"])
def test_rows(build, name, K, layout):
    i = ROWS_K.index(K) + list(GROUPS).index(name) + (layout == "MN")
    check_rows(build, *GROUPS[name][:2], K, layout, *KINDS[i % 4], "int", pad=i % 3 * 4)       # rows of C aligned and not


@pytest.mark.parametrize("layout", ["K", "MN"])
@pytest.mark.parametrize("kind,out", KINDS)
def test_rows_real(build, layout, kind, out):
    check_rows(build, *GROUPS["quarters"][:2], 520, layout, kind, out, "real")


@pytest.mark.parametrize("layout", ["K", "MN"])
def test_rows_empty_sum(build, layout):
    lib, h = build
    rows, N, _ = GROUPS["whole"]
    ends = ends_of(rows)
    C = torch.full((ends[-1] + 2, N), 5.0, device="cuda")
    ok(lib.gemm_grouped_run(h, None, None, C, torch.tensor(ends, dtype=torch.int32, device="cuda"), len(rows), ends[-1] + 2, N,
                            0, 0, 0, 0, N, LAYOUT[layout], lsm.GEMM_BF16_F32, torch.cuda.current_stream()), "gemm_grouped_run")
    assert bool((C[:ends[-1]] == 0).all()) and bool((C[ends[-1]:] == 5).all())


# -------------------------------------------------------------------- MXFP4

@pytest.mark.parametrize("name,K", [(n, K) for n in PRODUCTS for K in PRODUCTS[n][2]])
def test_product(build, name, K):
    i = MX_K.index(K) + list(PRODUCTS).index(name)
    check_product(build, *PRODUCTS[name][:2], K, sorted(DTYPE)[i % 3], "int", pad=i % 2 * 3)


@pytest.mark.parametrize("name", list(PRODUCTS))
@pytest.mark.parametrize("out", sorted(DTYPE))
def test_product_real(build, name, out):
    check_product(build, *PRODUCTS[name][:2], 1312, out, "real")


@pytest.mark.parametrize("K", [0, 64])
def test_product_of_many_tiles(build, K):
    """Eight rounds of tiles whose K loop is empty, or one K tile long."""
    lib, h = build
    M, N = 16384, 8192
    C = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
    print("CASE tile256 many tiles", K, flush=True)
    if K == 0:
        ok(lib.gemm_mxfp4_run(h, None, None, C, None, None, M, N, 0, 0, 0, N, 0, 0, lsm.GEMM_MXFP4_BF16,
                              torch.cuda.current_stream()), "gemm_mxfp4_run")
        assert bool((C == 0).all())
        return
    d = Data("many", K)
    a, b = Mx(d, M, K, "int"), Mx(d, N, K, "int")
    ok(lib.gemm_mxfp4_run(h, a.Q, b.Q, C, a.S, b.S, M, N, K, a.ldq, b.ldq, N, a.lds, b.lds, lsm.GEMM_MXFP4_BF16,
                          torch.cuda.current_stream()), "gemm_mxfp4_run")
    compare(C, a.v @ b.v.t(), None, "bf16", "many tiles")


@pytest.mark.parametrize("K", MX_K)
@pytest.mark.parametrize("name", list(GROUPS))
def test_mx_rows(build, name, K):
    i = MX_K.index(K) + list(GROUPS).index(name)
    check_mx_rows(build, *GROUPS[name][:2], K, sorted(DTYPE)[i % 3], "int", pad=i % 2 * 3)


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("out", sorted(DTYPE))
def test_mx_rows_real(build, name, out):
    check_mx_rows(build, *GROUPS[name][:2], 1312, out, "real")


# --------------------------------------------------------------------- sums

def sums_kinds(name):
    """(input, output) types of a case of SUMS."""
    return [(k, o) for k, o in KINDS if ("f32" if o == "f32" else "16") in SUMS[name][3]]


@pytest.mark.parametrize("name,kind,out", [(n, *k) for n in SUMS for k in sums_kinds(n)])
@pytest.mark.parametrize("dist", ["int", "real"])
def test_sums(build, name, kind, out, dist):
    check_sums(build, *SUMS[name][:3], kind, out, dist, pad=8 if kind == "bf16" else 3)


def test_sums_replay(build):
    """A captured gradient in halves, by size, follows the ends."""
    lib, h = build
    rows, M, N, _ = SUMS["more than a round, halves"]
    d, T = Data("replay"), sum(rows)
    a, b = d.values("int", T, M).bfloat16(), d.values("int", T, N).bfloat16()
    C = torch.zeros(len(rows), M, N, device="cuda")
    ends = torch.tensor(ends_of(rows), dtype=torch.int32, device="cuda")

    def call():
        status = lib.gemm_grouped_wgrad_run(h, a, b, C, ends, len(rows), T, M, N, M, N, N, M * N, lsm.GEMM_BF16_F32,
                                            torch.cuda.current_stream())
        assert status == lsm.GEMM_OK
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for r in (rows, rows[::-1], [T, 0, 0, 0], [0, 0, 0, 0], [5, 400, 2800, 60]):
        ends.copy_(torch.tensor(ends_of(r), dtype=torch.int32))
        C.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for g, (f, l) in enumerate(G.bounds(ends_of(r), T)):
            compare(C[g], matmul(a[f:l].t(), b[f:l]), None, "f32", f"group {g} of {r}")
