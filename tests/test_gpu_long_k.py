"""Every kernel of the grouped and of the MXFP4 products but the 256 x 256 one (test_gpu_tile256.py) over enough K tiles
for each of its rings of LDS stages to come round twice, the last K tile cut.  test_kernel_choice.py holds that these
sizes take these kernels.  On the library and on the poison build, against fp64 bit for bit on integers and within the
bounds of the sums on real values."""
import pytest

from test_gpu_tile256 import KINDS
from test_gpu_mxfp4 import DTYPE
from tile_checks import build, check_mx_rows, check_product, check_rows, check_sums, uneven  # noqa: F401

pytestmark = pytest.mark.gpu

# kernel: T, groups, N, K
ROWS_K = {"stream 16x16 of 8": (5, 3, 40, 2136), "stream 16x32 of 4": (20, 6, 1096, 1112), "stream 16x64 of 4": (60, 8, 4104, 1144),
          "stream 32x16 of 8": (70, 3, 72, 2136), "stream 32x32 of 4": (396, 20, 200, 1080), "stream 32x64 of 4": (735, 40, 400, 1176),
          "tile 128x128, 2 stages": (2773, 3, 1832, 344), "tile 128x128, 3 stages": (4600, 40, 280, 536),
          "tile 32x64, 3 stages, K by 2": (200, 3, 72, 920), "tile 64x128, 2 stages": (1197, 20, 1048, 344),
          "tile 64x128, 3 stages, K by 2": (2108, 40, 368, 856), "tile 64x64, 3 stages, K by 2": (4574, 5, 72, 856)}
ROWS_MN = {"stream 16x128 of 4": (50, 20, 776, 1112), "stream 16x64 of 4": (20, 6, 264, 1112), "stream 32x128 of 2": (211, 12, 1384, 632),
           "stream 32x64 of 4": (70, 3, 72, 1080), "tile 128x128, 2 stages": (2907, 1, 1752, 344),
           "tile 128x128, 3 stages": (5925, 2, 264, 536), "tile 32x64, 3 stages, K by 2": (200, 3, 72, 984),
           "tile 64x128, 2 stages": (1197, 20, 1048, 344), "tile 64x128, 3 stages, K by 2": (5692, 5, 144, 856),
           "tile 64x64, 3 stages, K by 2": (5248, 8, 72, 856)}
# kernel: T, groups, M, N, the types of C
SUMS = {"tile 128x128, 2 stages": (2700, 8, 1152, 896, ("f32", "16")), "tile 128x128, 3 stages": (33280, 40, 528, 72, ("f32", "16")),
        "tile 64x128, 3 stages, K by 2": (43520, 40, 16, 432, ("f32", "16")), "tile 64x64, 2 stages": (28160, 40, 440, 16, ("f32", "16")),
        "tile 64x64, 3 stages, K by 2": (2496, 3, 72, 40, ("f32", "16"))}
# kernel: M, N, K
PRODUCTS = {"stream 16x16 of 4": (5, 40, 4864), "stream 16x32 of 4": (2, 8390, 4448), "stream 16x64 of 2": (3, 17255, 2144),
            "stream 16x128 of 2": (4, 33000, 2144), "stream 32x32 of 4": (18, 40, 4320), "stream 32x64 of 2": (18, 18433, 2144),
            "tile 128x128, 2 stages": (7560, 651, 1376), "tile 128x128, 3 stages": (1247, 3154, 1888),
            "tile 32x64, 3 stages, K by 2": (67, 40, 3488), "tile 64x128, 2 stages": (891, 3344, 1120),
            "tile 64x128, 3 stages, K by 2": (1366, 746, 3424), "tile 64x64, 2 stages": (655, 1542, 1376),
            "tile 64x64, 3 stages, K by 2": (71, 40, 7712)}
# kernel: T, groups, N, K
MX_ROWS = {"stream 16x128 of 2": (36, 12, 2730, 2144), "stream 16x16 of 4": (20, 3, 40, 4448), "stream 16x32 of 4": (39, 20, 386, 4448),
           "stream 16x64 of 2": (73, 40, 415, 2144), "stream 32x32 of 4": (70, 3, 40, 4704), "stream 32x64 of 2": (115, 4, 4067, 2144),
           "tile 128x128, 2 stages": (4952, 4, 1192, 1120), "tile 128x128, 3 stages": (3799, 3, 999, 2080),
           "tile 32x64, 3 stages, K by 2": (150, 3, 41, 3488), "tile 64x128, 2 stages": (4731, 2, 589, 1376),
           "tile 64x128, 3 stages, K by 2": (5657, 3, 149, 3424), "tile 64x64, 2 stages": (4871, 3, 193, 1376),
           "tile 64x64, 3 stages, K by 2": (46, 1, 40, 8480)}


@pytest.mark.parametrize("layout,kernel", [(l, k) for l, cases in (("K", ROWS_K), ("MN", ROWS_MN)) for k in cases])
@pytest.mark.parametrize("dist", ["int", "real"])
def test_rows(build, layout, kernel, dist):
    T, groups, N, K = (ROWS_K if layout == "K" else ROWS_MN)[kernel]
    check_rows(build, uneven(T, groups), N, K, layout, *KINDS[(len(kernel) + T) % 4], dist, pad=T % 3 * 4)


def sums_kinds(kernel):
    """(input, output) types of a case of SUMS."""
    return [(k, o) for k, o in KINDS if ("f32" if o == "f32" else "16") in SUMS[kernel][4]]


@pytest.mark.parametrize("kernel,kind,out", [(k, *t) for k in SUMS for t in sums_kinds(k)])
@pytest.mark.parametrize("dist", ["int", "real"])
def test_sums(build, kernel, kind, out, dist):
    T, groups, M, N, _ = SUMS[kernel]
    check_sums(build, uneven(T, groups), M, N, kind, out, dist, pad=8 if kind == "bf16" else 3)


@pytest.mark.parametrize("kernel", list(PRODUCTS))
@pytest.mark.parametrize("dist", ["int", "real"])
def test_product(build, kernel, dist):
    M, N, K = PRODUCTS[kernel]
    check_product(build, M, N, K, sorted(DTYPE)[M % 3], dist, pad=M % 2 * 3)


@pytest.mark.parametrize("kernel", list(MX_ROWS))
@pytest.mark.parametrize("dist", ["int", "real"])
def test_mx_rows(build, kernel, dist):
    T, groups, N, K = MX_ROWS[kernel]
    check_mx_rows(build, uneven(T, groups), N, K, sorted(DTYPE)[T % 3], dist, pad=T % 2 * 3)
