"""The LDS-poison build (build variant "poison") on the kernels of the MXFP4 and of the grouped products: LDS
holds NaN bits until a stage's own writes reach it, so a read of a slot that they have not filled shows in
integer data's exact results (NaN elements in 16 bits, NaN scales of MXFP4)."""
import pytest

import lds_staged_matrix_amd as lsm
import test_gpu_grouped as T
import test_gpu_mxfp4 as X

pytestmark = pytest.mark.gpu

NAMES = ("gemm_mxfp4_quantize_run", "gemm_mxfp4_dequantize_run", "gemm_mxfp4_run", "gemm_grouped_run",
         "gemm_grouped_wgrad_run", "gemm_grouped_mxfp4_run")


@pytest.fixture(scope="module")
def build():
    lib = lsm.ablation_library("poison")
    h = lib.gemm_create()
    yield lib, h
    lib.gemm_destroy(h)


@pytest.fixture(autouse=True)
def poison(build, monkeypatch):
    """The package's entry points on the poison build; the calls that reached it."""
    lib, h = build
    calls = []

    def on(name):
        def run(handle, *args):
            calls.append(name)
            return getattr(lib, name)(h, *args)
        return run
    for name in NAMES:
        monkeypatch.setattr(lsm, name, on(name))
    yield calls
    assert calls


@pytest.mark.parametrize("T_,groups,N,K", T.ROWS)
@pytest.mark.parametrize("layout", ["K", "MN"])
def test_rows(T_, groups, N, K, layout):
    for how in ("skew", "gaps"):
        T.check_rows(T_, groups, N, K, "bf16", "f32", layout, how, "int")


@pytest.mark.parametrize("K", [8, 64, 136, 264])
@pytest.mark.parametrize("layout", ["K", "MN"])
def test_parts(K, layout):
    T.test_rows_256_tiles_by_k(K, layout)


@pytest.mark.parametrize("T_,groups,M,N", T.WGRAD)
def test_wgrad(T_, groups, M, N):
    for how in ("skew", "gaps"):
        T.check_wgrad(T_, groups, M, N, "f16", "f32", how, "int")


@pytest.mark.parametrize("T_,groups,N,K", T.MX)
def test_grouped_mxfp4(T_, groups, N, K):
    for how in ("skew", "gaps"):
        T.check_mx(T_, groups, N, K, "f32", how, "exact")


@pytest.mark.parametrize("M,N,K", X.PRODUCTS)
def test_mxfp4(M, N, K):
    X.check_product(M, N, K, "f32", "exact")


@pytest.mark.parametrize("layout", ["K", "MN"])
def test_quantize(layout):
    X.test_quantize_sizes(300, 1152, "bf16", layout)
    X.test_quantize_sizes(17, 1056, "f32", layout)
