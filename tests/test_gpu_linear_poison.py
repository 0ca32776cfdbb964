"""The LDS-poison build (build variant "poison") on the few-rows, 4-bit and split-K
kernels and on the scaled forms of the others: LDS holds NaN bits until a
stage's, a slice's or a sum's own writes reach it, so a read of a slot that they
have not filled shows in integer data's exact results.
"""
import pytest
import torch

import lds_staged_matrix_amd as lsm
import test_gpu_linear as T

pytestmark = pytest.mark.gpu

KC, MNC = T.KC, T.MNC


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
    for name in ("gemm_scaled_run", "gemm_w4_run", "gemm_rmsnorm_run"):
        monkeypatch.setattr(lsm, name, on(name))
    yield calls
    assert calls


# 8 and 16 rows, 32, 48 and 64; one and two blocks of columns; one block of k, a cut one, several a wave
@pytest.mark.parametrize("M", [1, 8, 13, 16, 29, 45, 64])
@pytest.mark.parametrize("N,K", [(40, 16), (200, 128), (200, 272), (4111, 144), (8300, 272), (250, 4240)])
@pytest.mark.parametrize("out", sorted(T.SCALED))
def test_few_rows(M, N, K, out):
    T.check_scaled(M, N, K, KC, KC, out, "int")


@pytest.mark.parametrize("M,N,K", [(64, 200, 272), (48, 4400, 400), (250, 2000, 1552)])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_few_rows_exact(monkeypatch, M, N, K, out):
    monkeypatch.setattr(T, "SCALED", {k: v + lsm.GEMM_EXACT_SUMS for k, v in T.SCALED.items()})
    T.check_scaled(M, N, K, KC, KC, out, "int")


# split K of two groups with four stages (four with two), and two with two: steps that divide over the groups and not,
# K cut inside a tile; the ring, ping-pong, 128 x 128 and both 64 x 64 kernels with scales
@pytest.mark.parametrize("M,N,K", [(208, 1040, 1024), (208, 1040, 1168), (208, 1040, 1296), (1040, 1088, 4096), (1040, 1088, 4240),
                                   (32, 1024, 1040), (4112, 4096, 144), (2064, 2048, 144), (528, 1088, 160),
                                   (1040, 2560, 3984)])
@pytest.mark.parametrize("la,lb", T.LAYOUTS)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_tiles(M, N, K, la, lb, out):
    T.check_scaled(M, N, K, la, lb, out, "int")


@pytest.mark.parametrize("kind,out", [("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 40, 32), (4, 4100, 160), (13, 40, 96), (16, 4100, 1184), (20, 40, 1184), (20, 4100, 288),
                                   (30, 8200, 160), (48, 40, 1120), (48, 4100, 96), (48, 8200, 1184)])
def test_w4(kind, out, group, M, N, K):
    T.check_w4(M, N, K, group, kind, out, M % 2 == 0, "int")


@pytest.mark.parametrize("N", [8, 300, 520, 8192, 20000, 33001])
def test_norm(N):
    T.check_norm(5, N, "bf16", "e4m3", T.run_norm(5, N, "bf16", "e4m3", True, True))


def test_layer():
    layer = T.Layer(24, 1024, 1152, 3)
    layer.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    layer.check()
