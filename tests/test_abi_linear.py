"""Argument checks of gemm_rmsnorm_run, gemm_scaled_run and gemm_w4_run, on the
CPU: every request below is answered before anything is launched.  Pointers are
made-up addresses; a request that passes every check stops at the device check
(GEMM_ERR_DEVICE), because the stand-in handle's device does not exist.
"""
import ctypes
import os
import subprocess

import pytest

import lds_staged_matrix_amd as lsm
import test_isa_hazards as isa

_FAKE_DEVICE = ctypes.c_int(1 << 20)
FAKE = ctypes.cast(ctypes.pointer(_FAKE_DEVICE), ctypes.c_void_p)
VALID, INVALID, UNSUPPORTED, OK = (lsm.GEMM_ERR_DEVICE, lsm.GEMM_ERR_INVALID_ARG, lsm.GEMM_ERR_UNSUPPORTED,
                                   lsm.GEMM_OK)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(lsm.library_path()):
        from lds_staged_matrix_amd import build
        build.build()
    return lsm.load_library()


def addr(i):
    return (i + 1) << 24


def call(fn, base, changes):
    a = dict(base)
    a.update(changes)
    handle = a.pop("h", FAKE)
    return fn(handle, **a)


NORM = dict(X=addr(0), R=addr(1), W=addr(2), H=addr(3), Y=addr(4), S=addr(5), M=16, N=64, ldx=64, ldr=64, ldh=64,
            ldy=64, eps=1e-5, dtype=lsm.GEMM_NORM_BF16_E4M3)
T16 = dict(dtype=lsm.GEMM_NORM_BF16_BF16)
NORM_CASES = [
    ({}, VALID), (dict(h=None), INVALID), (dict(dtype=4), INVALID), (dict(dtype=-1), INVALID),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(M=0), OK), (dict(N=0), OK),
    (dict(M=0, X=0, Y=0, W=0), OK),
    (dict(eps=-1e-9), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=0.0), VALID),
    (dict(X=0), INVALID), (dict(W=0), INVALID), (dict(Y=0), INVALID), (dict(S=0), INVALID),
    (dict(S=0, **T16), VALID), (dict(R=0, ldr=0), VALID), (dict(H=0, ldh=0), VALID),
    (dict(ldx=63), INVALID), (dict(ldr=63), INVALID), (dict(ldh=63), INVALID), (dict(ldy=63), INVALID),
    (dict(M=1 << 30), UNSUPPORTED), (dict(N=1 << 30, ldx=1 << 31, ldr=1 << 31, ldh=1 << 31, ldy=1 << 31), UNSUPPORTED),
    (dict(ldx=1 << 40), UNSUPPORTED), (dict(ldr=1 << 40), UNSUPPORTED), (dict(ldh=1 << 40), UNSUPPORTED),
    (dict(ldy=1 << 40), UNSUPPORTED),
    (dict(M=(1 << 30) - 1, ldx=(1 << 40) - 1), UNSUPPORTED),       # X spans 2^63 bytes or more
    (dict(X=addr(0) + 1), UNSUPPORTED), (dict(R=addr(1) + 1), UNSUPPORTED), (dict(W=addr(2) + 1), UNSUPPORTED),
    (dict(H=addr(3) + 1), UNSUPPORTED), (dict(S=addr(5) + 2), UNSUPPORTED), (dict(Y=addr(4) + 1), VALID),
    (dict(Y=addr(4) + 1, **T16), UNSUPPORTED), (dict(X=addr(0) + 2), VALID),
    # an output in an input's place
    (dict(H=addr(0)), VALID), (dict(H=addr(1)), VALID), (dict(Y=addr(0), **T16), VALID),
    (dict(Y=addr(1), H=addr(0), **T16), VALID),
    (dict(Y=addr(0)), INVALID),                                    # E4M3 over 16-bit
    (dict(H=addr(0), ldh=72), INVALID), (dict(H=addr(0), ldh=72, M=1), VALID),
    (dict(H=addr(0) + 2), INVALID), (dict(Y=addr(3), **T16), INVALID), (dict(H=addr(2)), INVALID),
    (dict(Y=addr(2) + 126, **T16), INVALID), (dict(Y=addr(2) + 128, **T16), VALID),
    (dict(S=addr(0)), INVALID), (dict(S=addr(4) + 1024), VALID), (dict(S=addr(4) + 1020), INVALID),
    (dict(S=addr(0), **T16), VALID),                               # S is not used
    (dict(R=addr(0)), VALID),                                      # inputs may be the same
]

SCALED = dict(A=addr(0), B=addr(1), C=addr(2), SA=addr(3), SB=addr(4), M=16, N=32, K=64, lda=64, ldb=64, ldc=32,
              incA=1, incB=1, layoutA=0, layoutB=0, dtype=lsm.GEMM_E4M3_F32)
SCALED_CASES = [
    ({}, VALID), (dict(h=None), INVALID), (dict(dtype=lsm.GEMM_E4M3_F16), VALID),
    (dict(dtype=lsm.GEMM_E4M3_BF16), VALID), (dict(dtype=lsm.GEMM_BF16_F32), INVALID), (dict(dtype=7), INVALID),
    (dict(M=-1), INVALID), (dict(K=-1), INVALID), (dict(M=0), OK), (dict(N=0), OK), (dict(K=0, A=0, B=0), VALID),
    (dict(SA=0), INVALID), (dict(SB=0), INVALID), (dict(SA=addr(3) + 2), UNSUPPORTED),
    (dict(SB=addr(4) + 1), UNSUPPORTED), (dict(incA=2), INVALID), (dict(incB=-1), INVALID),
    (dict(incA=0, incB=0), VALID), (dict(layoutA=2), INVALID), (dict(layoutB=-1), INVALID),
    (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID),
    (dict(lda=48), INVALID), (dict(ldb=48), INVALID), (dict(ldc=31), INVALID),
    (dict(K=56), UNSUPPORTED), (dict(lda=72), UNSUPPORTED), (dict(A=addr(0) + 8), UNSUPPORTED),
    (dict(layoutA=1, M=24, lda=32), UNSUPPORTED), (dict(N=33, ldc=33), VALID),
    (dict(C=addr(2) + 2), UNSUPPORTED), (dict(C=addr(2) + 2, dtype=lsm.GEMM_E4M3_BF16), VALID),
    (dict(C=addr(0) + 512), INVALID), (dict(C=addr(3) + 60), INVALID), (dict(C=addr(3) + 64), VALID),
    (dict(C=addr(3) + 4, incA=0), VALID), (dict(C=addr(4)), INVALID),
    (dict(A=1 << 40, M=1 << 16, lda=1 << 16), UNSUPPORTED),                   # A beyond 32-bit offsets
    (dict(M=1 << 29, ldc=(1 << 39) + 16), UNSUPPORTED),
]

W4 = dict(A=addr(0), B=addr(1), S=addr(2), Z=addr(3), C=addr(4), M=4, N=48, K=96, group=32, lda=96, ldb=96, lds=48,
          ldz=48, ldc=48, dtype=lsm.GEMM_BF16_F32)
W4_CASES = [
    ({}, VALID), (dict(h=None), INVALID), (dict(dtype=lsm.GEMM_E4M3_F32), INVALID), (dict(dtype=-1), INVALID),
    (dict(dtype=lsm.GEMM_F16_F16), VALID), (dict(Z=0, ldz=0), VALID),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-32), INVALID), (dict(M=0), OK), (dict(N=0), OK),
    (dict(K=0, A=0, B=0, S=0, Z=0, lda=0, ldb=0, lds=0, ldz=0), VALID),
    (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(S=0), INVALID), (dict(C=0), INVALID),
    (dict(group=0), INVALID), (dict(group=-32), INVALID), (dict(group=16), UNSUPPORTED), (dict(group=96), UNSUPPORTED),
    (dict(group=1 << 30), VALID), (dict(group=1 << 31), UNSUPPORTED), (dict(K=80), UNSUPPORTED),
    (dict(lda=88), INVALID), (dict(ldb=64), INVALID), (dict(lds=47), INVALID), (dict(ldz=47), INVALID),
    (dict(ldc=47), INVALID), (dict(lda=100), UNSUPPORTED), (dict(ldb=112), UNSUPPORTED), (dict(ldb=128), VALID),
    (dict(A=addr(0) + 8), UNSUPPORTED), (dict(B=addr(1) + 8), UNSUPPORTED), (dict(S=addr(2) + 1), UNSUPPORTED),
    (dict(S=addr(2) + 2), VALID), (dict(Z=addr(3) + 1), VALID), (dict(C=addr(4) + 2), UNSUPPORTED),
    (dict(C=addr(4) + 2, dtype=lsm.GEMM_BF16_BF16), VALID),
    (dict(M=1 << 30), UNSUPPORTED), (dict(lda=1 << 40), UNSUPPORTED), (dict(ldb=1 << 40), UNSUPPORTED),
    (dict(lda=1 << 24), UNSUPPORTED), (dict(lda=(1 << 24) - 8, A=1 << 40), VALID), (dict(ldb=1 << 25), UNSUPPORTED),
    (dict(ldb=(1 << 25) - 32, B=1 << 40), VALID),
    (dict(lds=1 << 40), UNSUPPORTED), (dict(ldz=1 << 40), UNSUPPORTED), (dict(ldc=1 << 40), UNSUPPORTED),
    (dict(M=(1 << 30) - 1, N=(1 << 30) - 1, lds=1 << 30, ldz=1 << 30, ldc=1 << 30), UNSUPPORTED),
    (dict(M=1 << 29, ldc=(1 << 39)), UNSUPPORTED),
    # 2^32 threads: tiles of 32 x 64 by eight waves from K = 1024 on, by one wave below 256
    (dict(A=1 << 40, B=1 << 44, S=1 << 48, Z=1 << 49, C=1 << 50, M=1 << 17, N=1 << 17, K=1024, lda=1024, ldb=1024,
          lds=1 << 17, ldz=1 << 17, ldc=1 << 17), UNSUPPORTED),
    (dict(A=1 << 40, B=1 << 44, S=1 << 48, Z=1 << 49, C=1 << 50, M=1 << 17, N=1 << 16, K=1024, lda=1024, ldb=1024,
          lds=1 << 17, ldz=1 << 17, ldc=1 << 17), VALID),
    (dict(A=1 << 40, B=1 << 44, S=1 << 48, Z=1 << 49, C=1 << 50, M=1 << 17, N=1 << 17, lds=1 << 17, ldz=1 << 17,
          ldc=1 << 17), VALID),
    (dict(C=addr(0) + 760), INVALID), (dict(C=addr(0) + 768), VALID),
    (dict(C=addr(1) + 48 * 47 + 44), INVALID), (dict(C=addr(1) + 48 * 48), VALID),
    (dict(C=addr(2) + 284), INVALID), (dict(C=addr(3) + 140), INVALID), (dict(C=addr(3) + 144), VALID),
]


def ids(cases):
    return [",".join(f"{k}={v}" for k, v in c.items())[:60] or "base" for c, _ in cases]


@pytest.mark.parametrize("changes,status", NORM_CASES, ids=ids(NORM_CASES))
def test_rmsnorm_checks(changes, status):
    assert call(lsm.gemm_rmsnorm_run, NORM, changes) == status


@pytest.mark.parametrize("changes,status", SCALED_CASES, ids=ids(SCALED_CASES))
def test_scaled_checks(changes, status):
    assert call(lsm.gemm_scaled_run, SCALED, changes) == status


@pytest.mark.parametrize("changes,status", W4_CASES, ids=ids(W4_CASES))
def test_w4_checks(changes, status):
    assert call(lsm.gemm_w4_run, W4, changes) == status


@pytest.mark.parametrize("fn,base,name,value", [
    (lsm.gemm_rmsnorm_run, NORM, "M", 1 << 64), (lsm.gemm_rmsnorm_run, NORM, "dtype", 1 << 32),
    (lsm.gemm_scaled_run, SCALED, "ldb", 1 << 63), (lsm.gemm_scaled_run, SCALED, "incA", (1 << 32) + 1),
    (lsm.gemm_w4_run, W4, "group", 1 << 64), (lsm.gemm_w4_run, W4, "dtype", -(1 << 31) - 1)])
def test_integers_that_the_abi_cannot_hold(fn, base, name, value):
    with pytest.raises(OverflowError):
        call(fn, base, {name: value})


class Pointer:
    def __init__(self, value):
        self.value = value

    def data_ptr(self):
        if isinstance(self.value, Exception):
            raise self.value
        return self.value


def test_what_the_binding_takes():
    """numpy and float sizes, pointer objects, stream objects, integer handles; errors pass through."""
    np = pytest.importorskip("numpy")
    run = lsm.gemm_w4_run
    assert call(run, W4, dict(M=np.int64(4), N=np.int32(48), K=96.0)) == VALID
    assert call(run, W4, {k: Pointer(v) for k, v in W4.items() if k in "ABSZC"}) == VALID
    assert call(run, W4, dict(A=Pointer(addr(0) + 8))) == UNSUPPORTED
    assert call(run, W4, dict(A=Pointer(0))) == INVALID
    assert call(run, W4, dict(h=ctypes.addressof(_FAKE_DEVICE))) == VALID
    assert call(run, W4, dict(stream=type("Stream", (), {"cuda_stream": 0})())) == VALID
    assert call(run, W4, dict(stream=0)) == VALID
    with pytest.raises(ValueError, match="gone"):
        call(run, W4, dict(A=Pointer(ValueError("gone"))))
    with pytest.raises((TypeError, ValueError)):
        call(run, W4, dict(M="many"))
    with pytest.raises(TypeError):
        call(lsm.gemm_rmsnorm_run, NORM, dict(eps="small"))
    from lds_staged_matrix_amd import _binding
    with pytest.raises(TypeError, match="gemm_run takes 14 arguments, got 1"):
        _binding.run(None)


def test_the_plain_product_refuses_the_scaled_product_s_type():
    assert lsm.gemm_run(FAKE, addr(0), addr(1), addr(2), 16, 16, 16, 16, 16, 16, 0, 0,
                        lsm.GEMM_E4M3_F16) == INVALID


@isa.needs_tools
def test_lds_dma_wait_states_of_the_scaled_product(tmp_path):
    """The wait-state rules of test_isa_hazards.py on the scaled product's own
    code object, which stands behind gemm_run's in the library."""
    obj = os.path.join(isa.PKG, "_build", "gemm_scaled.o")
    if not os.path.exists(obj):
        pytest.skip("library objects not built")
    ins = isa._disassemble(obj, tmp_path)
    loads = [i for i, t in enumerate(ins) if t and t.startswith("buffer_load") and t.endswith(" lds")]
    assert loads
    for i in loads:
        read = set().union(*(isa._sgprs(o) for o in ins[i].split(None, 1)[1].split(",")[1:]))
        waits = 0
        for prev in reversed(ins[max(0, i - 7):i]):
            if prev is None:
                break
            assert waits >= 1 or not prev.startswith("s_mov_b32 m0"), prev
            assert waits >= 5 or not (isa._scalar_dest(prev) & read), prev
            waits += isa._wait_states(prev)
