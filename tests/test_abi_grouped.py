"""Argument checks of the MXFP4 and the grouped entry points, on the CPU: every request below is answered
before anything is launched (see test_abi_linear.py: made-up addresses, a handle whose device does not
exist, so that a request that passes every check stops at GEMM_ERR_DEVICE)."""
import ctypes
import os

import pytest

import lds_staged_matrix_amd as lsm
import test_isa_hazards as isa
from test_abi_binding import Numbered, Valued
from test_abi_linear import FAKE, INVALID, OK, UNSUPPORTED, VALID, Pointer, addr, call, ids, lib  # noqa: F401

QUANTIZE = dict(X=addr(0), Q=addr(1), S=addr(2), M=20, K=64, ldx=64, ldq=64, lds=32, layoutX=0, dtype=0)
MN = dict(layoutX=1, ldx=20)
QUANTIZE_CASES = [
    ({}, VALID), (dict(h=None), INVALID), (dict(dtype=1), VALID), (dict(dtype=2), VALID), (dict(dtype=3), INVALID),
    (dict(dtype=-1), INVALID), (dict(layoutX=2), INVALID), (dict(layoutX=-1), INVALID), (MN, VALID),
    (dict(M=-1), INVALID), (dict(K=-32), INVALID), (dict(M=0), OK), (dict(K=0), OK), (dict(M=0, X=0, Q=0, S=0), OK),
    (dict(X=0), INVALID), (dict(Q=0), INVALID), (dict(S=0), INVALID),
    (dict(ldx=63), INVALID), (dict(layoutX=1, ldx=19), INVALID), (dict(ldx=67), VALID), (dict(layoutX=1, ldx=21), VALID),
    (dict(ldq=32), INVALID), (dict(ldq=80), UNSUPPORTED), (dict(ldq=96), VALID), (dict(lds=16), INVALID),
    (dict(lds=24), UNSUPPORTED), (dict(K=48), UNSUPPORTED), (dict(K=33, ldx=64), UNSUPPORTED),
    (dict(X=addr(0) + 1), UNSUPPORTED), (dict(X=addr(0) + 2), VALID), (dict(X=addr(0) + 2, dtype=2), UNSUPPORTED),
    (dict(Q=addr(1) + 8), UNSUPPORTED), (dict(S=addr(2) + 8), UNSUPPORTED),
    (dict(M=1 << 30, lds=1 << 31), UNSUPPORTED), (dict(ldx=1 << 40), UNSUPPORTED), (dict(ldq=1 << 40), UNSUPPORTED),
    (dict(lds=1 << 40), UNSUPPORTED),
    # 2^32 threads: tiles of 16 rows by 512 k
    (dict(X=1 << 40, Q=1 << 50, S=1 << 52, M=1 << 28, lds=1 << 28), UNSUPPORTED),
    (dict(X=1 << 40, Q=1 << 50, S=1 << 52, M=(1 << 28) - 16, lds=1 << 28), VALID),
    (dict(X=1 << 40, Q=1 << 50, S=1 << 52, M=1 << 28, lds=1 << 28, layoutX=1, ldx=1 << 28), VALID),
    (dict(Q=addr(0) + 2432), INVALID), (dict(Q=addr(0) + 2560), VALID), (dict(S=addr(0) + 2544), INVALID),
    (dict(S=addr(1) + 624), INVALID), (dict(S=addr(1) + 640), VALID),
]
DEQUANTIZE = dict(Q=addr(0), S=addr(1), Y=addr(2), M=20, K=64, ldq=64, lds=32, ldy=64, dtype=0)
DEQUANTIZE_CASES = [
    ({}, VALID), (dict(h=None), INVALID), (dict(dtype=2), VALID), (dict(dtype=3), INVALID), (dict(M=-1), INVALID),
    (dict(K=-1), INVALID), (dict(M=0), OK), (dict(K=0), OK), (dict(Q=0), INVALID), (dict(S=0), INVALID),
    (dict(Y=0), INVALID), (dict(ldy=63), INVALID), (dict(ldy=65), VALID), (dict(ldq=80), UNSUPPORTED),
    (dict(lds=20), UNSUPPORTED), (dict(K=40), UNSUPPORTED), (dict(Y=addr(2) + 1), UNSUPPORTED),
    (dict(Y=addr(2) + 2, dtype=2), UNSUPPORTED), (dict(Y=addr(0) + 512), INVALID), (dict(Y=addr(1)), INVALID),
    (dict(Q=addr(1)), VALID),                                     # inputs may overlap
    (dict(ldy=1 << 40), UNSUPPORTED),
]
PRODUCT = dict(A=addr(0), B=addr(1), C=addr(2), SA=addr(3), SB=addr(4), M=20, N=40, K=64, lda=64, ldb=64, ldc=40,
               ldsa=32, ldsb=48, dtype=2)
BIG = dict(A=1 << 40, B=1 << 44, C=1 << 50, SA=1 << 52, SB=1 << 53)
PRODUCT_CASES = [
    ({}, VALID), (dict(h=None), INVALID), (dict(dtype=0), VALID), (dict(dtype=1), VALID), (dict(dtype=3), INVALID),
    (dict(dtype=-1), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-32), INVALID), (dict(M=0), OK),
    (dict(N=0), OK), (dict(K=0, A=0, B=0, SA=0, SB=0, lda=0, ldb=0, ldsa=0, ldsb=0), VALID),
    (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID), (dict(SA=0), INVALID), (dict(SB=0), INVALID),
    (dict(lda=32), INVALID), (dict(ldb=32), INVALID), (dict(ldc=39), INVALID), (dict(ldsa=16), INVALID),
    (dict(ldsb=32), INVALID), (dict(lda=80), UNSUPPORTED), (dict(ldb=80), UNSUPPORTED), (dict(lda=96), VALID),
    (dict(ldsa=24), UNSUPPORTED), (dict(ldsb=56), UNSUPPORTED), (dict(K=48), UNSUPPORTED),
    (dict(A=addr(0) + 8), UNSUPPORTED), (dict(B=addr(1) + 8), UNSUPPORTED), (dict(SA=addr(3) + 4), UNSUPPORTED),
    (dict(SB=addr(4) + 8), UNSUPPORTED), (dict(C=addr(2) + 2), UNSUPPORTED), (dict(C=addr(2) + 2, dtype=0), VALID),
    (dict(lda=1 << 23), UNSUPPORTED), (dict(BIG, lda=(1 << 23) - 32), VALID), (dict(ldb=1 << 23), UNSUPPORTED),
    (dict(ldsa=1 << 27), UNSUPPORTED), (dict(BIG, ldsa=(1 << 27) - 16), VALID), (dict(ldc=1 << 40), UNSUPPORTED),
    (dict(M=1 << 30, ldsa=1 << 30), UNSUPPORTED),
    # 2^32 threads, 512 to a tile of 256 x 256
    (dict(BIG, M=1 << 26, N=1 << 13, ldc=1 << 13, ldsa=1 << 26, ldsb=1 << 13), UNSUPPORTED),
    (dict(BIG, M=(1 << 26) - 256, N=1 << 13, ldc=1 << 13, ldsa=1 << 26, ldsb=1 << 13), VALID),
    (dict(C=addr(0) + 636), INVALID), (dict(C=addr(0) + 640), VALID), (dict(C=addr(1) + 1276), INVALID),
    (dict(C=addr(3) + 60), INVALID),                              # 32 + 20 scales, up to a multiple of 16: 64
    (dict(C=addr(3) + 64), VALID), (dict(C=addr(4) + 92), INVALID), (dict(C=addr(4) + 96), VALID),
    (dict(A=addr(1), SA=addr(4)), VALID),                         # inputs may be the same
]
ROWS = dict(A=addr(0), B=addr(1), C=addr(2), ends=addr(3), G=3, T=20, N=40, K=64, lda=64, ldb=64, strideb=2560, ldc=40,
            layoutB=0, dtype=lsm.GEMM_BF16_F32)
BMN = dict(layoutB=1, ldb=40)
ROWS_CASES = [
    ({}, VALID), (dict(h=None), INVALID), (BMN, VALID), (dict(dtype=1), VALID), (dict(dtype=3), VALID),
    (dict(dtype=4), INVALID), (dict(dtype=-1), INVALID), (dict(layoutB=2), INVALID), (dict(G=-1), INVALID),
    (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(G=0), OK), (dict(T=0), OK),
    (dict(N=0), OK), (dict(K=0, A=0, B=0, lda=0, ldb=0, strideb=0), VALID),
    (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID), (dict(ends=0), INVALID),
    (dict(lda=56), INVALID), (dict(ldb=56), INVALID), (dict(layoutB=1, ldb=32), INVALID), (dict(ldc=39), INVALID),
    (dict(strideb=-8), INVALID), (dict(strideb=0), VALID), (dict(strideb=4), UNSUPPORTED), (dict(strideb=8), VALID),
    (dict(K=60), UNSUPPORTED), (dict(N=41, ldc=41), VALID), (dict(layoutB=1, N=41, ldb=48, ldc=41), UNSUPPORTED),
    (dict(lda=68), UNSUPPORTED), (dict(ldb=68), UNSUPPORTED), (dict(A=addr(0) + 8), UNSUPPORTED),
    (dict(B=addr(1) + 8), UNSUPPORTED), (dict(C=addr(2) + 2), UNSUPPORTED), (dict(C=addr(2) + 2, dtype=1), VALID),
    (dict(ends=addr(3) + 2), UNSUPPORTED), (dict(lda=1 << 21), UNSUPPORTED), (dict(lda=(1 << 21) - 8, A=1 << 40), VALID),
    (dict(ldb=1 << 21), UNSUPPORTED), (dict(strideb=1 << 40), UNSUPPORTED), (dict(ldc=1 << 40), UNSUPPORTED),
    (dict(T=1 << 30), UNSUPPORTED), (dict(G=1 << 30), UNSUPPORTED), (dict(K=1 << 30, lda=1 << 31, ldb=1 << 31), UNSUPPORTED),
    (dict(BIG_ROWS := dict(A=1 << 44, B=1 << 47, C=1 << 50, ends=1 << 52), T=1 << 28, N=8192, ldc=8192, strideb=0), UNSUPPORTED),
    (dict(BIG_ROWS, T=1 << 26, N=4096, ldc=4096, strideb=0), VALID),
    (dict(G=1 << 16, ends=1 << 52, strideb=0), VALID), (dict(G=(1 << 16) + 1, ends=1 << 52, strideb=0), UNSUPPORTED),
    (dict(C=addr(0) + 2556), INVALID), (dict(C=addr(0) + 2560), VALID), (dict(C=addr(1) + 15356), INVALID),
    (dict(C=addr(1) + 15360), VALID), (dict(C=addr(3) + 8), INVALID), (dict(C=addr(3) + 12), VALID),
    (dict(C=addr(0), K=0, A=0, B=0), VALID),
]
WGRAD = dict(A=addr(0), B=addr(1), C=addr(2), ends=addr(3), G=3, T=20, M=48, N=40, lda=48, ldb=40, ldc=40, stridec=1920,
             dtype=lsm.GEMM_BF16_F32)
WGRAD_CASES = [
    ({}, VALID), (dict(h=None), INVALID), (dict(dtype=2), VALID), (dict(dtype=4), INVALID), (dict(G=-1), INVALID),
    (dict(T=-1), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(G=0), OK), (dict(M=0), OK), (dict(N=0), OK),
    (dict(T=0, A=0, B=0, lda=0, ldb=0), VALID), (dict(T=0, ends=0), INVALID),
    (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID), (dict(ends=0), INVALID),
    (dict(lda=40), INVALID), (dict(ldb=32), INVALID), (dict(ldc=39), INVALID), (dict(stridec=1919), INVALID),
    (dict(stridec=1919, G=1), VALID), (dict(stridec=-1920), INVALID), (dict(ldc=44, stridec=2108), VALID),
    (dict(ldc=44, stridec=2107), INVALID), (dict(M=44), UNSUPPORTED), (dict(N=36), UNSUPPORTED),
    (dict(lda=52), UNSUPPORTED), (dict(ldb=44), UNSUPPORTED), (dict(A=addr(0) + 8), UNSUPPORTED),
    (dict(B=addr(1) + 2), UNSUPPORTED), (dict(C=addr(2) + 2), UNSUPPORTED), (dict(ends=addr(3) + 1), UNSUPPORTED),
    (dict(lda=1 << 21), UNSUPPORTED), (dict(T=1 << 30), UNSUPPORTED), (dict(stridec=1 << 60), UNSUPPORTED),
    (dict(C=addr(0) + 1916), INVALID), (dict(C=addr(0) + 1920), VALID), (dict(C=addr(3) - 23040), VALID),
    (dict(C=addr(3) - 23036), INVALID),
]
GROUPED_MX = dict(A=addr(0), B=addr(1), C=addr(2), SA=addr(3), SB=addr(4), ends=addr(5), G=3, T=20, N=40, K=64, lda=64,
                  ldb=64, strideb=2560, ldc=40, ldsa=32, ldsb=48, stridesb=96, dtype=2)
GROUPED_MX_CASES = [
    ({}, VALID), (dict(h=None), INVALID), (dict(dtype=3), INVALID), (dict(G=-1), INVALID), (dict(T=-1), INVALID),
    (dict(G=0), OK), (dict(T=0), OK), (dict(N=0), OK), (dict(ends=0), INVALID), (dict(SA=0), INVALID), (dict(SB=0), INVALID),
    (dict(K=0, A=0, B=0, SA=0, SB=0), VALID), (dict(strideb=16), UNSUPPORTED), (dict(strideb=0), VALID),
    (dict(strideb=-32), INVALID), (dict(stridesb=8), UNSUPPORTED), (dict(stridesb=0), VALID), (dict(stridesb=-16), INVALID),
    (dict(ends=addr(5) + 2), UNSUPPORTED), (dict(K=48), UNSUPPORTED), (dict(N=41, ldc=41), VALID),
    (dict(ldsa=16), INVALID), (dict(ldsb=32), INVALID), (dict(strideb=1 << 40), UNSUPPORTED),
    (dict(C=addr(1) + 3836), INVALID), (dict(C=addr(1) + 3840), VALID), (dict(C=addr(4) + 284), INVALID),
    (dict(C=addr(4) + 288), VALID), (dict(C=addr(5) + 8), INVALID), (dict(C=addr(5) + 12), VALID),
]
ENTRIES = [(lsm.gemm_mxfp4_quantize_run, QUANTIZE, QUANTIZE_CASES),
           (lsm.gemm_mxfp4_dequantize_run, DEQUANTIZE, DEQUANTIZE_CASES), (lsm.gemm_mxfp4_run, PRODUCT, PRODUCT_CASES),
           (lsm.gemm_grouped_run, ROWS, ROWS_CASES), (lsm.gemm_grouped_wgrad_run, WGRAD, WGRAD_CASES),
           (lsm.gemm_grouped_mxfp4_run, GROUPED_MX, GROUPED_MX_CASES)]
FLAT = [(fn, base, *c) for fn, base, cases in ENTRIES for c in cases]


@pytest.mark.parametrize("fn,base,changes,status", FLAT,
                         ids=[f"{f.__name__[5:-4]}-{i}" for f, _, cases in ENTRIES for i in ids(cases)])
def test_checks(fn, base, changes, status):
    assert call(fn, base, changes) == status


@pytest.mark.parametrize("fn,base", [e[:2] for e in ENTRIES], ids=[e[0].__name__ for e in ENTRIES])
def test_binding(fn, base):
    """Pointer and stream objects, sizes that the C ABI cannot hold, handles that are none."""
    pointers = {k: Pointer(v) for k, v in base.items() if v >= addr(0)}
    assert call(fn, base, pointers) == VALID
    assert call(fn, base, dict(stream=type("Stream", (), {"cuda_stream": 0})())) == VALID
    for name, bits in (("K" if "K" in base else "N", 64), ("dtype", 32)):
        with pytest.raises(OverflowError):
            call(fn, base, {name: 1 << bits})
    for handle in (Valued(), Numbered(), 1.0):
        with pytest.raises(ctypes.ArgumentError):
            call(fn, base, dict(h=handle))


@isa.needs_tools
@pytest.mark.parametrize("name", ["gemm_grouped", "gemm_mxfp4"])
def test_lds_dma_wait_states(name, tmp_path):
    """The wait-state rules of test_isa_hazards.py on these translation units."""
    obj = os.path.join(isa.PKG, "_build", name + ".o")
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
    # a register that is spilled in the K loop would be reloaded behind the loads in flight
    assert not [t for t in ins if t and t.startswith("scratch_")]
