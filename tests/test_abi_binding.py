"""What the binding takes for a handle, and what it is built on (CPU; no call
below passes the device check)."""
import ctypes
import shutil
import subprocess

import numpy as np
import pytest

import lds_staged_matrix_amd as lsm
from test_abi_linear import FAKE, NORM, SCALED, VALID, W4, _FAKE_DEVICE, addr, lib  # noqa: F401

RUN = dict(A=addr(0), B=addr(1), C=addr(2), M=16, N=16, K=16, lda=16, ldb=16, ldc=16, layoutA=0, layoutB=0,
           dtype=lsm.GEMM_BF16_F32)
ENTRIES = [(lsm.gemm_run, RUN), (lsm.gemm_scaled_run, SCALED), (lsm.gemm_w4_run, W4), (lsm.gemm_rmsnorm_run, NORM)]
ADDRESS = ctypes.addressof(_FAKE_DEVICE)           # below 2^53: a float holds it


class Valued:
    value = ADDRESS


class Numbered:
    def __int__(self):
        return ADDRESS
    __index__ = __int__


class AsParameter:
    _as_parameter_ = FAKE


class Handle(ctypes.c_void_p):
    pass


def ids(entries):
    return [fn.__name__ for fn, _ in entries]


@pytest.mark.parametrize("fn,base", ENTRIES, ids=ids(ENTRIES))
@pytest.mark.parametrize("handle", [float(ADDRESS), np.int64(ADDRESS), np.array([ADDRESS]), ctypes.c_int64(ADDRESS),
                                    Valued(), Numbered()], ids=lambda h: type(h).__name__)
def test_no_handle(fn, base, handle):
    with pytest.raises(ctypes.ArgumentError):
        fn(handle, **base)


@pytest.mark.parametrize("fn,base", ENTRIES, ids=ids(ENTRIES))
@pytest.mark.parametrize("handle", [FAKE, ADDRESS, ADDRESS + (1 << 64), Handle(ADDRESS),
                                    ctypes.pointer(_FAKE_DEVICE), ctypes.byref(_FAKE_DEVICE), AsParameter()],
                         ids=lambda h: type(h).__name__)
def test_handles(fn, base, handle):
    """What a ctypes c_void_p parameter takes."""
    assert fn(handle, **base) == VALID


@pytest.mark.parametrize("fn,base", ENTRIES, ids=ids(ENTRIES))
@pytest.mark.parametrize("handle", [None, 0, ctypes.c_void_p()], ids=str)
def test_null_handles(fn, base, handle):
    assert fn(handle, **base) == lsm.GEMM_ERR_INVALID_ARG


def test_a_tensor_is_no_handle():
    torch = pytest.importorskip("torch")
    with pytest.raises(ctypes.ArgumentError):
        lsm.gemm_run(torch.tensor(ADDRESS), **RUN)


def test_one_build_for_every_python():
    """The binding is compiled against the stable ABI: of Python's own symbols it asks for documented
    functions only, and reads none of its objects' fields."""
    from lds_staged_matrix_amd import _binding
    assert _binding.limited_api == 0x030A0000
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("no nm")
    out = subprocess.run([nm, "-D", "--undefined-only", _binding.__file__], capture_output=True, text=True, check=True)
    names = {line.split()[-1] for line in out.stdout.splitlines() if "Py" in line}
    assert "PyLong_FromLong" in names
    # what the stable ABI's own macros expand to
    assert {n for n in names if n.startswith("_Py")} <= {"_Py_Dealloc", "_Py_NoneStruct"}
    assert "PyType_GetFlags" in names          # PyLong_Check through a call, not through the type's fields


E4M3 = (lsm.GEMM_E4M3_F32, lsm.GEMM_E4M3_BF16, lsm.GEMM_E4M3_F16)


def test_where_exact_sums_may_be_asked_for():
    flag = lsm.GEMM_EXACT_SUMS
    for d in E4M3:
        assert lsm.gemm_scaled_run(FAKE, **{**SCALED, "dtype": d + flag}) == VALID
        assert lsm.gemm_scaled_run(FAKE, **{**SCALED, "dtype": d + 2 * flag}) == lsm.GEMM_ERR_INVALID_ARG
        assert lsm.gemm_scaled_run(FAKE, **{**SCALED, "dtype": d - (1 << 31)}) == lsm.GEMM_ERR_INVALID_ARG
        assert lsm.gemm_run(FAKE, **{**RUN, "dtype": d + flag}) == lsm.GEMM_ERR_INVALID_ARG
    for d in (0, 1, 2, 3, 7):
        assert lsm.gemm_scaled_run(FAKE, **{**SCALED, "dtype": d + flag}) == lsm.GEMM_ERR_INVALID_ARG
    assert lsm.gemm_w4_run(FAKE, **{**W4, "dtype": W4["dtype"] + flag}) == lsm.GEMM_ERR_INVALID_ARG
    assert lsm.gemm_rmsnorm_run(FAKE, **{**NORM, "dtype": NORM["dtype"] + flag}) == lsm.GEMM_ERR_INVALID_ARG


def test_strides_of_absent_operands_do_not_count():
    assert lsm.gemm_w4_run(FAKE, **{**W4, "Z": 0, "ldz": 1 << 40}) == VALID
    assert lsm.gemm_w4_run(FAKE, **{**W4, "Z": 0, "ldz": -1}) == VALID
    assert lsm.gemm_rmsnorm_run(FAKE, **{**NORM, "R": 0, "ldr": 1 << 40, "H": 0, "ldh": -1}) == VALID
