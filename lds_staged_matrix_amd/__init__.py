"""Python binding of the LDS-staged GEMM C ABI (include/lds_gemm.h).

Argument marshalling only: every step of C <- A*B runs in the HIP library
liblds_gemm.so built in this directory; the calls that enqueue work go through
_binding.so (csrc/binding.c), the others through ctypes.  There is no fallback:
if either is missing, the entry points raise.

Names mirror the C ABI: gemm_create, gemm_run, gemm_destroy, gemm_status_str,
and the operators of a quantised linear layer: gemm_rmsnorm_run (norm with the
residual's addition, 16-bit or scaled E4M3 output), gemm_scaled_run (E4M3
product with row and column scales) and gemm_w4_run (few rows times 4-bit
weights).
Pointers may be passed as integers or as objects with a ``data_ptr()`` method
(torch tensors); streams as integers, objects with a ``cuda_stream``
attribute (torch streams) or None for the null stream.
"""
import ctypes
import os

__all__ = [
    "GEMM_K_CONTIG", "GEMM_MN_CONTIG",
    "GEMM_BF16_F32", "GEMM_BF16_BF16", "GEMM_F16_F16", "GEMM_F16_F32", "GEMM_E4M3_F32",
    "GEMM_E4M3_BF16", "GEMM_E4M3_F16", "GEMM_EXACT_SUMS",
    "GEMM_NORM_BF16_BF16", "GEMM_NORM_BF16_E4M3", "GEMM_NORM_F16_F16", "GEMM_NORM_F16_E4M3",
    "GEMM_OK", "GEMM_ERR_INVALID_ARG", "GEMM_ERR_UNSUPPORTED", "GEMM_ERR_DEVICE",
    "GEMM_ERR_LAUNCH", "GemmError", "library_path", "load_library", "gemm_create",
    "gemm_run", "gemm_scaled_run", "gemm_w4_run", "gemm_rmsnorm_run", "gemm_destroy",
    "gemm_status_str", "EXPORTED_SYMBOLS", "Library", "ablation_library",
]

GEMM_K_CONTIG, GEMM_MN_CONTIG = 0, 1
GEMM_BF16_F32, GEMM_BF16_BF16, GEMM_F16_F16, GEMM_F16_F32 = 0, 1, 2, 3
GEMM_E4M3_F32, GEMM_E4M3_BF16, GEMM_E4M3_F16 = 4, 5, 6
GEMM_EXACT_SUMS = 0x100     # added to gemm_scaled_run's dtype
GEMM_NORM_BF16_BF16, GEMM_NORM_BF16_E4M3, GEMM_NORM_F16_F16, GEMM_NORM_F16_E4M3 = range(4)
GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_UNSUPPORTED, GEMM_ERR_DEVICE, GEMM_ERR_LAUNCH = range(5)
EXPORTED_SYMBOLS = ("gemm_create", "gemm_run", "gemm_scaled_run", "gemm_w4_run", "gemm_rmsnorm_run",
                    "gemm_destroy", "gemm_status_str")

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "liblds_gemm.so"
_lib = None
_native = None


class GemmError(RuntimeError):
    def __init__(self, status, what):
        super().__init__(f"{what}: {gemm_status_str(status)} (status {status})")
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


# The linear layer's entry points: pointers, 64-bit sizes and what follows them before the stream.
_LAYER = (("gemm_scaled_run", 5, 6, [ctypes.c_int] * 5), ("gemm_w4_run", 5, 9, [ctypes.c_int]),
          ("gemm_rmsnorm_run", 6, 6, [ctypes.c_float, ctypes.c_int]))


def _open(path):
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with lds_staged_matrix_amd/build.py "
                           "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(path)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.gemm_create.argtypes = [ctypes.POINTER(vp)]
    lib.gemm_create.restype = i32
    lib.gemm_run.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i32, i32, i32, vp]
    lib.gemm_run.restype = i32
    lib.gemm_destroy.argtypes = [vp]
    lib.gemm_destroy.restype = i32
    lib.gemm_status_str.argtypes = [i32]
    lib.gemm_status_str.restype = ctypes.c_char_p
    for name, pointers, sizes, tail in _LAYER:
        if hasattr(lib, name):          # not in the A/B builds of gemm_run alone
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = [vp] * (1 + pointers) + [i64] * sizes + tail + [vp], i32
    return lib


def load_library():
    """Load liblds_gemm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        _lib = _open(library_path())
    return _lib


def _bind():
    """The module _binding (csrc/binding.c) on load_library()'s entry points."""
    global _native
    lib = load_library()
    if not os.path.exists(os.path.join(_HERE, "_binding.so")):
        raise RuntimeError(f"_binding.so is missing from {_HERE}: build it with lds_staged_matrix_amd/build.py "
                           "(or __graft_entry__.build()); there is no fallback path")
    from . import _binding
    _binding.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                    for name in ("gemm_run", "gemm_scaled_run", "gemm_w4_run", "gemm_rmsnorm_run")))
    _native = _binding
    return _native


def _ptr(x):
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def _int(x, bits, name):
    """x as a Python int that fits the C ABI's signed `bits`-bit parameter.
    ctypes would silently keep only the low bits of a larger value."""
    v = int(x)
    if not -(1 << (bits - 1)) <= v < (1 << (bits - 1)):
        raise OverflowError(f"{name}={v} does not fit the C ABI's int{bits}_t parameter")
    return v


def _sizes(M, N, K, lda, ldb, ldc, layoutA, layoutB, dtype):
    return ([_int(v, 64, n) for v, n in zip((M, N, K, lda, ldb, ldc),
                                             ("M", "N", "K", "lda", "ldb", "ldc"))] +
            [_int(v, 32, n) for v, n in zip((layoutA, layoutB, dtype),
                                             ("layoutA", "layoutB", "dtype"))])


def _stream(s):
    if s is None:
        return None
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    return int(s)


def gemm_create():
    """Create a handle on the current device; raises GemmError on failure."""
    h = ctypes.c_void_p()
    st = load_library().gemm_create(ctypes.byref(h))
    if st != GEMM_OK:
        raise GemmError(st, "gemm_create")
    return h


def gemm_run(h, A, B, C, M, N, K, lda, ldb, ldc, layoutA, layoutB, dtype, stream=None) -> int:
    """Enqueue C <- A*B; returns the gemm_status code (0 on success)."""
    return (_native or _bind()).run(h, A, B, C, M, N, K, lda, ldb, ldc, layoutA, layoutB, dtype, stream)


def gemm_scaled_run(h, A, B, C, SA, SB, M, N, K, lda, ldb, ldc, incA, incB, layoutA, layoutB, dtype,
                    stream=None) -> int:
    """Enqueue C <- diag(SA) A B diag(SB) for E4M3 operands; returns the gemm_status code."""
    return (_native or _bind()).scaled(h, A, B, C, SA, SB, M, N, K, lda, ldb, ldc, incA, incB, layoutA, layoutB,
                                       dtype, stream)


def gemm_w4_run(h, A, B, S, Z, C, M, N, K, group, lda, ldb, lds, ldz, ldc, dtype, stream=None) -> int:
    """Enqueue the product of 16-bit rows with 4-bit weights; returns the gemm_status code."""
    return (_native or _bind()).w4(h, A, B, S, Z, C, M, N, K, group, lda, ldb, lds, ldz, ldc, dtype, stream)


def gemm_rmsnorm_run(h, X, R, W, H, Y, S, M, N, ldx, ldr, ldh, ldy, eps, dtype, stream=None) -> int:
    """Enqueue the RMS norm of X (+ R); returns the gemm_status code."""
    return (_native or _bind()).rmsnorm(h, X, R, W, H, Y, S, M, N, ldx, ldr, ldh, ldy, eps, dtype, stream)


def gemm_destroy(h) -> int:
    return load_library().gemm_destroy(h)


def gemm_status_str(status: int) -> str:
    return load_library().gemm_status_str(_int(status, 32, "status")).decode()


class Library:
    """gemm_create, gemm_run, gemm_destroy and gemm_status_str bound to one
    specific build of the library (the default build, or an A/B build from
    ablation_library()); the linear layer's entry points where the build has
    them (the default build and "poison")."""

    def __init__(self, path):
        self.path = path
        self._lib = _open(path)

    def gemm_create(self):
        h = ctypes.c_void_p()
        st = self._lib.gemm_create(ctypes.byref(h))
        if st != GEMM_OK:
            raise GemmError(st, "gemm_create")
        return h

    def gemm_run(self, h, A, B, C, M, N, K, lda, ldb, ldc, layoutA, layoutB, dtype,
                 stream=None) -> int:
        return self._lib.gemm_run(h, _ptr(A), _ptr(B), _ptr(C),
                                  *_sizes(M, N, K, lda, ldb, ldc, layoutA, layoutB, dtype),
                                  _stream(stream))

    def _layer(self, name, h, args, stream):
        _, np, nw, tail = next(e for e in _LAYER if e[0] == name)
        p, w, t = args[:np], args[np:np + nw], args[np + nw:]
        return getattr(self._lib, name)(h, *map(_ptr, p), *(_int(v, 64, name) for v in w),
                                        *(v if c is ctypes.c_float else _int(v, 32, name) for v, c in zip(t, tail)),
                                        _stream(stream))

    def gemm_scaled_run(self, h, A, B, C, SA, SB, M, N, K, lda, ldb, ldc, incA, incB, layoutA, layoutB, dtype,
                        stream=None) -> int:
        return self._layer("gemm_scaled_run", h, (A, B, C, SA, SB, M, N, K, lda, ldb, ldc, incA, incB, layoutA,
                                                  layoutB, dtype), stream)

    def gemm_w4_run(self, h, A, B, S, Z, C, M, N, K, group, lda, ldb, lds, ldz, ldc, dtype, stream=None) -> int:
        return self._layer("gemm_w4_run", h, (A, B, S, Z, C, M, N, K, group, lda, ldb, lds, ldz, ldc, dtype), stream)

    def gemm_rmsnorm_run(self, h, X, R, W, H, Y, S, M, N, ldx, ldr, ldh, ldy, eps, dtype, stream=None) -> int:
        return self._layer("gemm_rmsnorm_run", h, (X, R, W, H, Y, S, M, N, ldx, ldr, ldh, ldy, eps, dtype), stream)

    def gemm_destroy(self, h) -> int:
        return self._lib.gemm_destroy(h)

    def gemm_status_str(self, status: int) -> str:
        return self._lib.gemm_status_str(_int(status, 32, "status")).decode()


def ablation_library(name: str) -> Library:
    """An A/B build of the library that changes one design choice (names in
    build.VARIANTS); built by build.build_all().  Only benchmarks and tests
    use these."""
    from . import build as _build
    if name not in _build.VARIANTS:
        raise ValueError(f"unknown ablation build {name!r}; known: {sorted(_build.VARIANTS)}")
    return Library(_build.variant_path(name))
