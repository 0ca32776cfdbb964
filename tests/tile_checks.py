"""Checks of the grouped and of the MXFP4 products on the GPU against torch in fp64: rows of given groups, given
sizes, on the library or on the poison build.  Rows of no group, and what lies behind the operands' rows, are NaN."""
import numpy as np
import pytest
import torch

import gpu_harness as H
import grouped_reference as G
import lds_staged_matrix_amd as lsm
import linear_reference as R
from test_gpu_grouped import TYPE
from test_gpu_mxfp4 import DTYPE, LAYOUT

NAN = float("nan")
E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def uneven(T, groups):
    """The rows of `groups` groups of T rows, three of them in no group."""
    rng = np.random.default_rng([T, groups])
    return [int(n) for n in rng.multinomial(T - 3, rng.dirichlet(np.full(groups, 2.0)))] if T > 3 else [T] + [0] * (groups - 1)


def ends_of(rows):
    ends, at = [], 0
    for n in rows:
        at += n
        ends.append(at)
    return ends


def rows_in_all(rows):
    """Rows of the call's A: those of the groups and, of more than three, three of no group."""
    return sum(rows) + (3 if sum(rows) > 3 else 0)


@pytest.fixture(scope="module", params=["library", "poison"])
def build(request):
    if request.param == "library":
        yield lsm, H.handle()
        return
    lib = lsm.ablation_library("poison")
    h = lib.gemm_create()
    yield lib, h
    lib.gemm_destroy(h)


def ok(status, what):
    if status != lsm.GEMM_OK:
        raise lsm.GemmError(status, what)
    torch.cuda.synchronize()


class Data:
    def __init__(self, *key):
        self.g = torch.Generator(device="cuda").manual_seed(sum(ord(c) * (i + 1) for i, c in enumerate(repr(key))))

    def integers(self, lo, hi, *shape, dtype=torch.int64):
        return torch.randint(lo, hi, shape, generator=self.g, device="cuda", dtype=dtype)

    def values(self, dist, *shape):
        return self.integers(-2, 3, *shape).float() if dist == "int" else torch.randn(*shape, generator=self.g, device="cuda")


def padded(v, t, pad=8):
    """v in rows `pad` longer, NaN behind them."""
    buf = torch.full((*v.shape[:-1], v.shape[-1] + pad), NAN, dtype=t, device="cuda")
    buf[..., :v.shape[-1]] = v
    return buf


def matmul(a, b):
    return a.double() @ b.double()


def compare(got, ref, bound, out, what):
    """`bound` None: the rounding of ref."""
    if bound is None:
        bad = got.double() != ref.to(R.TORCH[out]).double()
    else:
        bad = ~((got.double() - ref).abs() <= bound + R.HALF_STEP[out] * (ref.abs() + bound) + R.SMALLEST[out])
    if bool(bad.any()):
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} entries off, first at {i}: got {float(got[i])!r} "
                             f"want {float(ref[i])!r}")


def check_rows(build, rows, N, K, layout, kind, out, dist, pad=8):
    lib, h = build
    ends, d = ends_of(rows), Data("rows", rows, N, K, layout, kind)
    T, n, t = rows_in_all(rows), len(rows), R.TORCH[kind]
    a = d.values(dist, T, K).to(t)
    a[ends[-1]:] = NAN                                        # rows of no group
    b = d.values(dist, n, *((N, K) if layout == "K" else (K, N))).to(t)
    A, B = padded(a, t), padded(b, t)
    C = torch.full((T + 1, N + pad), -99.0, dtype=R.TORCH[out], device="cuda")
    print("CASE rows", rows, N, K, layout, kind, out, dist, flush=True)
    ok(lib.gemm_grouped_run(h, A, B, C, torch.tensor(ends, dtype=torch.int32, device="cuda"), n, T, N, K, A.stride(0),
                            B.stride(1), B.stride(0), N + pad, LAYOUT[layout], TYPE[kind, out], torch.cuda.current_stream()),
       "gemm_grouped_run")
    assert bool((C[:, N:] == -99).all()) and bool((C[ends[-1]:] == -99).all())
    for g, (f, l) in enumerate(G.bounds(ends, T)):
        w = b[g].t() if layout == "K" else b[g]
        bound = None if dist == "int" else G.sum_bound(matmul(a[f:l].abs(), w.abs()), K)
        compare(C[f:l, :N], matmul(a[f:l], w), bound, out, f"group {g}")


class Mx:
    """A random MXFP4 matrix of M x K: its device arrays, padded with NaN scales and codes of 6, and its values (fp64)."""

    def __init__(self, d, M, K, dist, nan=()):
        code = d.integers(0, 16, M, K, dtype=torch.uint8)
        scale = d.integers(*((126, 129) if dist == "int" else (119, 128)), M, K // 32, dtype=torch.uint8)
        for row, block in nan:
            scale[row, block] = G.NAN_SCALE
        self.ldq, self.lds = K + 32, G.up(M, 16) + 16
        self.Q = torch.full((M, self.ldq // 2), 0x77, dtype=torch.uint8, device="cuda")
        self.Q[:, :K // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
        self.S = torch.full((K // 32, self.lds), G.NAN_SCALE, dtype=torch.uint8, device="cuda")
        self.S[:, :M] = scale.t()
        size = torch.where(scale == G.NAN_SCALE, NAN, torch.exp2(scale.double() - 127))
        self.v = E2M1.cuda()[code.long()] * size.repeat_interleave(32, 1)


def check_mx(got, a, b, K, out, dist, what):
    ref = a @ b.t()
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(got), nan), what
    bound = None if dist == "int" else (K / 128 + 8) * (2.0 ** -21 * (a.abs() @ b.abs().t())[~nan] + 2.0 ** -149)
    compare(got[~nan], ref[~nan], bound, out, what)


def check_product(build, M, N, K, out, dist, pad=3):
    lib, h = build
    d = Data("mx", M, N, K, out)
    last = K // 32 - 1
    a, b = Mx(d, M, K, dist, [(M // 3, last), (M - 1, last // 2)] if M > 16 else []), Mx(d, N, K, dist, [(N - 2, last)])
    C = torch.full((M + 1, N + pad), -99.0, dtype=R.TORCH[out], device="cuda")
    print("CASE mxfp4", M, N, K, out, dist, flush=True)
    ok(lib.gemm_mxfp4_run(h, a.Q, b.Q, C, a.S, b.S, M, N, K, a.ldq, b.ldq, N + pad, a.lds, b.lds, DTYPE[out],
                          torch.cuda.current_stream()), "gemm_mxfp4_run")
    assert bool((C[:, N:] == -99).all()) and bool((C[M:] == -99).all())
    check_mx(C[:M, :N], a.v, b.v, K, out, dist, "product")


def check_mx_rows(build, rows, N, K, out, dist, pad=3):
    lib, h = build
    ends, d, last = ends_of(rows), Data("mx rows", rows, N, K, out), K // 32 - 1
    T, n = rows_in_all(rows), len(rows)
    mine = [(rows[0] // 2, last), (ends[-1] - 5, last // 2)] if rows[0] and ends[-1] > 16 else []
    a = Mx(d, T, K, dist, mine + [(r, k) for r in range(ends[-1], T) for k in (0, last)])
    bs = [Mx(d, N, K, dist, [(N - 1, last)] if g == 0 else []) for g in range(n)]
    B, SB = torch.stack([b.Q for b in bs]), torch.stack([b.S for b in bs])
    C = torch.full((T + 1, N + pad), -99.0, dtype=R.TORCH[out], device="cuda")
    print("CASE mxfp4 rows", rows, N, K, out, dist, flush=True)
    ok(lib.gemm_grouped_mxfp4_run(h, a.Q, B, C, a.S, SB, torch.tensor(ends, dtype=torch.int32, device="cuda"), n, T, N, K, a.ldq,
                                  bs[0].ldq, 2 * B.stride(0), N + pad, a.lds, bs[0].lds, SB.stride(0), DTYPE[out],
                                  torch.cuda.current_stream()), "gemm_grouped_mxfp4_run")
    assert bool((C[:, N:] == -99).all()) and bool((C[ends[-1]:] == -99).all())
    for g, (f, l) in enumerate(G.bounds(ends, T)):
        check_mx(C[f:l, :N], a.v[f:l], bs[g].v, K, out, dist, f"group {g}")


def check_sums(build, rows, M, N, kind, out, dist, pad=8):
    lib, h = build
    ends, d = ends_of(rows), Data("sums", rows, M, N, kind, out)
    T, n, t = rows_in_all(rows), len(rows), R.TORCH[kind]
    a, b = d.values(dist, T, M).to(t), d.values(dist, T, N).to(t)
    a[ends[-1]:], b[ends[-1]:] = NAN, float("inf")            # rows of no group
    A, B = padded(a, t), padded(b, t)
    C = torch.full((n, M + 1, N + pad), -99.0, dtype=R.TORCH[out], device="cuda")
    print("CASE sums", rows, M, N, kind, out, dist, flush=True)
    ok(lib.gemm_grouped_wgrad_run(h, A, B, C, torch.tensor(ends, dtype=torch.int32, device="cuda"), n, T, M, N, A.stride(0),
                                  B.stride(0), N + pad, C.stride(0), TYPE[kind, out], torch.cuda.current_stream()),
       "gemm_grouped_wgrad_run")
    assert bool((C[:, M:] == -99).all()) and bool((C[:, :, N:] == -99).all())
    for g, (f, l) in enumerate(G.bounds(ends, T)):
        bound = None if dist == "int" else G.sum_bound(matmul(a[f:l].t().abs(), b[f:l].abs()), l - f)
        compare(C[g, :M, :N], matmul(a[f:l].t(), b[f:l]), bound, out, f"group {g}")
