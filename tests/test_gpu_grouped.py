"""gemm_grouped_run, gemm_grouped_wgrad_run and gemm_grouped_mxfp4_run on the GPU against fp64
(grouped_reference.py): group patterns, sizes, types, layouts, and runs of them together."""
import numpy as np
import pytest
import torch

import gpu_harness as H
import grouped_reference as G
import lds_staged_matrix_amd as lsm
import linear_reference as R
from test_gpu_mxfp4 import DTYPE as MXTYPE, LAYOUT, mx_operand, ok, operand, rng_of

pytestmark = pytest.mark.gpu

TYPE = {("bf16", "bf16"): lsm.GEMM_BF16_BF16, ("bf16", "f32"): lsm.GEMM_BF16_F32, ("f16", "f16"): lsm.GEMM_F16_F16,
        ("f16", "f32"): lsm.GEMM_F16_F32}
NAN = float("nan")


def split(rng, T, groups, how):
    """Ends of `groups` groups of T rows."""
    if how == "even":
        return np.arange(1, groups + 1) * T // groups
    if how == "skew":
        w = rng.random(groups) ** 6 + 1e-3
        return np.minimum(np.round(np.cumsum(w / w.sum()) * T).astype(int), T)
    if how == "gaps":            # every other group is empty, and rows are left at the end
        n = np.where(np.arange(groups) % 2 == 0, 1, 0) * rng.integers(1, max(2, T // max(1, groups)), groups)
        return np.minimum(np.cumsum(n), T)
    if how == "first":
        return np.full(groups, T)
    if how == "last":
        return np.where(np.arange(groups) == groups - 1, T, 0)
    if how == "none":
        return np.zeros(groups, int)
    # ends that mean less than they say: beyond T, negative, going back
    e = np.cumsum(rng.integers(0, 2 * T // groups + 2, groups))
    e[groups // 2] = -5
    e[groups // 3] = e[groups // 3] // 2
    e[-1] = T + 1000
    return e


def integers(rng, shape):
    return rng.integers(-2, 3, shape).astype(np.float64)


def data(rng, shape, kind, dist):
    return integers(rng, shape) if dist == "int" else R.round_to(rng.standard_normal(shape), kind)


def padded(values, kind, pad=8):
    """The last axis in rows `pad` longer, NaN behind it."""
    t = R.TORCH[kind]
    buf = torch.full((*values.shape[:-1], values.shape[-1] + pad), NAN).to(t).cuda()
    buf[..., :values.shape[-1]] = torch.from_numpy(values).to(t)
    return buf


def ends_of(ends):
    return torch.tensor(np.asarray(ends), dtype=torch.int32, device="cuda")


def compare(got, ref, size, K, out, dist, what):
    if dist == "int":
        bad = np.nonzero(got != R.round_to(ref, out))
        assert not bad[0].size, (what, bad[0].size, [int(b[0]) for b in bad], got[bad][:3], ref[bad][:3])
    else:
        bound = G.sum_bound(size, K)
        R.assert_within(got, ref, bound + R.HALF_STEP[out] * (np.abs(ref) + bound) + R.SMALLEST[out], what)


# --------------------------------------------------------------------- rows

def check_rows(T, groups, N, K, kind, out, layout, how, dist, pad=8, lib=None):
    rng = rng_of(T, groups, N, K, how, dist)
    ends = split(rng, T, groups, how)
    a, b = data(rng, (T, K), kind, dist), data(rng, (groups, N, K), kind, dist)
    spans = G.bounds(ends, T)
    if spans[-1][1] < T:
        a[spans[-1][1]:] = NAN                     # rows of no group
    A = padded(a, kind)
    B = padded(b if layout == "K" else np.ascontiguousarray(b.transpose(0, 2, 1)), kind)
    ldc = N + pad
    C = torch.full((T + 1, ldc), -99.0, dtype=R.TORCH[out], device="cuda")
    print("CASE grouped", T, groups, N, K, kind, out, layout, how, dist, flush=True)
    ok((lib or lsm).gemm_grouped_run(H.handle(), A, B, C, ends_of(ends), groups, T, N, K, A.stride(0), B.stride(1),
                                     B.stride(0), ldc, LAYOUT[layout], TYPE[kind, out], torch.cuda.current_stream()),
       "gemm_grouped_run")
    got = R.f64(C)
    assert (got[:, N:] == -99).all() and (got[spans[-1][1]:] == -99).all()
    for g, (f, l) in enumerate(spans):
        compare(got[f:l, :N], a[f:l] @ b[g].T, np.abs(a[f:l]) @ np.abs(b[g]).T, K, out, dist, f"group {g} rows {f}:{l}")


HOWS = ["even", "skew", "gaps", "first", "last", "none", "odd"]
# (T, groups, N, K): between them every kernel that the host chooses: streams of a mean of up to 16 and 32 rows in 16 to
# 128 columns; tiles that share K; 64 x 128, 128 x 128, also alone on a CU; 256 x 256 and its parts
ROWS = [(1, 1, 8, 8), (5, 3, 40, 72), (64, 16, 264, 520), (130, 130, 48, 136), (200, 9, 136, 64), (300, 12, 200, 1032),
        (700, 5, 400, 328), (1500, 8, 896, 1152), (500, 10, 2504, 200), (1000, 20, 2104, 136), (2000, 14, 2104, 136),
        (2600, 4, 4096, 136), (4096, 4, 4096, 200), (40, 40, 400, 64), (664, 40, 416, 64), (365, 20, 224, 64),
        (8157, 2, 80, 672), (3, 3, 5456, 64), (203, 12, 1400, 64), (36, 1, 24, 64), (7672, 40, 136, 352),
        (7903, 12, 136, 352), (1842, 20, 2512, 64), (4430, 40, 1032, 64)]


@pytest.mark.parametrize("T,groups,N,K", ROWS)
@pytest.mark.parametrize("layout", ["K", "MN"])
@pytest.mark.parametrize("how", HOWS)
def test_rows_exact(T, groups, N, K, layout, how):
    kind, out = sorted(TYPE)[(T + len(how)) % 4]
    check_rows(T, groups, N, K, kind, out, layout, how, "int", pad=len(how) % 4)


@pytest.mark.parametrize("T,groups,N,K", [(20, 4, 264, 1032), (100, 4, 264, 1032), (700, 5, 400, 1032), (4096, 4, 4096, 264)])
@pytest.mark.parametrize("layout", ["K", "MN"])
@pytest.mark.parametrize("kind,out", sorted(TYPE))
def test_rows_real(T, groups, N, K, layout, kind, out):
    check_rows(T, groups, N, K, kind, out, layout, "skew", "normal")


@pytest.mark.parametrize("N", [1, 31, 33, 127, 1151])
@pytest.mark.parametrize("T", [6, 50, 600])
def test_rows_odd_columns(N, T):
    check_rows(T, 3, N, 72, "bf16", "bf16", "K", "skew", "int", pad=1)


def test_rows_256_tiles_odd_columns():
    check_rows(5000, 4, 3585, 72, "bf16", "f32", "K", "skew", "int", pad=0)


@pytest.mark.parametrize("K", [8, 64, 72, 128, 136, 192, 264, 520])
@pytest.mark.parametrize("layout", ["K", "MN"])
def test_rows_256_tiles_by_k(K, layout):
    """One K tile, two, three and more, cut and whole, in tiles of 256 rows and in parts of 128 and 64."""
    ends = [256, 256 + 200, 256 + 200 + 128 + 100, 256 + 200 + 228 + 64, 748 + 33, 781 + 700, 1481 + 1]
    rng = rng_of(K)
    T, n, N = 1600, len(ends), 2048
    a, b = integers(rng, (T, K)), integers(rng, (n, N, K))
    A = padded(a, "bf16")
    B = padded(b if layout == "K" else np.ascontiguousarray(b.transpose(0, 2, 1)), "bf16")
    C = torch.full((T, N), -99.0, device="cuda")
    ok(lsm.gemm_grouped_run(H.handle(), A, B, C, ends_of(ends), n, T, N, K, A.stride(0), B.stride(1), B.stride(0), N,
                            LAYOUT[layout], lsm.GEMM_BF16_F32, torch.cuda.current_stream()), "gemm_grouped_run")
    got = R.f64(C)
    for g, (f, l) in enumerate(G.bounds(ends, T)):
        assert np.array_equal(got[f:l], a[f:l] @ b[g].T), (g, f, l)
    assert (got[ends[-1]:] == -99).all()


@pytest.mark.parametrize("groups", [63, 64, 65, 200])
def test_many_groups(groups):
    for how in ("skew", "gaps", "odd", "last"):
        check_rows(3 * groups + 1, groups, 40, 64, "bf16", "f32", "K", how, "int")


def test_one_matrix_for_all_groups():
    rng = rng_of(5)
    a, b = integers(rng, (50, 64)), integers(rng, (40, 64))
    A, B, C = padded(a, "bf16"), padded(b, "bf16"), torch.zeros(50, 40, device="cuda")
    ok(lsm.gemm_grouped_run(H.handle(), A, B, C, ends_of([7, 20, 50]), 3, 50, 40, 64, 72, 72, 0, 40, 0,
                            lsm.GEMM_BF16_F32, torch.cuda.current_stream()), "gemm_grouped_run")
    assert np.array_equal(R.f64(C), a @ b.T)


@pytest.mark.parametrize("T", [5, 40, 600])
def test_rows_empty_sum(T):
    C = torch.full((T, 40), 5.0, device="cuda")
    ok(lsm.gemm_grouped_run(H.handle(), None, None, C, ends_of([2, 4]), 2, T, 40, 0, 0, 0, 0, 40, 1,
                            lsm.GEMM_BF16_F32, torch.cuda.current_stream()), "gemm_grouped_run")
    assert bool((C[:4] == 0).all()) and bool((C[4:] == 5).all())


def test_infinities_stay_in_their_rows():
    rng = rng_of(8)
    for T in (12, 60, 600):
        a, b = integers(rng, (T, 64)), integers(rng, (2, 40, 64))
        a[T // 4, 3], a[T // 2, 7] = np.inf, np.nan
        A, B, C = padded(a, "bf16"), padded(b, "bf16"), torch.zeros(T, 40, device="cuda")
        ok(lsm.gemm_grouped_run(H.handle(), A, B, C, ends_of([T // 2, T]), 2, T, 40, 64, 72, 72, 40 * 72, 40, 0,
                                lsm.GEMM_BF16_F32, torch.cuda.current_stream()), "gemm_grouped_run")
        with np.errstate(invalid="ignore"):
            ref = np.concatenate([a[:T // 2] @ b[0].T, a[T // 2:] @ b[1].T])
        assert np.array_equal(R.f64(C), ref, equal_nan=True)


# -------------------------------------------------------------------- wgrad

def check_wgrad(T, groups, M, N, kind, out, how, dist, pad=8):
    rng = rng_of(T, groups, M, N, how, dist)
    ends = split(rng, T, groups, how)
    a, b = data(rng, (T, M), kind, dist), data(rng, (T, N), kind, dist)
    spans = G.bounds(ends, T)
    a[spans[-1][1]:], b[spans[-1][1]:] = NAN, np.inf          # rows of no group
    A, B = padded(a, kind), padded(b, kind)
    ldc = N + pad
    C = torch.full((groups, M + 1, ldc), -99.0, dtype=R.TORCH[out], device="cuda")
    print("CASE wgrad", T, groups, M, N, kind, out, how, dist, flush=True)
    ok(lsm.gemm_grouped_wgrad_run(H.handle(), A, B, C, ends_of(ends), groups, T, M, N, A.stride(0), B.stride(0), ldc,
                                  C.stride(0), TYPE[kind, out], torch.cuda.current_stream()), "gemm_grouped_wgrad_run")
    got = R.f64(C)
    assert (got[:, M:] == -99).all() and (got[:, :, N:] == -99).all()
    for g, (f, l) in enumerate(spans):
        compare(got[g, :M, :N], a[f:l].T @ b[f:l], np.abs(a[f:l]).T @ np.abs(b[f:l]), l - f, out, dist, f"group {g}")


WGRAD = [(1, 1, 8, 8), (5, 3, 40, 72), (64, 16, 136, 264), (130, 130, 16, 24), (700, 5, 264, 400), (1500, 8, 1152, 896),
         (700, 5, 784, 896), (900, 4, 2048, 2056), (2100, 4, 2048, 2056), (3004, 40, 16, 416), (3218, 8, 144, 7800),
         (1400, 70, 264, 520), (300, 130, 264, 264), (246, 2, 16, 8496), (262, 2, 80, 16320)]


@pytest.mark.parametrize("T,groups,M,N", WGRAD)
@pytest.mark.parametrize("how", HOWS)
def test_wgrad_exact(T, groups, M, N, how):
    kind, out = sorted(TYPE)[(T + len(how)) % 4]
    check_wgrad(T, groups, M, N, kind, out, how, "int", pad=len(how) % 4)


@pytest.mark.parametrize("T,groups,M,N", [(700, 5, 264, 400), (900, 4, 2048, 2056)])
@pytest.mark.parametrize("kind,out", sorted(TYPE))
def test_wgrad_real(T, groups, M, N, kind, out):
    check_wgrad(T, groups, M, N, kind, out, "skew", "normal")


def test_wgrad_without_rows():
    C = torch.full((2, 16, 24), 5.0, device="cuda")
    ok(lsm.gemm_grouped_wgrad_run(H.handle(), None, None, C, ends_of([0, 0]), 2, 0, 16, 24, 0, 0, 24, 16 * 24,
                                  lsm.GEMM_BF16_F32, torch.cuda.current_stream()), "gemm_grouped_wgrad_run")
    assert bool((C == 0).all())


# ------------------------------------------------------------ beyond 32 bits

def test_rows_and_sums_beyond_4_gib():
    """Operands of more than 2^32 bytes: the last rows, and a group's sum over all of them."""
    T, K, N = 300000, 8192, 64
    A = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    tail = torch.randint(-2, 3, (300, K), generator=g, device="cuda").bfloat16()
    A[-300:] = tail
    B = torch.randint(-2, 3, (2, N, K), generator=g, device="cuda").bfloat16()
    C = torch.full((T, N), 9.0, device="cuda")
    ends = ends_of([T - 100, T - 1])
    ok(lsm.gemm_grouped_run(H.handle(), A, B, C, ends, 2, T, N, K, K, K, N * K, N, lsm.GEMM_K_CONTIG, lsm.GEMM_BF16_F32,
                            torch.cuda.current_stream()), "gemm_grouped_run")
    t, w = R.f64(tail), R.f64(B)
    assert np.array_equal(R.f64(C[-300:-100]), t[:200] @ w[0].T)
    assert np.array_equal(R.f64(C[-100:-1]), t[200:-1] @ w[1].T)
    assert bool((C[:-300] == 0).all()) and bool((C[-1] == 9).all())
    # the sum over T - 100 rows, all but 200 of them zero, ends in rows beyond 2^32 bytes
    D = torch.randint(-2, 3, (T, 16), generator=g, device="cuda").bfloat16()
    W = torch.zeros(2, K, 16, device="cuda")
    ok(lsm.gemm_grouped_wgrad_run(H.handle(), A, D, W, ends, 2, T, K, 16, K, 16, 16, 16 * K, lsm.GEMM_BF16_F32,
                                  torch.cuda.current_stream()), "gemm_grouped_wgrad_run")
    d = R.f64(D[-300:])
    assert np.array_equal(R.f64(W[0]), t[:200].T @ d[:200])
    assert np.array_equal(R.f64(W[1]), t[200:-1].T @ d[200:-1])


# -------------------------------------------------------------------- MXFP4

def check_mx(T, groups, N, K, out, how, dist, pad=3):
    rng = rng_of(T, groups, N, K, how, dist)
    ends = split(rng, T, groups, how)
    spans = G.bounds(ends, T)
    ca, sa = operand(rng, T, K, dist)
    sa[spans[-1][1]:] = G.NAN_SCALE                           # rows of no group
    A, SA, lda, ldsa = mx_operand(ca, sa)
    weights = [operand(rng, N, K, dist) for _ in range(groups)]
    dev = [mx_operand(*w) for w in weights]
    B, SB = torch.stack([d[0] for d in dev]), torch.stack([d[1] for d in dev])
    ldb, ldsb, ldc = dev[0][2], dev[0][3], N + pad
    C = torch.full((T + 1, ldc), -99.0, dtype=R.TORCH[out], device="cuda")
    print("CASE grouped mxfp4", T, groups, N, K, out, how, dist, flush=True)
    ok(lsm.gemm_grouped_mxfp4_run(H.handle(), A, B, C, SA, SB, ends_of(ends), groups, T, N, K, lda, ldb,
                                  2 * B.stride(0), ldc, ldsa, ldsb, SB.stride(0), MXTYPE[out],
                                  torch.cuda.current_stream()), "gemm_grouped_mxfp4_run")
    got = R.f64(C)
    assert (got[:, N:] == -99).all() and (got[spans[-1][1]:] == -99).all()
    a = G.values(ca, sa)
    for g, (f, l) in enumerate(spans):
        ref, bound = G.product(a[f:l], G.values(*weights[g]))
        if dist == "exact":
            assert np.array_equal(got[f:l, :N], R.round_to(ref, out)), (g, f, l)
        else:
            R.assert_within(got[f:l, :N], ref, bound + R.HALF_STEP[out] * (np.abs(ref) + bound) + R.SMALLEST[out],
                            f"group {g}")


MX = [(1, 1, 8, 32), (5, 3, 40, 96), (64, 16, 264, 544), (130, 130, 48, 288), (200, 9, 136, 64), (300, 12, 200, 1056),
      (100, 50, 400, 96), (900, 40, 420, 96), (700, 5, 400, 320), (1500, 8, 897, 1152), (500, 10, 2500, 288),
      (1000, 20, 2100, 160), (2000, 14, 2100, 288), (4100, 4, 4096, 288), (8013, 40, 1080, 64), (7581, 20, 80, 896),
      (442, 5, 10776, 64), (37, 1, 24, 8512), (5311, 1, 672, 1696), (7963, 20, 72, 2016),
      (64, 32, 1032, 288)]


@pytest.mark.parametrize("T,groups,N,K", MX)
@pytest.mark.parametrize("how", HOWS)
def test_mx_exact(T, groups, N, K, how):
    check_mx(T, groups, N, K, sorted(MXTYPE)[(T + len(how)) % 3], how, "exact", pad=len(how) % 4)


@pytest.mark.parametrize("T,groups,N,K", [(20, 4, 264, 1056), (100, 4, 264, 1056), (700, 5, 400, 1056)])
@pytest.mark.parametrize("dist", ["normal", "wide"])
def test_mx_real(T, groups, N, K, dist):
    check_mx(T, groups, N, K, "f32", "skew", dist)


# ----------------------------------------------------- together, and captured

class Experts:
    """A feed-forward layer of experts, forward and backward: rows sorted by expert through two matrices
    with a squared ReLU between them."""

    def __init__(self, T, D, F, ends, seed):
        rng = rng_of(T, D, F, seed)
        self.T, self.D, self.F, self.ends, self.n = T, D, F, ends, len(ends)
        bf = lambda v: torch.from_numpy(v).bfloat16().cuda()
        self.x, self.w1 = bf(rng.standard_normal((T, D))), bf(rng.standard_normal((self.n, F, D)) / D ** 0.5)
        self.w2, self.dy = bf(rng.standard_normal((self.n, D, F)) / F ** 0.5), bf(rng.standard_normal((T, D)))
        self.end = ends_of(ends)
        z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")
        self.h, self.a, self.y = z(T, F), z(T, F), z(T, D, t=torch.float32)
        self.da, self.dh, self.dx = z(T, F), z(T, F), z(T, D, t=torch.float32)
        self.dw1, self.dw2 = z(self.n, F, D, t=torch.float32), z(self.n, D, F, t=torch.float32)

    def rows(self, A, B, C, N, K, layout, out):
        ok_async(lsm.gemm_grouped_run(H.handle(), A, B, C, self.end, self.n, self.T, N, K, A.stride(0), B.stride(1),
                                      B.stride(0), C.stride(0), layout, TYPE["bf16", out], torch.cuda.current_stream()))

    def grad(self, A, B, C):
        ok_async(lsm.gemm_grouped_wgrad_run(H.handle(), A, B, C, self.end, self.n, self.T, A.shape[1], B.shape[1],
                                            A.stride(0), B.stride(0), C.stride(1), C.stride(0), lsm.GEMM_BF16_F32,
                                            torch.cuda.current_stream()))

    def step(self):
        T, D, F = self.T, self.D, self.F
        self.rows(self.x, self.w1, self.h, F, D, lsm.GEMM_K_CONTIG, "bf16")
        torch.mul(self.h.clamp(min=0), self.h.clamp(min=0), out=self.a)
        self.rows(self.a, self.w2, self.y, D, F, lsm.GEMM_K_CONTIG, "f32")
        self.grad(self.dy, self.a, self.dw2)
        self.rows(self.dy, self.w2, self.da, F, D, lsm.GEMM_MN_CONTIG, "bf16")
        torch.mul(self.da, 2 * self.h.clamp(min=0), out=self.dh)
        self.rows(self.dh, self.w1, self.dx, D, F, lsm.GEMM_MN_CONTIG, "f32")
        self.grad(self.dh, self.x, self.dw1)

    OUT = ("h", "y", "da", "dx", "dw1", "dw2")

    def check(self):
        """Each product against fp64 on its own inputs, as the step left them."""
        f = R.f64
        x, w1, w2, dy, a, dh, h, da = (f(getattr(self, k)) for k in ("x", "w1", "w2", "dy", "a", "dh", "h", "da"))
        for g, (s, e) in enumerate(G.bounds(self.ends, self.T)):
            for got, p, q, K, out, what in ((h[s:e], x[s:e], w1[g].T, self.D, "bf16", "h"),
                                            (f(self.y)[s:e], a[s:e], w2[g].T, self.F, "f32", "y"),
                                            (da[s:e], dy[s:e], w2[g], self.D, "bf16", "da"),
                                            (f(self.dx)[s:e], dh[s:e], w1[g], self.F, "f32", "dx"),
                                            (f(self.dw2)[g], dy[s:e].T, a[s:e], e - s, "f32", "dw2"),
                                            (f(self.dw1)[g], dh[s:e].T, x[s:e], e - s, "f32", "dw1")):
                compare(got, p @ q, np.abs(p) @ np.abs(q), K, out, "normal", f"{what} group {g}")


def ok_async(st):
    if st != lsm.GEMM_OK:
        raise lsm.GemmError(st, "grouped")


@pytest.mark.parametrize("T", [24, 100, 900])
def test_experts_step(T):
    e = Experts(T, 256, 384, [T // 3, T // 3, T - 3], 1)
    e.step()
    torch.cuda.synchronize()
    e.check()


def test_gradients_against_differences():
    """The step's gradients along random directions against differences of the loss <y, dy> in fp64."""
    e = Experts(90, 64, 96, [30, 31, 90], 2)
    e.step()
    torch.cuda.synchronize()
    x, w1, w2, dy = (R.f64(getattr(e, k)) for k in ("x", "w1", "w2", "dy"))

    def loss(x, w1, w2):
        total = 0.0
        for g, (s, t) in enumerate(G.bounds(e.ends, e.T)):
            total += float((np.maximum(x[s:t] @ w1[g].T, 0) ** 2 @ w2[g].T * dy[s:t]).sum())
        return total

    rng = rng_of(9)
    for name, at, grad in (("x", 0, e.dx), ("w1", 1, e.dw1), ("w2", 2, e.dw2)):
        p = [x, w1, w2]
        d = rng.standard_normal(p[at].shape)
        up, down = list(p), list(p)
        up[at], down[at] = p[at] + 1e-5 * d, p[at] - 1e-5 * d
        diff = (loss(*up) - loss(*down)) / 2e-5
        got = float((R.f64(grad) * d).sum())
        # h, a, da and dh are rounded to bf16 on the way: each of the terms that the sum adds is off by
        # at most six half steps, independently and of either sign
        size = np.sqrt(((R.f64(grad) * d) ** 2).sum())
        assert abs(got - diff) <= 6 * 2.0 ** -8 * size * 4, (name, got, diff, size)


@pytest.mark.parametrize("T", [24, 900])
def test_captured_step_follows_the_ends(T):
    """A captured step replays with other ends and inputs, eager work in between."""
    e = Experts(T, 256, 384, [T // 3, T // 3, T - 3], 3)
    e.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e.step()
    other = Experts(T, 256, 384, [1, 2, T], 4)
    for ends in ([0, T, T], [T // 2, T // 2 + 1, T - 1], [T // 3, T // 3, T - 3]):
        e.ends = ends
        e.end.copy_(ends_of(ends))
        for k in e.OUT:
            getattr(e, k).zero_()
        other.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        e.check()


def test_two_streams_at_once():
    es = [Experts(200 + 50 * i, 256, 384, [50, 90, 180], 10 + i) for i in range(3)]
    streams = [torch.cuda.Stream() for _ in es]
    torch.cuda.synchronize()
    for _ in range(3):
        for e, s in zip(es, streams):
            with torch.cuda.stream(s):
                e.step()
    torch.cuda.synchronize()
    for e in es:
        e.check()


@pytest.mark.parametrize("T", [20, 333])
def test_served_experts(T):
    """A serving step: rows quantised to MXFP4, two grouped products with a quantisation between them."""
    D, F, n = 256, 512, 4
    rng = rng_of(T, 7)
    ends = [T // 4, T // 4, T - 2, T - 1]
    x = torch.from_numpy(rng.standard_normal((T, D))).bfloat16().cuda()
    s = torch.cuda.current_stream()

    def quantized(v):
        M, K = v.shape
        Q = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
        S = torch.full((K // 32, G.up(M, 16)), 255, dtype=torch.uint8, device="cuda")
        ok(lsm.gemm_mxfp4_quantize_run(H.handle(), v, Q, S, M, K, v.stride(0), K, S.stride(0), 0, lsm.GEMM_MXFP4_BF16, s),
           "quantize")
        return Q, S

    def back(Q, S):
        return G.values(G.unpack(Q.cpu().numpy()), S[:, :Q.shape[0]].cpu().numpy().T)

    def layer(v, w, N):
        Q, S = quantized(v)
        ws = [quantized(m) for m in w]
        B, SB = torch.stack([q for q, _ in ws]), torch.stack([c for _, c in ws])
        C = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
        K = v.shape[1]
        ok(lsm.gemm_grouped_mxfp4_run(H.handle(), Q, B, C, S, SB, ends_of(ends), n, T, N, K, K, K, N * K, N, S.stride(0),
                                      SB.stride(1), SB.stride(0), lsm.GEMM_MXFP4_BF16, s), "gemm_grouped_mxfp4_run")
        a = back(Q, S)
        for g, (f, l) in enumerate(G.bounds(ends, T)):
            ref, bound = G.product(a[f:l], back(*ws[g]))
            R.assert_within(R.f64(C)[f:l], ref, bound + 2.0 ** -8 * (np.abs(ref) + bound), f"group {g}")
        assert bool((C[T - 1:] == 0).all())
        return C

    w1 = torch.from_numpy(rng.standard_normal((n, F, D)) / 16).bfloat16().cuda()
    w2 = torch.from_numpy(rng.standard_normal((n, D, F)) / 22).bfloat16().cuda()
    layer(torch.relu(layer(x, w1, F)), w2, D)
