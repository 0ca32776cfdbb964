"""gemm_rmsnorm_run, gemm_scaled_run and gemm_w4_run on the GPU against their
fp64 definitions (linear_reference.py).

Integer-valued inputs with power-of-two scales make every product and sum
exact, so the outputs have to be equal bit for bit; real-valued ones are held
to the error bounds that linear_reference.py derives.  Buffers are padded, the
padding of inputs holds NaN and that of outputs a canary.
"""
import numpy as np
import pytest
import torch

import lds_staged_matrix_amd as lsm
import linear_reference as R
import gpu_harness as H

pytestmark = pytest.mark.gpu

FP8 = torch.float8_e4m3fn
KC, MNC = lsm.GEMM_K_CONTIG, lsm.GEMM_MN_CONTIG
NORM = {("bf16", "bf16"): lsm.GEMM_NORM_BF16_BF16, ("bf16", "e4m3"): lsm.GEMM_NORM_BF16_E4M3,
        ("f16", "f16"): lsm.GEMM_NORM_F16_F16, ("f16", "e4m3"): lsm.GEMM_NORM_F16_E4M3}
SCALED = {"f32": lsm.GEMM_E4M3_F32, "bf16": lsm.GEMM_E4M3_BF16, "f16": lsm.GEMM_E4M3_F16}
W4 = {("bf16", "f32"): lsm.GEMM_BF16_F32, ("bf16", "bf16"): lsm.GEMM_BF16_BF16,
      ("f16", "f16"): lsm.GEMM_F16_F16, ("f16", "f32"): lsm.GEMM_F16_F32}
NAN = float("nan")


def up(n, q):
    return -(-max(n, 1) // q) * q


def rng_of(*key):
    return np.random.default_rng([abs(hash(k)) % (1 << 31) if not isinstance(k, int) else k for k in key])


def padded(values, pitch, kind, fill=NAN, rows=0, shift=0):
    """values (2-d, fp64) in a device buffer of `pitch` elements a row, `shift`
    elements from its start, with `fill` around them; returns the M x N view."""
    M, N = values.shape
    flat = torch.full((shift + (M + rows) * pitch + 16,), fill, dtype=torch.float32)
    buf = flat.to(R.TORCH[kind]).cuda()
    v = buf[shift:shift + M * pitch].view(M, pitch)[:, :N]
    v.copy_(torch.from_numpy(np.ascontiguousarray(values)).float().to(R.TORCH[kind]).cuda())
    return v


class Out:
    """An output buffer: an M x N view of `pitch` a row between canaries."""
    CANARY = 0x5A

    def __init__(self, M, N, pitch, kind, shift=0):
        self.M, self.N, self.pitch, self.shift = M, N, pitch, shift
        t = R.TORCH[kind]
        self.size = torch.empty(0, dtype=t).element_size()
        n = (shift + M * pitch + 64) * self.size
        self.raw = torch.full((n,), self.CANARY, dtype=torch.uint8, device="cuda")
        self.view = self.raw.view(t)[shift:shift + M * pitch].view(M, pitch)[:, :N]

    def check(self, what):
        keep = torch.ones(self.raw.numel(), dtype=torch.bool)
        body = keep[self.shift * self.size:(self.shift + self.M * self.pitch) * self.size]
        body.view(self.M, self.pitch * self.size)[:, :self.N * self.size] = False
        assert bool((self.raw.cpu()[keep] == self.CANARY).all()), f"{what}: written outside the M x N block"


def ok(st, what):
    if st != lsm.GEMM_OK:
        raise lsm.GemmError(st, what)
    torch.cuda.synchronize()


# ------------------------------------------------------------------- norm

def run_norm(M, N, kind, out, residual, keep_h, pad=16, shift=0, eps=1e-5, x=None, seed=0):
    rng = rng_of(M, N, seed, 1)
    x = R.round_to(rng.standard_normal((M, N)) * (1 + 20 * (rng.random(N) > 0.98)) if x is None else x, kind)
    r = R.round_to(rng.standard_normal((M, N)) * 2, kind) if residual else None
    w = R.round_to(1 + 0.25 * rng.standard_normal((1, N)), kind)
    pitch = up(N, pad) + (pad if pad > 1 else 3)
    X = padded(x, pitch, kind, shift=shift)
    Rr = padded(r, pitch + pad, kind, shift=shift) if residual else None
    W = padded(w, N, kind, shift=shift)
    Y, S = Out(M, N, pitch, out, shift), Out(1, M, M, "f32")
    Hh = Out(M, N, pitch, kind, shift) if keep_h else None
    print("CASE norm", M, N, kind, out, residual, keep_h, pad, shift, flush=True)
    ok(lsm.gemm_rmsnorm_run(H.handle(), X, Rr, W, Hh.view if Hh else None, Y.view, S.view if out == "e4m3" else None,
                            M, N, pitch, pitch + pad if residual else 0, pitch if Hh else 0, pitch, eps,
                            NORM[kind, out], torch.cuda.current_stream()), "gemm_rmsnorm_run")
    Y.check("Y")
    S.check("S")
    if Hh:
        Hh.check("H")
    h, y = R.rmsnorm(x, r, w, eps)
    return h, y, (R.f64(Hh.view) if Hh else None), R.f64(Y.view), R.f64(S.view)[0]


def check_norm(M, N, kind, out, result):
    h, y, H_, Y, S = result
    what = f"norm {M}x{N} {kind}->{out}"
    slack = R.rmsnorm_slack(N)
    if H_ is not None:
        R.assert_rounded(H_, h, 2.0 ** -24, kind, what + " H")
    if out == "e4m3":
        s = R.row_scale(y)
        R.assert_within(S, s, slack * s, what + " S")
        R.assert_rounded(Y, y / s[:, None], 2 * slack, "e4m3", what + " Y")
    else:
        R.assert_rounded(Y, y, slack, kind, what + " Y")


NORM_SIZES = [(1, 1), (1, 8), (3, 7), (5, 64), (4, 65), (9, 511), (2, 520), (7, 1024), (5, 1151), (3, 2048),
              (2, 2056), (1, 4096), (3, 4100), (2, 8192), (2, 8200), (1, 16384), (2, 20000), (1, 32768), (2, 33000),
              (1, 70001)]


@pytest.mark.parametrize("M,N", NORM_SIZES)
@pytest.mark.parametrize("kind,out", sorted(NORM))
def test_norm_sizes(M, N, kind, out):
    for residual in (True, False):
        check_norm(M, N, kind, out, run_norm(M, N, kind, out, residual, keep_h=residual))


@pytest.mark.parametrize("M,N", [(3, 1), (5, 63), (2, 513), (3, 1151), (2, 5000), (1, 9001), (2, 17001), (2, 33003)])
@pytest.mark.parametrize("out", ["f16", "e4m3"])
@pytest.mark.parametrize("pad,shift", [(1, 0), (8, 1)])
def test_norm_unaligned_rows(M, N, out, pad, shift):
    check_norm(M, N, "f16", out, run_norm(M, N, "f16", out, True, True, pad=pad, shift=shift))


@pytest.mark.parametrize("M", [1, 4, 5, 257, 1500])
def test_norm_many_rows(M):
    check_norm(M, 384, "bf16", "e4m3", run_norm(M, 384, "bf16", "e4m3", True, True))


def test_norm_more_rows_than_one_grid_dimension_holds():
    M = (1 << 26) + 3                    # of 64 threads each
    X = torch.full((M, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    X[-1] = 0
    W = torch.ones(1, dtype=torch.bfloat16, device="cuda")
    Y, S = torch.zeros(M, 1, dtype=FP8, device="cuda"), torch.zeros(M, device="cuda")
    print("CASE norm rows", M, flush=True)
    ok(lsm.gemm_rmsnorm_run(H.handle(), X, None, W, None, Y, S, M, 1, 1, 0, 0, 1, 0.0, lsm.GEMM_NORM_BF16_E4M3,
                            torch.cuda.current_stream()), "gemm_rmsnorm_run")
    # 448 is the byte 0x7E; a row of zeros with eps 0 has no root
    assert int((Y.view(torch.uint8)[:-1] != 0x7E).sum()) == 0 and bool(S[:-1].eq(1 / 448).all())
    assert bool(S[-1].isnan()) and int(Y.view(torch.uint8)[-1]) & 0x7F == 0x7F


def test_norm_h_without_residual_and_residual_without_h():
    check_norm(4, 640, "bf16", "bf16", run_norm(4, 640, "bf16", "bf16", False, True))
    check_norm(4, 640, "bf16", "e4m3", run_norm(4, 640, "bf16", "e4m3", True, False))


@pytest.mark.parametrize("N", [256, 1024, 40000])
def test_norm_special_rows(N):
    """All-zero rows, the smallest and largest normal values, and rows with a
    NaN or an infinity, beside ordinary rows."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((8, N))
    x[1] = 0
    x[2] *= 1e-20
    x[3] *= 1e15
    x[4, N // 2] = np.nan
    x[5, N - 1] = np.inf
    x[6] = 0
    x[6, 3] = 2.0
    h, y, _, Y, S = run_norm(8, N, "bf16", "e4m3", False, False, x=x)
    assert np.isnan(S[4]) and np.isnan(Y[4]).all()
    assert np.isnan(S[5]) and np.isnan(Y[5]).all()
    fine = [0, 1, 2, 3, 6, 7]
    check_norm(8, N, "bf16", "e4m3", (h[fine], y[fine], None, Y[fine], S[fine]))
    assert (Y[1] == 0).all() and S[1] == np.float32(2.0 ** -100) / np.float32(448)
    assert Y[6, 3] == 448
    h, y, _, Y, _ = run_norm(8, N, "bf16", "bf16", False, False, x=x)
    assert np.isnan(Y[4]).all() and np.isnan(Y[5, N - 1]) and (Y[5, :N - 1] == 0).all()
    check_norm(8, N, "bf16", "bf16", (h[fine], y[fine], None, Y[fine], None))


def test_norm_zero_eps():
    x = np.ones((2, 96))
    h, y, _, Y, _ = run_norm(2, 96, "f16", "f16", False, False, x=x, eps=0.0)
    check_norm(2, 96, "f16", "f16", (h, y, None, Y, None))


@pytest.mark.parametrize("N", [5, 9, 500, 520, 1151, 4096, 9001, 33000, 33003])
@pytest.mark.parametrize("into", ["X", "R"])
def test_norm_in_place(N, into):
    """H in the residual's or the input's place, Y in the other's."""
    rng = np.random.default_rng(9)
    x, r = (R.round_to(rng.standard_normal((3, N)), "bf16") for _ in range(2))
    w = R.round_to(1 + 0.1 * rng.standard_normal((1, N)), "bf16")
    X, Rr, W = padded(x, up(N, 8), "bf16"), padded(r, up(N, 8), "bf16"), padded(w, N, "bf16")
    hh, yy = (X, Rr) if into == "X" else (Rr, X)
    print("CASE norm in place", N, into, flush=True)
    ld = X.stride(0)
    ok(lsm.gemm_rmsnorm_run(H.handle(), X, Rr, W, hh, yy, None, 3, N, ld, ld, ld, ld, 1e-6,
                            lsm.GEMM_NORM_BF16_BF16, torch.cuda.current_stream()), "gemm_rmsnorm_run")
    h, y = R.rmsnorm(x, r, w, 1e-6)
    check_norm(3, N, "bf16", "bf16", (h, y, R.f64(hh), R.f64(yy), None))


# ----------------------------------------------------------------- scaled

def run_scaled(M, N, K, la, lb, out, a, b, sa, sb, incs=(1, 1), extra=0):
    """a (M x K) and b (N x K) in fp64, stored in layouts la, lb."""
    def store(v, layout):
        v = v if layout == KC else v.T
        return padded(v, up(v.shape[1], 16) + 16 * extra, "e4m3")
    A, B = store(a, la), store(b, lb)
    SA, SB = (padded(np.asarray(s, dtype=np.float64)[None], len(s), "f32") for s in (sa, sb))
    C = Out(M, N, N + extra, out)
    print("CASE scaled", M, N, K, la, lb, out, incs, flush=True)
    ok(lsm.gemm_scaled_run(H.handle(), A, B, C.view, SA, SB, M, N, K, A.stride(0), B.stride(0), C.pitch, *incs,
                           la, lb, SCALED[out], torch.cuda.current_stream()), "gemm_scaled_run")
    C.check("C")
    return R.f64(C.view)


def check_scaled(M, N, K, la, lb, out, dist, incs=(1, 1), extra=0):
    rng = rng_of(M, N, K, la, lb)
    if dist == "int":
        a, b = (rng.integers(-2, 3, (m, K)).astype(np.float64) for m in (M, N))
        sa, sb = (2.0 ** rng.integers(-3, 2, m) for m in (M, N))
    else:
        a, b = (R.round_to(rng.standard_normal((m, K)) * 60, "e4m3") for m in (M, N))
        sa, sb = (R.round_to((0.5 + rng.random(m)) * 1e-3, "f32") for m in (M, N))
    sa, sb = (s if i else s[:1] for s, i in zip((sa, sb), incs))
    got = run_scaled(M, N, K, la, lb, out, a, b, sa, sb, incs, extra)
    ref, bound = R.scaled(a, b, np.broadcast_to(sa, M), np.broadcast_to(sb, N), fp8_mfma=out != "f32" and M > 32)
    what = f"scaled {M}x{N}x{K} {la}{lb} {out} {dist}"
    if dist == "int":
        assert np.array_equal(got, R.round_to(ref, out)), what
    else:
        R.assert_within(got, ref, bound + (bound + np.abs(ref)) * R.HALF_STEP[out] + R.SMALLEST[out], what)


LAYOUTS = [(KC, KC), (KC, MNC), (MNC, KC), (MNC, MNC)]


# ping-pong (two of it: 256 tiles and fewer), 128 x 128, 64 x 64 with two and with four stages, split K with up to
# and over 256 tiles (each also cut short in all extents), M <= 32
@pytest.mark.parametrize("M,N,K", [(4112, 4096, 144), (1040, 8208, 144), (2064, 2048, 144), (528, 272, 160), (1040, 2560, 3984),
                                   (512, 512, 8192), (208, 1040, 1040), (1040, 1088, 4112), (32, 1024, 1040)])
@pytest.mark.parametrize("la,lb", LAYOUTS)
@pytest.mark.parametrize("out", sorted(SCALED))
def test_scaled_every_kernel(M, N, K, la, lb, out):
    for dist in ("int", "real"):
        check_scaled(M, N, K, la, lb, out, dist)


@pytest.mark.parametrize("M", [1, 2, 8, 15, 16, 17, 31, 32, 33, 48, 49, 65, 190])
@pytest.mark.parametrize("N,K", [(1, 16), (17, 48), (100, 128), (257, 1040), (4099, 144), (8209, 272), (16400, 160)])
def test_scaled_few_rows(M, N, K):
    for dist in ("int", "real"):
        check_scaled(M, N, K, KC, KC, "f32" if N % 2 else "bf16", dist, extra=N % 3)


@pytest.mark.parametrize("M,N,K", [(260, 1000, 272), (1040, 200, 272), (4100, 47, 144), (250, 2000, 1552), (500, 1001, 2064),
                                   (300, 600, 2048), (60, 8190, 1536)])
@pytest.mark.parametrize("out", sorted(SCALED))
def test_scaled_few_tiles(M, N, K, out):
    """The few-rows kernel with many row tiles, one and two column blocks, cut in all extents."""
    for dist in ("int", "real"):
        check_scaled(M, N, K, KC, KC, out, dist, extra=M % 3)


@pytest.mark.parametrize("M,N", [(201, 333), (1000, 1101)])
@pytest.mark.parametrize("K", [1024, 1152, 1168, 4096, 4112, 4240])
@pytest.mark.parametrize("out", ["f16", "f32"])
def test_scaled_split_k_ragged(M, N, K, out):
    """Steps that do not divide over the groups, cut tiles, rows of C at odd pitches."""
    for extra in (0, 3):
        check_scaled(M, N, K, KC, KC, out, "int", extra=extra)
    check_scaled(M, N, K, KC, KC, out, "real")


@pytest.mark.parametrize("K", [16, 112, 128, 144, 256, 1936, 2048, 4096, 8208])
def test_scaled_few_rows_lengths_of_k(K):
    for M in (3, 20):
        check_scaled(M, 80, K, KC, KC, "f32", "int")


@pytest.mark.parametrize("M,N,K", [(5, 96, 64), (300, 160, 96)])
@pytest.mark.parametrize("incs", [(0, 0), (0, 1), (1, 0)])
def test_scaled_one_scale_for_all(M, N, K, incs):
    for la, lb in LAYOUTS:
        if (la == MNC and M % 16) or (lb == MNC and N % 16):
            continue
        check_scaled(M, N, K, la, lb, "f32", "int", incs=incs)


@pytest.mark.parametrize("M", [7, 100])
def test_scaled_non_finite(M):
    """A NaN in A, an infinite scale and a NaN scale reach their row or column and no other entry."""
    rng = np.random.default_rng(3)
    N, K = 96, 144
    a, b = (rng.integers(-2, 3, (m, K)).astype(np.float64) for m in (M, N))
    sa, sb = np.ones(M), np.ones(N)
    a[2, K - 1], sa[4], sb[5] = np.nan, np.inf, np.nan
    got = run_scaled(M, N, K, KC, KC, "f32", a, b, sa, sb)
    ref, _ = R.scaled(a, b, sa, sb)
    assert np.array_equal(got, ref, equal_nan=True)


@pytest.mark.parametrize("root", [448.0, 64.0, 1.0])
def test_what_the_fp8_mfma_drops(root):
    """root^2 - root^2 + v in one group of eight products: v survives to within
    2^-13 of the power of two under root^2, which is what the bound of 16-bit
    outputs counts on; fp32 outputs keep v exactly."""
    M, N, K = 64, 64, 128
    a, b = np.zeros((M, K)), np.zeros((N, K))
    a[:, 0], b[:, 0] = root, root
    a[:, 5], b[:, 5] = root, -root
    v = 2.0 ** np.arange(8, -9, -1.0)
    a[:len(v), 1], b[:, 1] = v, 1.0
    one = np.ones(64)
    low = 2.0 ** (2 * np.floor(np.log2(root)))
    got = run_scaled(M, N, K, KC, KC, "bf16", a, b, one, one)
    assert (np.abs(got[:len(v)] - v[:, None]) <= low * 2.0 ** -13).all()
    assert np.array_equal(run_scaled(M, N, K, KC, KC, "f32", a, b, one, one), np.repeat(a[:, 1:2], N, 1))


@pytest.mark.parametrize("M", [4, 70])
def test_scaled_empty_sum(M):
    got = run_scaled(M, 48, 0, KC, KC, "f32", np.zeros((M, 0)), np.zeros((48, 0)), np.ones(M), np.ones(48))
    assert (got == 0).all()


# --------------------------------------------------------------------- w4

def run_w4(a, q, s, z, group, kind, out, extra=0):
    M, K = a.shape
    N = q.shape[0]
    A = padded(a, K + 8 * (1 + extra), kind)
    row = K // 2 + 16 * (1 + extra)
    B = torch.full((N, row), 0xFF, dtype=torch.uint8)
    B[:, :K // 2] = torch.from_numpy(R.pack4(q))
    B = B.cuda()
    S = padded(s, N + extra, kind)
    Z = None
    if z is not None:
        Z = torch.full((z.shape[0], N + 1 + extra), 0xFF, dtype=torch.uint8)
        Z[:, :N] = torch.from_numpy(z.astype(np.uint8))
        Z = Z.cuda()
    C = Out(M, N, N + extra, out)
    print("CASE w4", M, N, K, group, kind, out, z is not None, extra, flush=True)
    ok(lsm.gemm_w4_run(H.handle(), A, B, S, Z, C.view, M, N, K, group, A.stride(0), 2 * row, S.stride(0),
                       Z.stride(0) if Z is not None else 0, C.pitch, W4[kind, out],
                       torch.cuda.current_stream()), "gemm_w4_run")
    C.check("C")
    return R.f64(C.view)


def w4_inputs(M, N, K, group, kind, zeros, dist, seed=0):
    rng = rng_of(M, N, K, group, seed)
    G = -(-K // group)
    q = rng.integers(0, 16, (N, K))
    z = rng.integers(0, 16, (G, N)).astype(np.float64) if zeros else None
    if dist == "int":
        a = rng.integers(-2, 3, (M, K)).astype(np.float64)
        s = 2.0 ** rng.integers(-2, 2, (G, N))
    else:
        a = R.round_to(rng.standard_normal((M, K)) + 0.5, kind)
        s = R.round_to((0.5 + rng.random((G, N))) / 16, kind)
    return a, q, s, z


def check_w4(M, N, K, group, kind, out, zeros, dist, extra=0):
    a, q, s, z = w4_inputs(M, N, K, group, kind, zeros, dist)
    got = run_w4(a, q, s, z, group, kind, out, extra)
    ref, bound = R.w4(a, q, s, z, group)
    what = f"w4 {M}x{N}x{K} group {group} {kind}->{out} zeros {zeros} {dist}"
    if dist == "int":
        # |sums| < 2^24 in units of 1/4: every step is exact
        assert 2 * 31 * 2 * 4 * K < 1 << 24
        assert np.array_equal(got, R.round_to(ref, out)), what
    else:
        R.assert_within(got, ref, bound + (bound + np.abs(ref)) * R.HALF_STEP[out] + R.SMALLEST[out], what)


@pytest.mark.parametrize("kind,out", sorted(W4))
@pytest.mark.parametrize("group", [32, 64, 128, 256, 4096])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_groups(kind, out, group, zeros):
    for M in (1, 17, 40):
        for dist in ("int", "real"):
            check_w4(M, 150, 1056, group, kind, out, zeros, dist, extra=M % 3)


@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 32, 33, 48, 64, 65, 130])
@pytest.mark.parametrize("N,K", [(1, 32), (16, 96), (1151, 896), (4100, 160), (8203, 288), (16390, 64)])
def test_w4_sizes(M, N, K):
    for dist in ("int", "real"):
        check_w4(M, N, K, 32 if N % 2 else 64, "bf16", "f32", N % 2 == 0, dist)


@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N", [(3, 4100), (16, 4100), (20, 4090), (20, 4100), (20, 8200), (48, 8260), (64, 4100)])
def test_w4_column_blocks(kind, out, group, M, N):
    """One, two and four blocks of 16 columns to a workgroup, several blocks of k to a wave."""
    for dist in ("int", "real"):
        check_w4(M, N, 1184, group, kind, out, M % 2 == 0, dist)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 256, 512, 1984, 2048, 2080, 4096, 8192])
def test_w4_lengths_of_k(K):
    for M in (1, 20, 64):
        check_w4(M, 48, K, 128, "f16", "f32", True, "int")


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M", [1, 20, 50])
def test_w4_non_finite(kind, M):
    """Infinite, NaN and very large activations and scales give what the definition gives."""
    a, q, s, z = w4_inputs(M, 70, 288, 32, kind, True, "int")
    big = 2.0 ** 127 if kind == "bf16" else 2.0 ** 15
    q[:, 5] = np.arange(70) % 16
    z[0, :] = 3
    a[0, 5] = np.inf
    if M > 1:
        a[1, 200] = np.nan
        a[2, :] = 0
        a[2, 5] = big              # 31 times it overflows bf16's range
        s[0, :] = 2.0 ** -6
        s[3, 9], s[4, 11] = np.inf, np.nan
    got = run_w4(a, q, s, z, 32, kind, "f32")
    ref, _ = R.w4(a, q, s, z, 32)
    with np.errstate(over="ignore"):
        want = R.round_to(ref, "f32")
    assert np.array_equal(got, want, equal_nan=True)


def test_w4_byte_zero_points():
    """Zero points outside 0..15 are legal bytes."""
    a, q, s, z = w4_inputs(5, 40, 128, 64, "bf16", True, "int")
    z[0, :], z[1, 7] = 200, 255
    got = run_w4(a, q, s, z, 64, "bf16", "f32")
    assert np.array_equal(got, R.w4(a, q, s, z, 64)[0])


def test_w4_empty_sum():
    C = Out(3, 40, 40, "f32")
    ok(lsm.gemm_w4_run(H.handle(), None, None, None, None, C.view, 3, 40, 0, 128, 0, 0, 0, 0, 40,
                       lsm.GEMM_BF16_F32, torch.cuda.current_stream()), "gemm_w4_run")
    assert (R.f64(C.view) == 0).all()


# ------------------------------------------------- together, graphs, streams

class Layer:
    """x -> norm -> E4M3 product -> + residual, norm -> 4-bit product, on device buffers."""

    def __init__(self, M, D, F, seed):
        rng = np.random.default_rng(seed)
        self.M, self.D, self.F = M, D, F
        self.x = R.round_to(rng.standard_normal((M, D)), "bf16")
        self.w1, self.w2 = (R.round_to(1 + 0.1 * rng.standard_normal((1, D)), "bf16") for _ in range(2))
        b = rng.standard_normal((D, D)) / np.sqrt(D)
        self.sb = R.round_to(np.abs(b).max(1) / 448, "f32")
        self.b = R.round_to(b / self.sb[:, None], "e4m3")
        self.q = rng.integers(0, 16, (F, D))
        self.s = R.round_to((0.5 + rng.random((D // 64, F))) / 64, "bf16")
        self.z = rng.integers(5, 11, (D // 64, F)).astype(np.float64)
        dev = lambda v, kind: torch.from_numpy(np.ascontiguousarray(v)).float().to(R.TORCH[kind]).cuda()
        self.X, self.W1, self.W2 = dev(self.x, "bf16"), dev(self.w1, "bf16"), dev(self.w2, "bf16")
        self.B, self.SB = dev(self.b, "e4m3"), dev(self.sb, "f32")
        self.Q = torch.from_numpy(R.pack4(self.q)).cuda()
        self.Sc, self.Z = dev(self.s, "bf16"), torch.from_numpy(self.z.astype(np.uint8)).cuda()
        e = lambda *n, t: torch.zeros(*n, dtype=R.TORCH[t], device="cuda")
        self.Y8, self.S8 = e(M, D, t="e4m3"), e(M, t="f32")
        self.P, self.H2, self.Y16, self.C = e(M, D, t="bf16"), e(M, D, t="bf16"), e(M, D, t="bf16"), e(M, F, t="f32")

    def outputs(self):
        return [self.Y8.view(torch.uint8), self.S8, self.P, self.H2, self.Y16, self.C]

    def run(self, stream):
        h, M, D, F = H.handle(), self.M, self.D, self.F
        st = [lsm.gemm_rmsnorm_run(h, self.X, None, self.W1, None, self.Y8, self.S8, M, D, D, 0, 0, D, 1e-5,
                                   lsm.GEMM_NORM_BF16_E4M3, stream),
              lsm.gemm_scaled_run(h, self.Y8, self.B, self.P, self.S8, self.SB, M, D, D, D, D, D, 1, 1, KC, KC,
                                  lsm.GEMM_E4M3_BF16, stream),
              lsm.gemm_rmsnorm_run(h, self.P, self.X, self.W2, self.H2, self.Y16, None, M, D, D, D, D, D, 1e-5,
                                   lsm.GEMM_NORM_BF16_BF16, stream),
              lsm.gemm_w4_run(h, self.Y16, self.Q, self.Sc, self.Z, self.C, M, F, D, 64, D, D, F, F, F,
                              lsm.GEMM_BF16_F32, stream)]
        assert st == [lsm.GEMM_OK] * 4

    def check(self):
        """Every stage against fp64, on what the stage before it wrote."""
        M, D = self.M, self.D
        _, y = R.rmsnorm(self.x, None, self.w1, 1e-5)
        check_norm(M, D, "bf16", "e4m3", (None, y, None, R.f64(self.Y8), R.f64(self.S8)))
        ref, bound = R.scaled(R.f64(self.Y8), self.b, R.f64(self.S8), self.sb, fp8_mfma=M > 32)
        R.assert_within(R.f64(self.P), ref, bound + (bound + np.abs(ref)) * 2.0 ** -8, "layer product")
        h, y = R.rmsnorm(R.f64(self.P), self.x, self.w2, 1e-5)
        check_norm(M, D, "bf16", "bf16", (h, y, R.f64(self.H2), R.f64(self.Y16), None))
        ref, bound = R.w4(R.f64(self.Y16), self.q, self.s, self.z, 64)
        R.assert_within(R.f64(self.C), ref, bound + np.abs(ref) * 2.0 ** -24, "layer 4-bit product")


@pytest.mark.parametrize("M", [1, 24, 130])
def test_layer(M):
    layer = Layer(M, 1024, 1152, M)
    print("CASE layer", M, flush=True)
    layer.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    layer.check()


def test_layers_on_two_streams_at_once():
    layers = [Layer(3, 1024, 640, 1), Layer(40, 512, 1152, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for layer, s in zip(layers, streams):
            layer.run(s)
    torch.cuda.synchronize()
    for layer in layers:
        layer.check()


@pytest.mark.parametrize("M", [1, 40])
def test_layer_in_a_graph(M):
    layer = Layer(M, 1024, 1152, 7)
    layer.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    layer.check()
    eager = [o.clone() for o in layer.outputs()]
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(g, stream=side):
            layer.run(torch.cuda.current_stream())
    torch.cuda.current_stream().wait_stream(side)
    other = Layer(M, 1024, 1152, 8)
    for rep in range(3):
        for o in layer.outputs():
            o.fill_(1)
        other.run(torch.cuda.current_stream())      # eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for o, e in zip(layer.outputs(), eager):
            assert torch.equal(o, e), f"replay {rep}"
    other.check()


def test_results_do_not_depend_on_timing():
    """The same call twice gives the same bits, alone and among other work."""
    layer = Layer(16, 2048, 4096, 11)
    layer.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    first = [o.clone() for o in layer.outputs()]
    s = torch.cuda.Stream()
    other = Layer(33, 1024, 640, 12)
    torch.cuda.synchronize()
    for _ in range(3):
        other.run(s)
        layer.run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for o, e in zip(layer.outputs(), first):
        assert torch.equal(o, e)
