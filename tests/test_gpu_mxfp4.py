"""MXFP4 on the GPU: gemm_mxfp4_quantize_run and gemm_mxfp4_dequantize_run bit for bit, and
gemm_mxfp4_run against fp64 (grouped_reference.py)."""
import numpy as np
import pytest
import torch

import gpu_harness as H
import grouped_reference as G
import lds_staged_matrix_amd as lsm
import linear_reference as R

pytestmark = pytest.mark.gpu

DTYPE = {"bf16": lsm.GEMM_MXFP4_BF16, "f16": lsm.GEMM_MXFP4_F16, "f32": lsm.GEMM_MXFP4_F32}
LAYOUT = {"K": lsm.GEMM_K_CONTIG, "MN": lsm.GEMM_MN_CONTIG}
CANARY = 0x5A


def rng_of(*key):
    return np.random.default_rng([k if isinstance(k, int) else sum(map(ord, k)) for k in key])


def ok(st, what):
    if st != lsm.GEMM_OK:
        raise lsm.GemmError(st, what)
    torch.cuda.synchronize()


def device(values, pitch, kind, shift=0):
    """values (fp64, 2-d) in rows of `pitch` elements from element `shift` on, NaN around them."""
    rows, cols = values.shape
    t = R.TORCH[kind]
    buf = torch.full((shift + rows * pitch + 16,), float("nan")).to(t).cuda()
    v = buf[shift:shift + rows * pitch].view(rows, pitch)[:, :cols]
    v.copy_(torch.from_numpy(np.ascontiguousarray(values)).to(t if kind != "f32" else torch.float32))
    return v


def raw(rows, pitch, fill=CANARY):
    """`rows` rows of `pitch` bytes, 64 more on either side."""
    buf = torch.full((128 + rows * pitch,), fill, dtype=torch.uint8, device="cuda")
    return buf, buf[64:64 + rows * pitch].view(rows, pitch)


def untouched(buf, rows, pitch, cols):
    keep = torch.ones(buf.numel(), dtype=torch.bool)
    keep[64:64 + rows * pitch].view(rows, pitch)[:, :cols] = False
    return bool((buf.cpu()[keep] == CANARY).all())


# --------------------------------------------------------------- conversions

def check_quantize(x, kind, layout, shift=0):
    """x: fp64 values, exact in `kind`."""
    M, K = x.shape
    inner = K if layout == "K" else M
    pitch, ldq, lds = inner + 3, G.up(K, 32) + 32, G.up(M, 16) + 16
    X = device(x if layout == "K" else x.T, pitch, kind, shift)
    qbuf, Q = raw(M, ldq // 2)
    sbuf, S = raw(K // 32, lds)
    ybuf = torch.full((M * (K + 5) + 8,), 7.0, dtype=R.TORCH[kind], device="cuda")
    Y = ybuf[:M * (K + 5)].view(M, K + 5)
    print("CASE quantize", M, K, kind, layout, shift, flush=True)
    ok(lsm.gemm_mxfp4_quantize_run(H.handle(), X, Q, S, M, K, pitch, ldq, lds, LAYOUT[layout], DTYPE[kind],
                                   torch.cuda.current_stream()), "quantize")
    ok(lsm.gemm_mxfp4_dequantize_run(H.handle(), Q, S, Y, M, K, ldq, lds, K + 5, DTYPE[kind],
                                     torch.cuda.current_stream()), "dequantize")
    code, scale = G.quantize(x)
    got_s = S[:, :M].cpu().numpy().T
    assert np.array_equal(got_s, scale)
    got = G.unpack(Q[:, :K // 2].cpu().numpy())
    bad = np.nonzero(got != code)
    assert not bad[0].size, (bad[0][0], bad[1][0], x[bad][0], got[bad][0], code[bad][0])
    assert untouched(qbuf, M, ldq // 2, K // 2) and untouched(sbuf, K // 32, lds, M)
    with np.errstate(over="ignore"):
        want = R.round_to(G.values(code, scale), kind)
    assert np.array_equal(R.f64(Y[:, :K]), want, equal_nan=True)
    assert bool((Y[:, K:] == 7).all()) and bool((ybuf[M * (K + 5):] == 7).all())


SIZES = [(1, 32), (1, 512), (1, 4096), (2, 96), (15, 544), (16, 512), (17, 1056), (63, 64), (64, 2048), (65, 160),
         (300, 1152), (1500, 896)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("kind", sorted(DTYPE))
@pytest.mark.parametrize("layout", sorted(LAYOUT))
def test_quantize_sizes(M, K, kind, layout):
    rng = rng_of(M, K, kind)
    x = rng.standard_normal((M, K)) * np.exp2(rng.integers(-10, 6, (M, K // 32))).repeat(32, 1)
    check_quantize(R.round_to(x, kind), kind, layout, shift=M % 3)


@pytest.mark.parametrize("kind", sorted(DTYPE))
@pytest.mark.parametrize("layout", sorted(LAYOUT))
def test_quantize_borders(kind, layout):
    """Every tie and its neighbours under a block maximum of 4, 6, just below 8 and 8."""
    eps = float(torch.finfo(R.TORCH[kind]).eps)
    mids = (G.E2M1[1:] + G.E2M1[:-1]) / 2
    pts = np.concatenate([G.E2M1, mids, mids * (1 + eps), mids * (1 - eps / 2), [5.5, 7, 7.5]])
    pts = np.concatenate([pts, -pts])
    rows = []
    for top in (4.0, 6.0, 8 * (1 - eps / 2), 8.0):
        row = np.zeros(96)
        row[:pts.size] = np.where(np.abs(pts) <= top, pts, 0)
        row[::32] = top
        rows.append(row)
    x = np.stack(rows)
    for scale in (1.0, 2.0 ** -9, 2.0 ** 7):
        check_quantize(R.round_to(x * scale, kind), kind, layout)


@pytest.mark.parametrize("kind", sorted(DTYPE))
@pytest.mark.parametrize("layout", sorted(LAYOUT))
def test_quantize_extremes(kind, layout):
    """Zeros, negative zeros, the smallest and largest numbers, infinities and NaNs; none spreads beyond its block."""
    f = torch.finfo(R.TORCH[kind])
    x = np.zeros((8, 128))
    x[0, 5] = -0.0
    x[1, :4] = f.smallest_normal, f.tiny, -f.tiny * 0.75, f.tiny * 0.5
    x[1, 32:36] = 2.0 ** -126, 2.0 ** -127, 2.0 ** -133, -2.0 ** -130
    x[2, :3] = f.max, -f.max, f.max / 2
    x[3, 40] = np.inf
    x[3, 41] = 3
    x[4, 70] = -np.inf
    x[5, 10] = np.nan
    x[5, 96:] = 1.5
    x[6] = 1
    x[7, :64] = -0.25
    check_quantize(R.round_to(x, kind), kind, layout)


def test_round_trip_in_every_scale():
    """All 16 codes under all 256 scales back to fp32, bf16 and fp16."""
    code = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    scale = np.arange(256, dtype=np.uint8)[:, None]
    Q = torch.from_numpy(G.pack(code)).cuda()
    S = torch.from_numpy(np.ascontiguousarray(scale.T)).cuda()
    for kind in DTYPE:
        Y = torch.zeros(256, 32, dtype=R.TORCH[kind], device="cuda")
        ok(lsm.gemm_mxfp4_dequantize_run(H.handle(), Q, S, Y, 256, 32, 32, 256, 32, DTYPE[kind],
                                         torch.cuda.current_stream()), "dequantize")
        with np.errstate(over="ignore"):
            want = R.round_to(G.values(code, scale), kind)
        assert np.array_equal(R.f64(Y), want, equal_nan=True), kind


def test_quantize_beyond_32_bits():
    """2^31 elements and more: the last rows of a tall matrix."""
    M, K = (1 << 25) + 5, 64
    X = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    X[-1] = 3.0
    X[-2, 32:] = -0.75
    Q = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
    lds = G.up(M, 16)
    S = torch.zeros(K // 32, lds, dtype=torch.uint8, device="cuda")
    Y = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    ok(lsm.gemm_mxfp4_quantize_run(H.handle(), X, Q, S, M, K, K, K, lds, lsm.GEMM_K_CONTIG, lsm.GEMM_MXFP4_BF16,
                                   torch.cuda.current_stream()), "quantize")
    ok(lsm.gemm_mxfp4_dequantize_run(H.handle(), Q, S, Y, M, K, K, lds, K, lsm.GEMM_MXFP4_BF16,
                                     torch.cuda.current_stream()), "dequantize")
    assert torch.equal(X, Y)
    assert bool((S[:, M:] == 0).all())


# ------------------------------------------------------------------ product

def mx_operand(code, scale, shift_rows=0):
    """Device arrays of codes and scales, their padding filled with NaN scales and codes of 6."""
    M, K = code.shape
    ldq, lds = G.up(K, 32) + 32, G.up(M, 16) + 16
    Q = torch.full((M, ldq // 2), 0x77, dtype=torch.uint8, device="cuda")
    Q[:, :K // 2] = torch.from_numpy(G.pack(code)).cuda()
    S = torch.full((max(K // 32, 1), lds), G.NAN_SCALE, dtype=torch.uint8, device="cuda")
    if K:
        S[:K // 32, :M] = torch.from_numpy(np.ascontiguousarray(scale.T)).cuda()
    return Q, S, ldq, lds


def operand(rng, M, K, dist):
    if dist == "exact":            # products and sums of multiples of 2^-4 below 2^20: exact in fp32
        code = rng.integers(0, 16, (M, K), dtype=np.uint8)
        return code, rng.integers(126, 129, (M, K // 32)).astype(np.uint8)
    if dist == "wide":
        code = rng.integers(0, 16, (M, K), dtype=np.uint8)
        return code, rng.integers(107, 147, (M, K // 32)).astype(np.uint8)
    return G.quantize(rng.standard_normal((M, K)) * (1 + 20 * (rng.random(K) > 0.97)))


def check_product(M, N, K, out, dist, pad=3, shift=0):
    rng = rng_of(M, N, K, out, dist)
    ca, sa = operand(rng, M, K, dist)
    cb, sb = operand(rng, N, K, dist)
    A, SA, lda, ldsa = mx_operand(ca, sa)
    B, SB, ldb, ldsb = mx_operand(cb, sb)
    t = R.TORCH[out]
    ldc = N + pad
    buf = torch.full((shift + M * ldc + 64,), -99.0, dtype=t, device="cuda")
    C = buf[shift:shift + M * ldc].view(M, ldc)
    print("CASE mxfp4", M, N, K, out, dist, flush=True)
    ok(lsm.gemm_mxfp4_run(H.handle(), A, B, C, SA, SB, M, N, K, lda, ldb, ldc, ldsa, ldsb, DTYPE[out],
                          torch.cuda.current_stream()), "gemm_mxfp4_run")
    assert bool((buf[:shift] == -99).all()) and bool((buf[shift + M * ldc:] == -99).all())
    assert bool((C[:, N:] == -99).all())
    ref, bound = G.product(G.values(ca, sa), G.values(cb, sb))
    got = R.f64(C[:, :N])
    what = f"mxfp4 {M}x{N}x{K} {out} {dist}"
    if dist == "exact":
        assert np.array_equal(got, R.round_to(ref, out)), what
    else:
        R.assert_within(got, ref, bound + R.HALF_STEP[out] * (np.abs(ref) + bound) + R.SMALLEST[out], what)


# every kernel: streams of 16, 32 and 64 columns, up to 16 rows and more, tiles that share K (32 x 64, 64 x 64, 64 x 128),
# 256 x 256 tiles, whole and in parts; whole tiles and cut ones, K of one block, of part of a K tile, of many
PRODUCTS = [(1, 1, 32), (1, 4096, 4096), (3, 37, 64), (16, 130, 544), (7, 9000, 1056), (16, 8200, 2080), (5, 16400, 96),
            (17, 40, 96), (32, 1100, 4128), (20, 16400, 96), (33, 64, 288), (100, 65, 32), (64, 64, 256), (250, 300, 1312),
            (700, 1000, 416), (1500, 1152, 896), (2049, 2100, 320), (2048, 2048, 512), (2048, 2048, 256), (4100, 4097, 288),
            (4096, 4096, 544), (6169, 904, 64), (7670, 72, 864), (355, 5472, 1088), (33, 19152, 2304),
            (7967, 400, 1664), (3, 32800, 288)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("out", sorted(DTYPE))
def test_product_exact(M, N, K, out):
    check_product(M, N, K, out, "exact", pad=M % 2 * 3, shift=N % 3)


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("dist", ["normal", "wide"])
def test_product_real(M, N, K, dist):
    check_product(M, N, K, "f32", dist)


@pytest.mark.parametrize("M,N,K", [(5, 70, 4096), (40, 70, 4096), (300, 400, 1024)])
@pytest.mark.parametrize("out", ["bf16", "f16"])
def test_product_rounds_once(M, N, K, out):
    check_product(M, N, K, out, "normal")


@pytest.mark.parametrize("M,N", [(3, 50), (20, 50), (100, 100), (2048, 2100), (4200, 4200)])
def test_nan_scales_stay_in_their_rows(M, N):
    K = 320
    rng = rng_of(M, N)
    ca, sa = operand(rng, M, K, "exact")
    cb, sb = operand(rng, N, K, "exact")
    sa[M // 2, 3] = G.NAN_SCALE
    sb[N - 1, 9] = G.NAN_SCALE
    A, SA, lda, ldsa = mx_operand(ca, sa)
    B, SB, ldb, ldsb = mx_operand(cb, sb)
    C = torch.zeros(M, N, device="cuda")
    ok(lsm.gemm_mxfp4_run(H.handle(), A, B, C, SA, SB, M, N, K, lda, ldb, N, ldsa, ldsb, lsm.GEMM_MXFP4_F32,
                          torch.cuda.current_stream()), "gemm_mxfp4_run")
    nan = np.isnan(R.f64(C))
    want = np.zeros((M, N), bool)
    want[M // 2] = True
    want[:, N - 1] = True
    assert np.array_equal(nan, want)
    ref, _ = G.product(G.values(ca, sa), G.values(cb, sb))
    assert np.array_equal(R.f64(C)[~nan], ref[~nan])


@pytest.mark.parametrize("M,N", [(2, 40), (30, 40), (90, 300), (4100, 4100)])
def test_empty_sum(M, N):
    C = torch.full((M, N + 1), 5.0, device="cuda")
    ok(lsm.gemm_mxfp4_run(H.handle(), None, None, C, None, None, M, N, 0, 0, 0, N + 1, 0, 0, lsm.GEMM_MXFP4_F32,
                          torch.cuda.current_stream()), "gemm_mxfp4_run")
    assert bool((C[:, :N] == 0).all()) and bool((C[:, N] == 5).all())
