"""The linear-layer operators where values meet the ends of their types' ranges,
against the fp64 definitions of linear_reference.py."""
import numpy as np
import pytest
import torch

import gpu_harness as H
import lds_staged_matrix_amd as lsm
import linear_reference as R
import test_gpu_linear as T

pytestmark = pytest.mark.gpu

# rows by waves, one, two and four chunks a thread, rows read twice (with and without whole chunks)
NORM_LENGTHS = [256, 1031, 16384, 20000, 40003, 5]


def norm(x, w, eps, kind, out):
    """(Y, S) in fp64."""
    M, N = x.shape
    X, W = T.padded(x, N, kind), T.padded(w, N, kind)
    Y, S = T.Out(M, N, N, out), T.Out(1, M, M, "f32")
    print("CASE norm range", M, N, kind, out, eps, flush=True)
    T.ok(lsm.gemm_rmsnorm_run(H.handle(), X, None, W, None, Y.view, S.view, M, N, N, 0, 0, N, eps,
                              T.NORM[kind, out], torch.cuda.current_stream()), "gemm_rmsnorm_run")
    Y.check("Y")
    S.check("S")
    return R.f64(Y.view), R.f64(S.view)[0]


@pytest.mark.parametrize("N", NORM_LENGTHS)
@pytest.mark.parametrize("rows,weight,eps", [((1e15, 1e10, 1.0), 3e24, 1e-5), ((1e-18, 1e-10, 1.0), 1e-28, 0.0),
                                             ((1e-18, 1e-10, 1.0), 1e-25, 0.0)])
def test_norm_whose_products_leave_the_range(N, rows, weight, eps):
    """h w overflows or is subnormal, or vanishes, in some rows; y = h w / root is an ordinary number in all."""
    rng = np.random.default_rng(N)
    x = R.round_to(rng.standard_normal((len(rows), N)) * np.array(rows)[:, None], "bf16")
    w = R.round_to((1 + 0.25 * rng.standard_normal((1, N))) * weight, "bf16")
    _, y = R.rmsnorm(x, None, w, eps)
    for out in ("e4m3", "bf16"):
        Y, S = norm(x, w, eps, "bf16", out)
        T.check_norm(len(rows), N, "bf16", out, (None, y, None, Y, S))


@pytest.mark.parametrize("N", NORM_LENGTHS)
def test_norm_whose_squares_overflow(N):
    """Rows of finite values whose squares' sum overflows fp32 give zeros, whatever h w does; the others
    are untouched."""
    x = np.ones((4, N))
    x[0], x[1], x[2, N - 1] = 3e38, 1e20, -3e38
    x, w = R.round_to(x, "bf16"), np.full((1, N), 2.0)
    for out in ("e4m3", "bf16"):
        Y, S = norm(x, w, 1e-5, "bf16", out)
        assert (Y[:3] == 0).all()
        if out == "e4m3":
            assert (S[:3] == np.float32(2.0 ** -100) / np.float32(448)).all()
        _, y = R.rmsnorm(x[3:], None, w, 1e-5)
        T.check_norm(1, N, "bf16", out, (None, y, None, Y[3:], S[3:]))


@pytest.mark.parametrize("M,N", [(1, 40), (20, 40), (40, 4200)])
def test_w4_terms_beyond_the_range(M, N):
    """Entries whose factors or partial sums overflow fp32 where the formula's sum does not: a scale so
    large that (q - z) s overflows beside activations that are zero or tiny, and large terms that cancel."""
    K, group = 64, 32
    q, z, s, a = np.full((N, K), 15), np.full((2, N), 3.0), np.ones((2, N)), np.zeros((M, K))
    s[0] = 2.0 ** 125                              # 12 * 2^125 is beyond fp32
    a[:, 1], a[:, 40] = -2.0 ** -60, np.inf
    got = T.run_w4(a, q, s, z, group, "bf16", "f32")
    assert (got == np.inf).all()

    s[0], a[:, 1], a[:, 40] = 1.0, 0.0, 0.0
    z[1], q[:, 33], q[:, 34], q[:, 35] = 8, 13, 3, 9
    a[:, 33:36] = 2.0 ** 127, 2.0 ** 127, 3.0      # 5 * 2^127 - 5 * 2^127 + 3
    got = T.run_w4(a, q, s, z, group, "bf16", "f32")
    assert (got == 3.0).all()


@pytest.mark.parametrize("kind,out", sorted(T.W4))
@pytest.mark.parametrize("M", [1, 16, 20, 48])
@pytest.mark.parametrize("data", ["biased", "loud"])
def test_w4_activations_with_a_mean_and_with_outliers(kind, out, M, data):
    """The header's bound where the zero point's correction cancels most: activations far from zero in
    the mean, and outliers that meet weights of zero (q = z)."""
    N, K, group = 272, 4096, 128
    rng = np.random.default_rng([M, len(data)])
    a = rng.standard_normal((M, K)) + (2 if data == "biased" else 0)
    q, z = rng.integers(0, 16, (N, K)), rng.integers(0, 16, (K // group, N)).astype(np.float64)
    s = R.round_to((0.5 + rng.random(z.shape)) / 64, kind)
    if data == "loud":
        for k in range(5, K, 500):
            a[:, k], q[:, k] = 1e4, z[k // group]
    a = R.round_to(a, kind)
    got = T.run_w4(a, q, s, z, group, kind, out)
    ref, bound = R.w4(a, q, s, z, group)
    R.assert_within(got, ref, bound + (bound + np.abs(ref)) * R.HALF_STEP[out] + R.SMALLEST[out], "w4 " + data)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N", [(1, 40), (5, 40), (5, 4100), (20, 40), (20, 4100), (20, 8200), (48, 40), (48, 4100),
                                 (48, 8200)])
def test_w4_zero_points_of_every_byte(kind, group, M, N):
    """Zero points from 0 to 255, in one, two and four blocks of columns."""
    K = 288
    a, q, s, _ = T.w4_inputs(M, N, K, group, kind, True, "int")
    z = np.random.default_rng([M, N, group]).integers(0, 256, s.shape).astype(np.float64)
    # |a| <= 2, 16 + q <= 31, 16 + z <= 271 and s >= 1/4: sums below 2^24 in units of 1/4
    assert 2 * (31 + 271) * 4 * K < 1 << 24
    got = T.run_w4(a, q, s, z, group, kind, "f32")
    assert np.array_equal(got, R.w4(a, q, s, z, group)[0])


@pytest.mark.parametrize("M", [1, 3, 8, 9, 16, 17, 32, 33, 48, 49, 64])
@pytest.mark.parametrize("N,K", [(33, 48), (200, 1040), (4099, 272), (8208, 144)])
def test_scaled_few_rows_fp16(M, N, K):
    for dist in ("int", "real"):
        T.check_scaled(M, N, K, T.KC, T.KC, "f16", dist, extra=N % 3)
