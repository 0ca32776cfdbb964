"""gemm_mxfp4_run and gemm_grouped_mxfp4_run over the whole range of the E8M0 scales, 2^-127 to 2^127, in each
kernel: products of the two scales from 2^-254 to 2^254, of which fp32 holds those between 2^-149 and 2^128.

The header's bound: (K/128 + 8) times 2^-21 of the sum of sizes and 2^-149 more, the smallest step of fp32 for each
of the sums on the way; where the sum of sizes reaches 2^127 sums on the way may overflow, and nothing is said of
the entry.  The second term is needed: of 32 products below 2^-126 in every entry, one in ten is off by more than the
first (by 2^-150)."""
import numpy as np
import pytest
import torch

import gpu_harness as H
import grouped_reference as G
import lds_staged_matrix_amd as lsm
import linear_reference as R
from test_gpu_mxfp4 import DTYPE, mx_operand, ok, rng_of

pytestmark = pytest.mark.gpu

# streams, tiles, 256 x 256 tiles
SIZES = [(24, 40, 32), (17, 70, 1312), (300, 616, 160), (4100, 4097, 288)]


def product(ca, sa, cb, sb, out, groups=False):
    """The kernel's C (fp64) and the operands' values; as one product, or as one of a single group."""
    (M, K), N = ca.shape, cb.shape[0]
    A, SA, lda, ldsa = mx_operand(ca, sa)
    B, SB, ldb, ldsb = mx_operand(cb, sb)
    C = torch.full((M, N), 7.0, dtype=R.TORCH[out], device="cuda")
    print("CASE mxfp4 range", M, N, K, out, groups, flush=True)
    s = torch.cuda.current_stream()
    if groups:
        ends = torch.tensor([M], dtype=torch.int32, device="cuda")
        ok(lsm.gemm_grouped_mxfp4_run(H.handle(), A, B, C, SA, SB, ends, 1, M, N, K, lda, ldb, 0, N, ldsa, ldsb, 0, DTYPE[out],
                                      s), "gemm_grouped_mxfp4_run")
    else:
        ok(lsm.gemm_mxfp4_run(H.handle(), A, B, C, SA, SB, M, N, K, lda, ldb, N, ldsa, ldsb, DTYPE[out], s), "gemm_mxfp4_run")
    return R.f64(C), G.values(ca, sa), G.values(cb, sb)


def extreme_scales(rng, rows, blocks):
    """0 to 254, a third of them at the ends."""
    s = rng.integers(0, 255, (rows, blocks))
    ends = np.array([0, 1, 2, 252, 253, 254])[rng.integers(0, 6, (rows, blocks))]
    return np.where(rng.random((rows, blocks)) < 1 / 3, ends, s).astype(np.uint8)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("groups", [False, True])
def test_one_product(M, N, K, groups):
    """One product an entry, of every size that two scales give: exact where fp32 holds it, infinite beyond,
    and within a step of 2^-149 below 2^-126."""
    rng = rng_of(M, N, K, 1)
    k = int(rng.integers(0, K))
    ca, cb = np.zeros((M, K), np.uint8), np.zeros((N, K), np.uint8)
    ca[:, k], cb[:, k] = rng.integers(0, 16, M), rng.integers(0, 16, N)
    got, a, b = product(ca, extreme_scales(rng, M, K // 32), cb, extreme_scales(rng, N, K // 32), "f32", groups)
    ref = np.outer(a[:, k], b[:, k])
    assert (np.abs(ref) >= 2.0 ** 128).any() and ((np.abs(ref) < 2.0 ** -149) & (ref != 0)).any()
    large = np.abs(ref) >= 2.0 ** 128
    assert np.array_equal(got[large], np.sign(ref[large]) * np.inf)
    normal = ~large & (np.abs(ref) >= 2.0 ** -126)
    assert np.array_equal(got[normal], ref[normal])
    small = ~large & ~normal
    R.assert_within(got[small], ref[small], 2.0 ** -149, "below 2^-126")


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out", sorted(DTYPE))
@pytest.mark.parametrize("low", [False, True])
def test_sums(M, N, K, out, low):
    """Sums under scales of every size whose products are 2^-120 to 2^120, and (`low`) under products about
    2^-140: within the header's bound."""
    rng = rng_of(M, N, K, 2)
    ca, cb = (rng.integers(0, 16, (n, K), dtype=np.uint8) for n in (M, N))
    if low:
        sa, sb = (rng.integers(50, 66, (n, K // 32)).astype(np.uint8) for n in (M, N))
    else:
        at = rng.integers(0, 255, K // 32)
        sa, sb = (np.clip(c + rng.integers(-60, 61, (n, K // 32)), 0, 254).astype(np.uint8) for n, c in ((M, at), (N, 254 - at)))
    got, a, b = product(ca, sa, cb, sb, out)
    ref, bound = G.product(a, b)
    size = np.abs(a) @ np.abs(b).T
    bound = bound + (K / 128 + 8) * 2.0 ** -149
    said, most = size < 2.0 ** 127, float(torch.finfo(R.TORCH[out]).max)
    assert said.any()
    beyond = said & (np.abs(ref) - bound > most * (1 + 2.0 ** -8))        # rounds to an infinity of C's type
    assert np.array_equal(got[beyond], np.sign(ref[beyond]) * np.inf)
    within = said & (np.abs(ref) + bound <= most)
    assert (beyond | within).sum() > 0.9 * said.sum()
    R.assert_within(got[within], ref[within], (bound + R.HALF_STEP[out] * (np.abs(ref) + bound) + R.SMALLEST[out])[within],
                    f"{M}x{N}x{K} {out}")
