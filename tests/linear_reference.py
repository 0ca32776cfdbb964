"""fp64 definitions of the linear-layer operators and the bounds that their
tests hold the kernels to.

Unit roundings: fp32 2^-24; a sum inside the matrix instruction may be cut
instead of rounded, so sums count 2^-23 an addition.  A rounding to a narrower
type is off by half a step: 2^-8 (bf16) or 2^-11 (fp16) of the value, and half
the smallest step for subnormal fp16 results.
"""
import numpy as np
import torch

FP8 = torch.float8_e4m3fn
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": FP8}
HALF_STEP = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
SMALLEST = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
AMAX_MIN = 2.0 ** -100


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def round_to(v, kind):
    """fp64 values rounded to `kind`, back in fp64."""
    return f64(torch.from_numpy(np.ascontiguousarray(v)).to(torch.float32).to(TORCH[kind]))


def assert_within(got, ref, bound, what):
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - ref) <= bound) & ~((got == ref) | (np.isnan(got) & np.isnan(ref)))
    if bad.any():
        i = tuple(int(x[0]) for x in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.size} entries off, first at {i}: got {got[i]!r} "
                             f"want {ref[i]!r} bound {np.broadcast_to(bound, got.shape)[i]!r}")


def assert_rounded(got, v, slack, kind, what):
    """Each entry is the rounding to `kind` of a value within a relative `slack` of v."""
    lo, hi = v * (1 - slack), v * (1 + slack)
    a, b = round_to(np.minimum(lo, hi), kind), round_to(np.maximum(lo, hi), kind)
    bad = ~((got >= a) & (got <= b)) & ~(np.isnan(got) & np.isnan(v))
    if bad.any():
        i = tuple(int(x[0]) for x in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {got.size} entries off, first at {i}: got {got[i]!r} "
                             f"want the rounding of {v[i]!r}")


# ------------------------------------------------------------------ norm

def rmsnorm(x, r, w, eps):
    """(h, y) in fp64."""
    h = x if r is None else x + r
    with np.errstate(invalid="ignore", over="ignore"):
        y = h * w / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h, y


def rmsnorm_slack(N):
    """Relative error of y in fp32: h and h*root*w*(448/max) are 5 roundings;
    the mean of squares has one rounding a square and an addition for each of
    a thread's elements (32, or N / 1024 of a longer row), 6 across a wave and
    16 across waves, the division and eps -- halved by the root, whose own
    error is 2 -- and the scale's max, root and quotients are 4 more."""
    adds = max(32, -(-N // 1024) + 8) + 6 + 16 + 3
    return (5 + adds / 2 + 2 + 4) * 2.0 ** -24


def row_scale(y):
    return np.maximum(np.max(np.abs(y), axis=1), AMAX_MIN) / 448.0


# ---------------------------------------------------------------- scaled

FP8_MFMA_DROP = 2.0 ** -10


def scaled(a, b, sa, sb, fp8_mfma=False):
    """(C, bound of the fp32 sum and its two factors) for a (M x K), b (N x K).

    `fp8_mfma`: the sum comes from the fp8 matrix instructions.  They align the
    eight products of a group, and the sum so far, to the largest product and
    drop what lies 13 or more bits below the largest exponent
    (test_gpu_linear.py checks this): at most 8 terms lose at most 2^-13 times
    the group's largest product each, that product is no more than the group's
    sum of sizes, and so the groups together lose no more than
    8 * 2^-13 = 2^-10 times the sum of all sizes."""
    with np.errstate(invalid="ignore", over="ignore"):
        c = a @ b.T
        scale = sa[:, None] * sb[None, :]
        size = np.abs(a) @ np.abs(b).T
        drop = FP8_MFMA_DROP if fp8_mfma else 0.0
        return c * scale, ((a.shape[1] + 16) * 2.0 ** -23 + drop) * size * np.abs(scale) + \
            2 * 2.0 ** -24 * np.abs(c * scale)


# -------------------------------------------------------------------- w4

def pack4(q):
    """N x K values 0..15 as N x K/2 bytes, even k in the low half."""
    return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8)


def w4(a, q, s, z, group):
    """(C, bound of the fp32 arithmetic) for a (M x K), q (N x K), s and z (G x N; z may be None).

    Per group the kernel sums a (16 + q) and a, at most `group` additions each,
    forms s (sum1 - (16 + z) sum2) in 4 roundings of terms no larger than their
    sizes, and adds G groups and 16 partial sums."""
    K = a.shape[1]
    of = np.arange(K) // group
    zz = np.full_like(s, 8.0) if z is None else z
    w = (q.astype(np.float64) - zz[of].T) * s[of].T
    with np.errstate(invalid="ignore", over="ignore"):
        c = a @ w.T
        bound = np.zeros_like(c)
        for g in range(s.shape[0]):
            n = min(group, K - g * group)
            size = np.abs(a[:, of == g]).sum(1)[:, None] * (np.abs(s[g]) * (31 + 16 + zz[g]))[None, :]
            bound += (n + 4 + s.shape[0] + 16) * 2.0 ** -23 * size
    return c, bound
