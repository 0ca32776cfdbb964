"""fp64 definitions of MXFP4 and of the grouped products, and the bounds that their
tests hold the kernels to (unit roundings: see linear_reference.py).

MXFP4: E2M1 elements, two a byte, and E8M0 scales, a row of M bytes for every 32 k.
"""
import numpy as np

BLOCK = 32
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
NAN_SCALE = 255


def up(n, q):
    return -(-max(n, 1) // q) * q


# ------------------------------------------------------------------ MXFP4

def quantize(x):
    """(codes M x K, scales M x K/32) of fp64 values."""
    M, K = x.shape
    b = x.reshape(M, K // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(2)
    b = np.where(bad[:, :, None], 0.0, b)
    amax = np.abs(b).max(2)
    e = np.where(amax > 0, np.clip(np.frexp(amax)[1] - 1 - 2, -127, 127), -127)
    size = np.abs(b) * np.exp2(-e.astype(np.float64))[:, :, None]
    # nearest of the eight sizes; a tie goes to the even code
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    code = np.zeros(size.shape, dtype=np.uint8)
    for i, m in enumerate(mid):
        code += (size > m) | ((size == m) & (i % 2 == 1))
    code |= (np.signbit(b) << 3).astype(np.uint8)
    code[bad] = 0
    return code.reshape(M, K), np.where(bad, NAN_SCALE, e + 127).astype(np.uint8)


def values(code, scale):
    """fp64 values of codes (M x K) and scales (M x K/32)."""
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    s = np.where(scale == NAN_SCALE, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return v * np.repeat(s, BLOCK, axis=1)


def pack(code):
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)


def unpack(q):
    return np.stack((q & 15, q >> 4), 2).reshape(q.shape[0], -1)


def product(a, b):
    """(a b^T, bound of the matrix instruction's sums): an instruction of 128 k is off by 5.4 2^-24 of
    its terms' sizes and of the sum so far at most (measured), for which 2^-21 is counted; splitting K
    over waves adds at most 8 additions."""
    with np.errstate(invalid="ignore", over="ignore"):
        size = np.abs(a) @ np.abs(b).T
        return a @ b.T, (a.shape[1] / 128 + 8) * 2.0 ** -21 * size


# ----------------------------------------------------------------- groups

def bounds(ends, T):
    """[(first, last)] of the groups that the ends mean."""
    out, at = [], 0
    for e in ends:
        last = max(at, min(max(int(e), 0), T))
        out.append((at, last))
        at = last
    return out


def sum_bound(size, K):
    """Sums of K terms in fp32 (2^-23 an addition: a matrix instruction may cut instead of round)."""
    return (K + 16) * 2.0 ** -23 * size
