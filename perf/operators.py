"""The operators of a quantised linear layer, as cases to be measured.

Three operators work together around the library's matrix product:

``norm``    the root-mean-square norm with the residual's addition, whose output is either the
            16-bit type of its input or E4M3 with one fp32 scale a row (the A operand of the next
            two);
``scaled``  the product of two E4M3 matrices whose rows (A) and columns (B) carry fp32 scales;
``w4``      the product of a few 16-bit rows with a matrix of 4-bit weights, scales and zero
            points by groups of K.

``run`` computes a case in plain torch operations in fp32 (``own`` false) or calls the library
(``own`` true).  ``exact`` gives the same outputs from the definitions in fp64.
"""
import math

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
AMAX_MIN = 2.0 ** -100          # a row's largest value counts as at least this
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-5


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a decode step, normalised for an 8-bit product
        dict(name="norm one token", op="norm", M=1, N=4096, type="bf16", out="e4m3", residual=True),
        # a serving batch of the 1152-wide layer the library's tests use, in fp16
        dict(name="norm 1500x1152", op="norm", M=1500, N=1152, type="f16", out="e4m3", residual=False),
        # rows of odd length in a padded buffer, 16-bit output
        dict(name="norm odd rows", op="norm", M=300, N=1151, type="bf16", out="bf16", residual=True),
        # a long prompt at the library's large size
        dict(name="norm 8192x8192", op="norm", M=8192, N=8192, type="bf16", out="e4m3", residual=True),
        # one token through a square projection
        dict(name="scaled one token", op="scaled", M=1, N=4096, K=4096, out="bf16"),
        # a decode batch at the library's skinny shape
        dict(name="scaled 32 rows", op="scaled", M=32, N=16384, K=8192, out="bf16"),
        # the library's ragged shape (no extent a multiple of a large tile), fp16 output
        dict(name="scaled 1500x1152x896", op="scaled", M=1500, N=1152, K=896, out="f16"),
        # a long prompt at the library's headline shape
        dict(name="scaled 8192 cubed", op="scaled", M=8192, N=8192, K=8192, out="f32"),
        # one token through a small projection: launch and latency
        dict(name="w4 one token small", op="w4", M=1, N=2048, K=2048, group=128, type="bf16", out="bf16", zeros=False),
        # one token through the skinny shape's weights
        dict(name="w4 one token", op="w4", M=1, N=16384, K=8192, group=128, type="f16", out="f16", zeros=True),
        # seven drafted tokens, ragged sizes, the smallest groups, fp32 logits
        dict(name="w4 seven rows", op="w4", M=7, N=1151, K=896, group=32, type="bf16", out="f32", zeros=True),
        # a decode batch
        dict(name="w4 48 rows", op="w4", M=48, N=8192, K=8192, group=64, type="bf16", out="bf16", zeros=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "scaled", "w4"])
    if op == "norm":
        kind = rng.choice(["bf16", "f16"])
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 64, 8192), type=kind,
                    out=rng.choice(["e4m3", kind]), residual=rng.random() < 0.7)
    if op == "scaled":
        # whole 16-byte pieces of K, as 8-bit operands need them; M and N as they come
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 256, 8192),
                    K=16 * _log_int(rng, 16, 512), out=rng.choice(["bf16", "f16", "f32"]))
    kind = rng.choice(["bf16", "f16"])
    return dict(op=op, M=_log_int(rng, 1, 64), N=_log_int(rng, 256, 16384),
                K=32 * _log_int(rng, 8, 256), group=rng.choice([32, 64, 128]), type=kind,
                out=rng.choice([kind, "f32"]), zeros=rng.random() < 0.5)


# ----------------------------------------------------------------- the inputs

def _up(n, q):
    return -(-n // q) * q


def _quantise_rows(v):
    """v (fp32) as E4M3 with one scale a row."""
    s = v.abs().amax(1).clamp_min(AMAX_MIN) / FP8_MAX
    return (v / s[:, None]).clamp(-FP8_MAX, FP8_MAX).to(FP8), s


def _padded(rows, cols, pitch, dtype):
    """A rows x cols view into rows of `pitch` elements."""
    return torch.zeros(rows, pitch, dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    M, N = case["M"], case["N"]
    s = dict(case)
    if case["op"] == "norm":
        t = TYPES[case["type"]]
        pitch = _up(N, 16)
        # a hidden state: a few channels far larger than the others
        loud = 1 + 20 * (torch.rand(N, generator=g, device="cuda") > 0.99).float()
        s["X"] = _padded(M, N, pitch, t)
        s["X"].copy_(randn(M, N) * loud)
        s["R"] = None
        s["H"] = None
        if case["residual"]:
            s["R"] = _padded(M, N, pitch, t)
            s["R"].copy_(randn(M, N) * 2)
            s["H"] = _padded(M, N, pitch, t)
        s["W"] = (1 + 0.1 * randn(N)).to(t)
        s["Y"] = _padded(M, N, pitch, FP8 if case["out"] == "e4m3" else t)
        s["S"] = torch.zeros(M, dtype=torch.float32, device="cuda") if case["out"] == "e4m3" else None
    elif case["op"] == "scaled":
        K = case["K"]
        # activations row by row and weights column by column, both K-contiguous
        s["A"], s["SA"] = _quantise_rows(randn(M, K) * (0.5 + torch.rand(M, 1, generator=g, device="cuda")))
        s["B"], s["SB"] = _quantise_rows(randn(N, K) / math.sqrt(K))
        s["C"] = torch.zeros(M, N, dtype=TYPES[case["out"]], device="cuda")
    else:
        K, group = case["K"], case["group"]
        t = TYPES[case["type"]]
        G = -(-K // group)
        s["A"] = randn(M, K).to(t)
        # weights quantised group by group, as a checkpoint holds them: scales and zero points
        # K group by K group, two weights a byte
        w = torch.zeros(N, G * group, device="cuda")
        w[:, :K] = randn(N, K) / math.sqrt(K)
        w = w.view(N, G, group)
        if case["zeros"]:
            lo, hi = w.amin(2), w.amax(2)
            scale = ((hi - lo).clamp_min(1e-4) / 15).to(t)
            zero = (-lo / scale.float()).round().clamp(0, 15)
        else:
            scale = (w.abs().amax(2).clamp_min(1e-4) / 7).to(t)
            zero = torch.full_like(w[:, :, 0], 8)
        q = (w / scale.float()[:, :, None] + zero[:, :, None]).round().clamp(0, 15)
        q = q.view(N, G * group)[:, :K].to(torch.uint8)
        s["B"] = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
        s["S"] = scale.t().contiguous()
        s["Z"] = zero.to(torch.uint8).t().contiguous() if case["zeros"] else None
        s["C"] = torch.zeros(M, N, dtype=TYPES[case["out"]], device="cuda")
    return s


# ----------------------------------------------------------------- the operators

_library = None


def _lib():
    """The library and a handle, as a program keeps them."""
    global _library
    if _library is None:
        import lds_staged_matrix_amd as lsm
        _library = lsm, lsm.gemm_create()
    return _library


def _stream():
    """The stream that the inputs were made on and the outputs are read on, by its handle alone:
    torch.cuda.current_stream() would make a Stream object of it first, in 2.7 us."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _check(lsm, status, what):
    if status != lsm.GEMM_OK:
        raise lsm.GemmError(status, what)


def _own_norm(s):
    lsm, h = _lib()
    X, R, H, Y = s["X"], s["R"], s["H"], s["Y"]
    dtype = {("bf16", "bf16"): lsm.GEMM_NORM_BF16_BF16, ("bf16", "e4m3"): lsm.GEMM_NORM_BF16_E4M3,
             ("f16", "f16"): lsm.GEMM_NORM_F16_F16, ("f16", "e4m3"): lsm.GEMM_NORM_F16_E4M3}[s["type"], s["out"]]
    _check(lsm, lsm.gemm_rmsnorm_run(h, X, R, s["W"], H, Y, s["S"], s["M"], s["N"], X.stride(0),
                                     R.stride(0) if R is not None else 0,
                                     H.stride(0) if H is not None else 0, Y.stride(0), EPS, dtype,
                                     _stream()),
           "gemm_rmsnorm_run")
    return {"Y": Y, "S": s["S"], "H": H}


def _own_scaled(s):
    lsm, h = _lib()
    A, B, C = s["A"], s["B"], s["C"]
    dtype = {"bf16": lsm.GEMM_E4M3_BF16, "f16": lsm.GEMM_E4M3_F16, "f32": lsm.GEMM_E4M3_F32}[s["out"]]
    _check(lsm, lsm.gemm_scaled_run(h, A, B, C, s["SA"], s["SB"], s["M"], s["N"], s["K"], A.stride(0),
                                    B.stride(0), C.stride(0), 1, 1, lsm.GEMM_K_CONTIG,
                                    lsm.GEMM_K_CONTIG, dtype, _stream()),
           "gemm_scaled_run")
    return C


def _own_w4(s):
    lsm, h = _lib()
    A, B, S, Z, C = s["A"], s["B"], s["S"], s["Z"], s["C"]
    dtype = {("bf16", "bf16"): lsm.GEMM_BF16_BF16, ("bf16", "f32"): lsm.GEMM_BF16_F32,
             ("f16", "f16"): lsm.GEMM_F16_F16, ("f16", "f32"): lsm.GEMM_F16_F32}[s["type"], s["out"]]
    _check(lsm, lsm.gemm_w4_run(h, A, B, S, Z, C, s["M"], s["N"], s["K"], s["group"], A.stride(0),
                                2 * B.stride(0), S.stride(0), Z.stride(0) if Z is not None else 0,
                                C.stride(0), dtype, _stream()),
           "gemm_w4_run")
    return C


def _plain_norm(s):
    t = TYPES[s["type"]]
    h = s["X"].float()
    if s["R"] is not None:
        h = h + s["R"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * s["W"].float()
    H = h.to(t) if s["R"] is not None else None
    if s["out"] != "e4m3":
        return {"Y": y.to(t), "S": None, "H": H}
    scale = y.abs().amax(1).clamp_min(AMAX_MIN) / FP8_MAX
    return {"Y": (y / scale[:, None]).clamp(-FP8_MAX, FP8_MAX).to(FP8), "S": scale, "H": H}


def _plain_scaled(s):
    c = s["A"].float() @ s["B"].float().t()
    return (c * s["SA"][:, None] * s["SB"]).to(TYPES[s["out"]])


def _plain_w4(s):
    N, K, group = s["N"], s["K"], s["group"]
    q = torch.stack((s["B"] & 15, s["B"] >> 4), 2).view(N, K).float()
    of = torch.arange(K, device="cuda") // group
    zero = s["Z"].float()[of].t() if s["Z"] is not None else 8.0
    w = (q - zero) * s["S"].float()[of].t()
    return (s["A"].float() @ w.t()).to(TYPES[s["out"]])


def run(state):
    if own:
        return {"norm": _own_norm, "scaled": _own_scaled, "w4": _own_w4}[state["op"]](state)
    return {"norm": _plain_norm, "scaled": _plain_scaled, "w4": _plain_w4}[state["op"]](state)


# ----------------------------------------------------------------- the work and the exact values

def work(case):
    M, N = case["M"], case["N"]
    if case["op"] == "norm":
        per = 2 + (1 if case["out"] == "e4m3" else 2) + (4 if case["residual"] else 0)
        return {"bytes": M * N * per + 2 * N + (4 * M if case["out"] == "e4m3" else 0), "flops": 6 * M * N}
    K = case["K"]
    out = 4 if case["out"] == "f32" else 2
    if case["op"] == "scaled":
        return {"bytes": M * K + N * K + 4 * (M + N) + out * M * N, "flops": 2 * M * N * K}
    groups = -(-K // case["group"])
    return {"bytes": 2 * M * K + N * K // 2 + N * groups * (3 if case["zeros"] else 2) + out * M * N,
            "flops": 2 * M * N * K}


def exact(case, seed):
    """The outputs before their last rounding, in fp64.  A quantised output is given as the value
    that its 8 bits stand for, not yet rounded to them."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["X"].to(torch.float64)
        if case["residual"]:
            h += s["R"].to(torch.float64)
        root = ((h * h).sum(1) / case["N"] + EPS).sqrt()
        y = h / root[:, None] * s["W"].to(torch.float64)
        out = {"Y": y, "S": None, "H": h if case["residual"] else None}
        if case["out"] == "e4m3":
            out["S"] = y.abs().max(1).values.clamp(min=AMAX_MIN) / FP8_MAX
            out["Y"] = y / out["S"][:, None]
        return out
    if case["op"] == "scaled":
        a = s["A"].to(torch.float64) * s["SA"].to(torch.float64)[:, None]
        b = s["B"].to(torch.float64) * s["SB"].to(torch.float64)[:, None]
        return torch.matmul(a, b.t())
    N, K, group = case["N"], case["K"], case["group"]
    G = s["S"].shape[0]
    w = torch.zeros(N, G * group, dtype=torch.float64, device="cuda")
    w[:, 0:K:2] = s["B"].bitwise_and(15).to(torch.float64)
    w[:, 1:K:2] = (s["B"] // 16).to(torch.float64)
    w = w.view(N, G, group)
    w -= 8.0 if s["Z"] is None else s["Z"].t().to(torch.float64)[:, :, None]
    w *= s["S"].t().to(torch.float64)[:, :, None]
    return torch.matmul(s["A"].to(torch.float64), w.view(N, G * group)[:, :K].t())
