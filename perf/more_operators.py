"""Products grouped by expert and products of 4-bit microscaled numbers, as cases to be measured.

``quantize``      16-bit (or fp32) matrices to MXFP4 and back: E2M1 elements, two a byte, with one
                  E8M0 scale for every 32 consecutive k.  A pass quantises and returns the values
                  that the 4 bits and the scales stand for;
``mxfp4``         the product of two MXFP4 matrices;
``grouped``       rows sorted by expert, each expert's rows times its own matrix (the forward pass,
                  and with the other layout of B the gradient of the rows);
``wgrad``         the gradient of the experts' matrices;
``grouped_mxfp4`` the grouped product with MXFP4 rows and matrices.

The groups' ends stand on the device: ``ends[g]`` is the row behind group g's last, group g starts
where group g - 1 ends, and rows behind the last group belong to no expert and are left alone.

``run`` computes a case in plain torch operations in fp32 (``own`` false) or calls the library
(``own`` true).  ``exact`` gives the same outputs from the definitions in fp64.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32                      # k that share a scale
EMAX = 2                        # exponent of the largest E2M1 number, 6 = 1.5 * 2^2
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # one token's activations before a 4-bit projection
        dict(name="quantize one token", op="quantize", M=1, K=4096, type="bf16", layout="K"),
        # a long prompt's activations at the library's large size
        dict(name="quantize 8192x8192", op="quantize", M=8192, K=8192, type="bf16", layout="K"),
        # one token through a square projection: the weights' bytes and the call
        dict(name="mxfp4 one token", op="mxfp4", M=1, N=4096, K=4096, out="bf16"),
        # the library's ragged shape (no extent a multiple of a large tile), fp16 output
        dict(name="mxfp4 1500x1152x896", op="mxfp4", M=1500, N=1152, K=896, out="f16"),
        # a long prompt at the library's headline shape
        dict(name="mxfp4 8192 cubed", op="mxfp4", M=8192, N=8192, K=8192, out="bf16"),
        # a decode step: a few rows for each expert, the weights read once
        dict(name="grouped decode", op="grouped", T=64, G=16, N=4096, K=4096, type="bf16", out="bf16", layout="K"),
        # the gradient of a short ragged batch's rows: the forward's weights read along their other side
        dict(name="grouped 1500 rows", op="grouped", T=1500, G=8, N=896, K=1152, type="f16", out="f16", layout="MN"),
        # a training batch's forward pass
        dict(name="grouped 16384 rows", op="grouped", T=16384, G=8, N=4096, K=4096, type="bf16", out="bf16", layout="K"),
        # the weights' gradient of the short batch, some experts with a handful of rows
        dict(name="wgrad 1500 rows", op="wgrad", T=1500, G=8, M=1152, N=896, type="f16", out="f32"),
        # the weights' gradient of the training batch, kept in fp32 for the optimiser
        dict(name="wgrad 16384 rows", op="wgrad", T=16384, G=8, M=4096, N=4096, type="bf16", out="f32"),
        # a decode step with 4-bit experts
        dict(name="grouped mxfp4 decode", op="grouped_mxfp4", T=64, G=16, N=4096, K=4096, out="bf16"),
        # a prompt through 4-bit experts
        dict(name="grouped mxfp4 8192 rows", op="grouped_mxfp4", T=8192, G=8, N=4096, K=4096, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "mxfp4", "grouped", "wgrad", "grouped_mxfp4"])
    if op == "quantize":
        # whole blocks of K; the rows as they come, in whole 16-byte pieces where they are contiguous
        layout = rng.choice(["K", "K", "MN"])
        return dict(op=op, M=_log_int(rng, 1, 8192), K=BLOCK * _log_int(rng, 4, 256),
                    type=rng.choice(["bf16", "f16", "f32"]), layout=layout)
    if op == "mxfp4":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 256, 8192), K=BLOCK * _log_int(rng, 8, 256),
                    out=rng.choice(["bf16", "f16", "f32"]))
    # the experts' matrices together hold no more than the listed ones'
    G = rng.choice([1, 4, 7, 8, 16, 32])
    T = _log_int(rng, 1, 16384 if op != "grouped_mxfp4" else 8192)
    N = _log_int(rng, 256, 4096)
    if op == "grouped_mxfp4":
        return dict(op=op, T=T, G=G, N=N, K=BLOCK * _log_int(rng, 8, 4096 // BLOCK),
                    out=rng.choice(["bf16", "f16", "f32"]))
    kind = rng.choice(["bf16", "f16"])
    out = rng.choice([kind, "f32"])
    if op == "wgrad":
        return dict(op=op, T=T, G=min(G, 8), M=8 * _log_int(rng, 32, 512), N=8 * _log_int(rng, 32, 512),
                    type=kind, out=out)
    layout = rng.choice(["K", "MN"])
    return dict(op=op, T=T, G=G, N=8 * (N // 8) if layout == "MN" else N, K=8 * _log_int(rng, 32, 512), type=kind,
                out=out, layout=layout)


# ----------------------------------------------------------------- the inputs

def _up(n, q):
    return -(-n // q) * q


def _pack(code, sign):
    """E2M1 codes and signs, even k in the low half of a byte."""
    v = code | (sign << 3)
    return v[..., 0::2] | (v[..., 1::2] << 4)


def _quantize(v):
    """fp32 rows as (packed E2M1 elements, E8M0 bytes of the blocks): the scale is two to the
    exponent of the block's largest size, less that of 6; elements round to the nearest, ties to
    even, and stop at 6."""
    b = v.reshape(*v.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 1 - EMAX).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    a = torch.ldexp(b.abs(), -e[..., None])
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    sign = torch.signbit(b).to(torch.uint8)
    return _pack(code.reshape(v.shape), sign.reshape(v.shape)), (e + 127).to(torch.uint8)


def _scales(s):
    """E8M0 bytes, row by row, as the library keeps them: one row of M for every 32 k, rows padded
    to 16 bytes."""
    s = s.transpose(-1, -2)
    buf = torch.zeros(*s.shape[:-1], _up(s.shape[-1], 16), dtype=torch.uint8, device=s.device)
    buf[..., :s.shape[-1]] = s
    return buf


def _ends(case, g):
    """The rows of each group, from a router that likes some experts better: about one row in 64
    belongs to none (a padded batch)."""
    T, G = case["T"], case["G"]
    rows = T - T // 64
    like = torch.softmax(0.5 * torch.randn(G, generator=g), 0)
    to = torch.multinomial(like, rows, replacement=True, generator=g) if rows else torch.zeros(0, dtype=torch.int64)
    return torch.cumsum(torch.bincount(to, minlength=G), 0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def activations(rows, k):
        # a hidden state: a few channels far larger than the others
        loud = 1 + 20 * (torch.rand(k, generator=g, device="cuda") > 0.99).float()
        return randn(rows, k) * loud

    s = dict(case)
    op = case["op"]
    if op == "quantize":
        M, K, t = case["M"], case["K"], TYPES[case["type"]]
        x = activations(M, K).to(t)
        if case["layout"] == "MN":
            x = x.t().contiguous()
        s["X"] = x
        s["Q"] = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
        s["S"] = torch.zeros(K // BLOCK, _up(M, 16), dtype=torch.uint8, device="cuda")
        s["Y"] = torch.zeros(M, K, dtype=t, device="cuda")
        return s
    if op == "mxfp4":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"], sa = _quantize(activations(M, K))
        s["B"], sb = _quantize(randn(N, K) / math.sqrt(K))
        s["SA"], s["SB"] = _scales(sa), _scales(sb)
        s["C"] = torch.zeros(M, N, dtype=TYPES[case["out"]], device="cuda")
        return s
    T, G = case["T"], case["G"]
    ends = _ends(case, torch.Generator().manual_seed(seed))
    s["host_ends"] = ends.tolist()             # what the plain form's loop goes by
    s["ends"] = ends.to(torch.int32).cuda()
    if op == "wgrad":
        M, N, t = case["M"], case["N"], TYPES[case["type"]]
        s["A"] = activations(T, M).to(t)
        s["B"] = (randn(T, N) / math.sqrt(N)).to(t)
        s["C"] = torch.zeros(G, M, N, dtype=TYPES[case["out"]], device="cuda")
        return s
    N, K = case["N"], case["K"]
    s["C"] = torch.zeros(T, N, dtype=TYPES[case["out"]], device="cuda")
    if op == "grouped_mxfp4":
        s["A"], sa = _quantize(activations(T, K))
        b, sb = zip(*(_quantize(randn(N, K) / math.sqrt(K)) for _ in range(G)))
        s["B"] = torch.stack(b)
        s["SA"], s["SB"] = _scales(sa), _scales(torch.stack(sb))
        return s
    t = TYPES[case["type"]]
    s["A"] = activations(T, K).to(t)
    s["B"] = torch.empty(G, *((N, K) if case["layout"] == "K" else (K, N)), dtype=t, device="cuda")
    for b in s["B"]:
        b.copy_(randn(*b.shape) / math.sqrt(K))
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
    """The stream that the inputs were made on and the outputs are read on, by its handle alone."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _check(lsm, status, what):
    if status != lsm.GEMM_OK:
        raise lsm.GemmError(status, what)


def _mxfp4_type(lsm, kind):
    return {"bf16": lsm.GEMM_MXFP4_BF16, "f16": lsm.GEMM_MXFP4_F16, "f32": lsm.GEMM_MXFP4_F32}[kind]


def _type(lsm, kind, out):
    return {("bf16", "bf16"): lsm.GEMM_BF16_BF16, ("bf16", "f32"): lsm.GEMM_BF16_F32,
            ("f16", "f16"): lsm.GEMM_F16_F16, ("f16", "f32"): lsm.GEMM_F16_F32}[kind, out]


def _layout(lsm, layout):
    return lsm.GEMM_K_CONTIG if layout == "K" else lsm.GEMM_MN_CONTIG


def _own_quantize(s):
    lsm, h = _lib()
    X, Q, S, Y, M, K = s["X"], s["Q"], s["S"], s["Y"], s["M"], s["K"]
    dtype, stream = _mxfp4_type(lsm, s["type"]), _stream()
    _check(lsm, lsm.gemm_mxfp4_quantize_run(h, X, Q, S, M, K, X.stride(0), 2 * Q.stride(0), S.stride(0),
                                            _layout(lsm, s["layout"]), dtype, stream), "gemm_mxfp4_quantize_run")
    _check(lsm, lsm.gemm_mxfp4_dequantize_run(h, Q, S, Y, M, K, 2 * Q.stride(0), S.stride(0), Y.stride(0), dtype,
                                              stream), "gemm_mxfp4_dequantize_run")
    return Y


def _own_mxfp4(s):
    lsm, h = _lib()
    A, B, C, SA, SB = s["A"], s["B"], s["C"], s["SA"], s["SB"]
    _check(lsm, lsm.gemm_mxfp4_run(h, A, B, C, SA, SB, s["M"], s["N"], s["K"], 2 * A.stride(0), 2 * B.stride(0),
                                   C.stride(0), SA.stride(0), SB.stride(0), _mxfp4_type(lsm, s["out"]), _stream()),
           "gemm_mxfp4_run")
    return C


def _own_grouped(s):
    lsm, h = _lib()
    A, B, C = s["A"], s["B"], s["C"]
    _check(lsm, lsm.gemm_grouped_run(h, A, B, C, s["ends"], s["G"], s["T"], s["N"], s["K"], A.stride(0), B.stride(1),
                                     B.stride(0), C.stride(0), _layout(lsm, s["layout"]),
                                     _type(lsm, s["type"], s["out"]), _stream()), "gemm_grouped_run")
    return C


def _own_wgrad(s):
    lsm, h = _lib()
    A, B, C = s["A"], s["B"], s["C"]
    _check(lsm, lsm.gemm_grouped_wgrad_run(h, A, B, C, s["ends"], s["G"], s["T"], s["M"], s["N"], A.stride(0),
                                           B.stride(0), C.stride(1), C.stride(0), _type(lsm, s["type"], s["out"]),
                                           _stream()), "gemm_grouped_wgrad_run")
    return C


def _own_grouped_mxfp4(s):
    lsm, h = _lib()
    A, B, C, SA, SB = s["A"], s["B"], s["C"], s["SA"], s["SB"]
    _check(lsm, lsm.gemm_grouped_mxfp4_run(h, A, B, C, SA, SB, s["ends"], s["G"], s["T"], s["N"], s["K"],
                                           2 * A.stride(0), 2 * B.stride(1), 2 * B.stride(0), C.stride(0),
                                           SA.stride(0), SB.stride(1), SB.stride(0), _mxfp4_type(lsm, s["out"]),
                                           _stream()), "gemm_grouped_mxfp4_run")
    return C


def _values(q, s, rows):
    """The fp32 values of packed elements and of their blocks' scales (as _scales lays them out)."""
    code = torch.stack((q & 15, q >> 4), -1).flatten(-2).long()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    e = s[..., :rows].transpose(-1, -2).to(torch.int32) - 127
    v = table[code].unflatten(-1, (-1, BLOCK))
    return torch.ldexp(v, e[..., None]).flatten(-2)


def _plain_quantize(s):
    x = s["X"].float()
    if s["layout"] == "MN":
        x = x.t()
    q, e = _quantize(x)
    return _values(q, e.t(), s["M"]).to(TYPES[s["type"]])


def _plain_mxfp4(s):
    a, b = _values(s["A"], s["SA"], s["M"]), _values(s["B"], s["SB"], s["N"])
    return (a @ b.t()).to(TYPES[s["out"]])


def _plain_grouped(s):
    c = torch.zeros(s["T"], s["N"], dtype=TYPES[s["out"]], device="cuda")
    first = 0
    for b, end in zip(s["B"], s["host_ends"]):
        if end > first:
            w = b.float()
            c[first:end] = s["A"][first:end].float() @ (w.t() if s["layout"] == "K" else w)
        first = end
    return c


def _plain_wgrad(s):
    c = torch.zeros(s["G"], s["M"], s["N"], dtype=TYPES[s["out"]], device="cuda")
    first = 0
    for g, end in enumerate(s["host_ends"]):
        if end > first:
            c[g] = s["A"][first:end].float().t() @ s["B"][first:end].float()
        first = end
    return c


def _plain_grouped_mxfp4(s):
    c = torch.zeros(s["T"], s["N"], dtype=TYPES[s["out"]], device="cuda")
    a = _values(s["A"], s["SA"], s["T"])
    first = 0
    for b, sb, end in zip(s["B"], s["SB"], s["host_ends"]):
        if end > first:
            c[first:end] = a[first:end] @ _values(b, sb, s["N"]).t()
        first = end
    return c


def run(state):
    if own:
        return {"quantize": _own_quantize, "mxfp4": _own_mxfp4, "grouped": _own_grouped, "wgrad": _own_wgrad,
                "grouped_mxfp4": _own_grouped_mxfp4}[state["op"]](state)
    return {"quantize": _plain_quantize, "mxfp4": _plain_mxfp4, "grouped": _plain_grouped, "wgrad": _plain_wgrad,
            "grouped_mxfp4": _plain_grouped_mxfp4}[state["op"]](state)


# ----------------------------------------------------------------- the work and the exact values

def _used(case):
    """Experts with at least one of T rows, as a router without preferences would give them."""
    G = case["G"]
    return max(1, round(G * (1 - (1 - 1 / G) ** case["T"])))


def work(case):
    op = case["op"]
    if op == "quantize":
        M, K = case["M"], case["K"]
        size = 4 if case["type"] == "f32" else 2
        # read, 4 bits and scales written, those read again, the values written
        return {"bytes": 2 * (M * K * size + M * K // 2 + M * K // BLOCK), "flops": 4 * M * K}
    out = 4 if case["out"] == "f32" else 2
    if op == "mxfp4":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * (K // 2 + K // BLOCK) + out * M * N, "flops": 2 * M * N * K}
    T, G, N = case["T"], case["G"], case["N"]
    if op == "wgrad":
        return {"bytes": 2 * T * (case["M"] + N) + 4 * G + out * G * case["M"] * N, "flops": 2 * T * case["M"] * N}
    K, used = case["K"], _used(case)
    if op == "grouped":
        return {"bytes": 2 * T * K + 2 * used * N * K + 4 * G + out * T * N, "flops": 2 * T * N * K}
    return {"bytes": (T + used * N) * (K // 2 + K // BLOCK) + 4 * G + out * T * N, "flops": 2 * T * N * K}


def _exact_values(q, s, rows):
    """The values of packed elements from the bits of E2M1: sign, two bits of exponent (bias 1), one
    of fraction; exponent 0 is subnormal."""
    n = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.uint8, device=q.device)
    n[..., 0::2] = q.bitwise_and(15)
    n[..., 1::2] = q.bitwise_right_shift(4)
    n = n.to(torch.float64)
    negative = n >= 8
    n = torch.where(negative, n - 8, n)
    e = torch.floor(n / 2)
    f = (n - 2 * e) / 2
    v = torch.where(e > 0, (1 + f) * torch.exp2(e - 1), f)
    v = torch.where(negative, -v, v)
    scale = torch.exp2(s[..., :rows].to(torch.float64) - 127)
    return v * scale.repeat_interleave(BLOCK, dim=-2).transpose(-1, -2)


def exact(case, seed):
    """The outputs before their last rounding, in fp64."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["X"].to(torch.float64)
        x = x if case["layout"] == "K" else x.t().contiguous()
        b = x.view(case["M"], -1, BLOCK)
        top = b.abs().max(2, keepdim=True).values
        scale = torch.exp2((torch.floor(torch.log2(top.clamp(min=2.0 ** -160))) - EMAX).clamp(-127, 127))
        v = b / scale
        size = v.abs()
        step = torch.where(size < 2, 0.5, torch.where(size < 4, 1.0, 2.0))
        v = torch.sign(v) * (torch.round(size / step) * step).clamp(max=6.0)
        return (v * scale).view(case["M"], case["K"])
    if op == "mxfp4":
        a = _exact_values(s["A"], s["SA"], case["M"])
        return torch.matmul(a, _exact_values(s["B"], s["SB"], case["N"]).t())
    bounds = [0] + s["ends"].cpu().tolist()
    c = torch.zeros(s["C"].shape, dtype=torch.float64, device="cuda")
    for g in range(case["G"]):
        rows = slice(bounds[g], bounds[g + 1])
        if rows.start == rows.stop:
            continue
        if op == "grouped_mxfp4":
            # the rows' bytes and scales alone, and the expert's
            a = _exact_values(s["A"][rows], s["SA"][:, rows], rows.stop - rows.start)
            c[rows] = torch.matmul(a, _exact_values(s["B"][g], s["SB"][g], case["N"]).t())
            continue
        a, b = s["A"][rows].to(torch.float64), s["B"]
        if op == "wgrad":
            c[g] = torch.matmul(a.t(), b[rows].to(torch.float64))
        else:
            w = b[g].to(torch.float64)
            c[rows] = torch.matmul(a, w if case["layout"] == "MN" else w.t())
    return c
