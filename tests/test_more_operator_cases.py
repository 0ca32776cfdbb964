"""perf/more_operators.py calls the library on torch's current stream: the calls it makes, on the CPU
against a stand-in; its plain form against its fp64 values; and every operator on a side stream and in
a captured graph on the GPU."""
import importlib.util
import os
import random

import pytest
import torch

import lds_staged_matrix_amd as lsm

CASES = [dict(op="quantize", M=5, K=160, type="bf16", layout="K"), dict(op="quantize", M=40, K=96, type="f32", layout="MN"),
         dict(op="mxfp4", M=3, N=264, K=320, out="bf16"), dict(op="mxfp4", M=300, N=264, K=320, out="f32"),
         dict(op="grouped", T=70, G=4, N=264, K=136, type="bf16", out="bf16", layout="K"),
         dict(op="grouped", T=300, G=4, N=264, K=136, type="f16", out="f32", layout="MN"),
         dict(op="wgrad", T=300, G=4, M=136, N=264, type="bf16", out="f32"),
         dict(op="grouped_mxfp4", T=300, G=4, N=264, K=320, out="f16")]
NAMES = [f"{c['op']}-{c.get('out') or c['type']}-{c.get('layout', '')}" for c in CASES]
CALLS = dict(quantize=2)


@pytest.fixture
def cases():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "more_operators.py")
    spec = importlib.util.spec_from_file_location("more_operator_cases", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


class Recorder:
    """The package's names, with entry points that record their last argument."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.endswith("_run"):
            def call(*args):
                self.streams.append(args[-1])
                return lsm.GEMM_OK
            return call
        return getattr(lsm, name)


@pytest.mark.parametrize("case", CASES, ids=NAMES)
def test_calls_pass_the_current_stream(cases, monkeypatch, case):
    handle = 0x5ead
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: handle, raising=False)
    recorder = Recorder()
    cases._library, cases.own = (recorder, None), True
    t = torch.zeros(4, 4, 4)
    cases.run(dict(case, X=t, Q=t, S=t, Y=t, A=t, B=t, C=t, SA=t, SB=t, ends=t))
    assert recorder.streams == [handle] * CALLS.get(case["op"], 1)


def test_cases_are_valid(cases):
    """Listed and drawn cases have the sizes that the entry points ask for."""
    rng = random.Random(3)
    listed = cases.listed()
    assert len({c["name"] for c in listed}) == len(listed)
    for c in listed + [cases.draw(rng) for _ in range(200)]:
        if c["op"] in ("mxfp4", "grouped_mxfp4", "quantize"):
            assert c["K"] % 32 == 0
        if c["op"] == "grouped":
            assert c["K"] % 8 == 0 and (c["layout"] == "K" or c["N"] % 8 == 0)
        if c["op"] == "wgrad":
            assert c["M"] % 8 == 0 and c["N"] % 8 == 0
        assert all(v > 0 for v in cases.work(c).values())


def bits(out):
    return out.contiguous().view(torch.uint8).clone()


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=NAMES)
def test_both_forms_against_fp64(cases, case):
    """The plain form and the library's, each within its type's rounding and the fp32 sums of the
    values in fp64."""
    exact = cases.exact(case, 5)
    kind = cases.TYPES[case.get("out") or case["type"]]
    half = torch.finfo(kind).eps / 2
    terms = {"quantize": 0, "wgrad": case.get("T")}.get(case["op"], case.get("K"))
    # |sum| <= sizes, taken as the largest of the operands' sums of squares (Cauchy-Schwarz)
    state = cases.prepare(case, 5)
    if terms:
        if case["op"] in ("mxfp4", "grouped_mxfp4"):
            a = cases._values(state["A"], state["SA"], case.get("M") or case["T"]).double()
            b = cases._values(state["B"], state["SB"], case["N"]).double()
        else:
            a, b = state["A"].double(), state["B"].double()
        along = 0 if case["op"] == "wgrad" else -1
        alongb = 0 if case["op"] == "wgrad" else -2 if case.get("layout") == "MN" else -1
        size = float(a.square().sum(along).max().sqrt() * b.square().sum(alongb).max().sqrt())
        sums = size * ((terms + 1) * 2.0 ** -24 + (2.0 ** -21 * (terms / 128 + 8) if "mxfp4" in case["op"] else 0))
    else:
        sums = 0.0
    for own in (False, True):
        cases.own = own
        got = cases.run(cases.prepare(case, 5)).double()
        assert got.shape == exact.shape
        assert torch.all((got - exact).abs() <= exact.abs() * half + sums * (1 + half)), own


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=NAMES)
def test_side_stream_and_graph(cases, case):
    """The inputs are written, the operator run and its output read on one side stream, which waits
    behind a long kernel; and a captured call replays."""
    cases.own = True
    state, other = cases.prepare(case, 1), cases.prepare(case, 2)
    out = cases.run(state)
    want = bits(out)
    out.zero_()
    inputs = {k: v for k, v in state.items() if isinstance(v, torch.Tensor)}
    kept = {k: v.clone() for k, v in inputs.items()}
    torch.cuda.synchronize()
    side, busy = torch.cuda.Stream(), torch.ones(4096, 4096, device="cuda")
    for v in inputs.values():
        v.zero_()
    torch.cuda.synchronize()
    print("CASE side stream", case, flush=True)
    with torch.cuda.stream(side):
        for _ in range(20):
            busy @ busy
        for k, v in inputs.items():
            v.copy_(kept[k])
        got = bits(cases.run(state))
    side.synchronize()
    assert torch.equal(got, want)

    print("CASE graph", case, flush=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cases.run(state)
    for _ in range(3):
        out.zero_()
        cases.run(other)                # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), want)
