"""perf/operators.py calls the library on torch's current stream: the calls it makes, on the CPU
against a stand-in, and every operator on a side stream and in a captured graph on the GPU."""
import importlib.util
import os

import pytest
import torch

import lds_staged_matrix_amd as lsm

CASES = [dict(op="norm", M=3, N=130, type="bf16", out="e4m3", residual=True),
         dict(op="norm", M=5, N=64, type="f16", out="f16", residual=False),
         dict(op="scaled", M=40, N=272, K=256, out="bf16"), dict(op="scaled", M=2, N=272, K=256, out="f32"),
         dict(op="w4", M=2, N=272, K=256, group=64, type="bf16", out="f32", zeros=True),
         dict(op="w4", M=20, N=272, K=256, group=32, type="f16", out="f16", zeros=False)]


@pytest.fixture
def operators():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")
    spec = importlib.util.spec_from_file_location("operator_cases", path)
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


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['op']}-{c['out']}")
def test_calls_pass_the_current_stream(operators, monkeypatch, case):
    handle = 0x5ead
    current = type("Stream", (), {"cuda_stream": handle})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: handle, raising=False)
    recorder = Recorder()
    operators._library, operators.own = (recorder, None), True
    t = torch.zeros(4, 4)
    operators.run(dict(case, X=t, R=t if case.get("residual") else None, H=t if case.get("residual") else None, W=t, Y=t,
                       S=t, A=t, B=t, C=t, SA=t, SB=t, Z=t if case.get("zeros") else None))
    assert recorder.streams in ([current], [handle])


def bits(out):
    """The outputs' bytes."""
    out = out if isinstance(out, dict) else {"C": out}
    return {k: v.contiguous().view(torch.uint8).clone() for k, v in out.items() if v is not None}


def blank(out):
    for v in (out.values() if isinstance(out, dict) else [out]):
        if v is not None:
            v.zero_()


def same(got, want):
    return got.keys() == want.keys() and all(torch.equal(got[k], want[k]) for k in got)


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c['op']}-{c['out']}")
def test_side_stream_and_graph(operators, case):
    """The inputs are written, the operator run and its output read on one side stream, which waits
    behind a long kernel; and a captured call replays."""
    operators.own = True
    state, other = operators.prepare(case, 1), operators.prepare(case, 2)
    out = operators.run(state)
    want = bits(out)
    blank(out)
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
        got = bits(operators.run(state))
    side.synchronize()
    assert same(got, want)

    print("CASE graph", case, flush=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = operators.run(state)
    for _ in range(3):
        blank(out)
        operators.run(other)                # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(bits(out), want)
