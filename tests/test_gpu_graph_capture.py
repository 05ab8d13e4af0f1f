"""Calls captured into graphs on a stream that the library has not seen before: the
workspaces are not the graph's, so that other graphs and plain calls on the stream
may use them after it."""
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg
from tests.test_gpu_moe import Layer, _x

pytestmark = pytest.mark.gpu


def _calls():
    """Calls with a workspace, small and large: (call, buffer, result on a warm stream)."""
    layer = Layer(1024, 512, 16, seed=21)
    g = torch.Generator(device="cuda").manual_seed(5)
    made = []
    for T, topk in ((1, 2), (40, 4)):
        x = _x(T, 1024, "float32", seed=T)
        y = torch.empty_like(x)
        out = dict(logits=torch.empty(T, 16, device="cuda"), indices=torch.empty(T, topk, device="cuda", dtype=torch.int32),
                   weights=torch.empty(T, topk, device="cuda"))
        made.append((lambda x=x, y=y, topk=topk, out=out: sg.moe(
            x, *(layer.dev[n] for n in ("router", "gate", "s_gate", "up", "s_up", "down", "s_down")), topk, y=y, **out), y))
    for M, N, K in ((100, 200, 1001), (1500, 1100, 1301)):        # rows of codes off 16 bytes: copied first
        qa, sa = sg.fp8_quantize(torch.randn((M, K), generator=g, device="cuda"))
        qb, sb = sg.fp8_quantize(torch.randn((N, K), generator=g, device="cuda"), (128, 128))
        C = torch.empty((M, N), device="cuda")
        made.append((lambda qa=qa, sa=sa, qb=qb, sb=sb, C=C: sg.fp8_gemm(qa, sa, qb, sb, C), C))
    for n in (300, 1100):
        A, B = (torch.randn((n, n), generator=g, device="cuda") for _ in range(2))
        C = torch.empty((n, n), device="cuda")
        made.append((lambda A=A, B=B, C=C: sg.gemm(A, B, C, path=sg.PATH_3XTF32), C))
    with torch.cuda.stream(torch.cuda.Stream()):
        want = []
        for call, out in made:
            call()
            torch.cuda.synchronize()
            want.append(out.clone())
    torch.cuda.synchronize()
    return [(call, out, w) for (call, out), w in zip(made, want)]


def _capture(call, s):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    return g


def _right(run, out, want):
    out.fill_(float("nan"))
    torch.cuda.synchronize()
    run()
    torch.cuda.synchronize()
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    assert torch.equal(out, want)


def test_graphs_and_calls_on_a_stream_first_used_under_capture():
    calls = _calls()
    s = torch.cuda.Stream()
    graphs = [_capture(call, s) for call, _, _ in calls]          # (the workspaces grow between them)
    for _ in range(2):
        for g, (call, out, want) in zip(graphs, calls):
            _right(g.replay, out, want)
    with torch.cuda.stream(s):
        for call, out, want in calls:
            _right(call, out, want)
    for i in range(len(graphs)):                                  # graphs go, the others and the calls stay
        graphs[i] = None
        torch.cuda.synchronize()
        for g, (call, out, want) in zip(graphs, calls):
            if g is not None:
                _right(g.replay, out, want)
        with torch.cuda.stream(s):
            _right(*calls[i])


def test_a_second_capture_grows_the_workspace_of_plain_calls():
    calls = _calls()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _right(*calls[0])
        _right(*calls[2])
    graphs = [_capture(calls[i][0], s) for i in (1, 3, 5)]
    for _ in range(2):
        for g, i in zip(graphs, (1, 3, 5)):
            _right(g.replay, *calls[i][1:])
        with torch.cuda.stream(s):
            for c in calls:
                _right(*c)


def test_a_graph_after_larger_calls_on_its_stream():
    calls = _calls()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for i in (0, 2, 4):
            _right(*calls[i])
    graphs = [_capture(calls[i][0], s) for i in (0, 2, 4)]        # their workspaces were there before
    with torch.cuda.stream(s):
        for i in (1, 3, 5):                                       # larger ones
            _right(*calls[i])
        scribble = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(8)]
    for g, i in zip(graphs, (0, 2, 4)):
        _right(g.replay, *calls[i][1:])
    del scribble
