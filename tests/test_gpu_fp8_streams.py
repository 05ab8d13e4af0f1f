"""The 8-bit tensor calls on a stream that is given: what they allocate is that stream's."""
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg
from tests.test_gpu_moe import Layer, _x

pytestmark = pytest.mark.gpu


def _stream_of(t):
    """The stream that torch's allocator keeps a tensor's memory for."""
    at = t.data_ptr()
    for segment in torch.cuda.memory_snapshot():
        if segment["address"] <= at < segment["address"] + segment["total_size"]:
            return segment["stream"]
    raise AssertionError("not in the allocator")


@pytest.mark.parametrize("form", ["object", "address"])
def test_new_buffers_belong_to_the_stream_of_the_call(form):
    s = torch.cuda.Stream()
    given = s if form == "object" else s.cuda_stream
    layer = Layer(256, 128, 4)
    x = _x(8, 256, "float32")
    want_q = sg.fp8_quantize(x, (128, 128))
    want = layer.run(x, 2, True)
    torch.cuda.synchronize()
    got_q = sg.fp8_quantize(x, (128, 128), stream=given)
    got = layer.run(x, 2, True, stream=given)
    s.synchronize()
    for a, b in zip((*want_q, *want), (*got_q, *got)):
        assert _stream_of(a) == torch.cuda.current_stream().cuda_stream
        assert _stream_of(b) == s.cuda_stream
        assert torch.equal(a.float(), b.float())


def test_buffers_that_the_caller_gives_are_taken_as_they_are():
    s = torch.cuda.Stream()
    x = _x(8, 256, "float32")
    Q, S = torch.empty(8, 256, device="cuda", dtype=torch.float8_e5m2), torch.empty(2, 8, device="cuda")
    torch.cuda.synchronize()
    q, sc = sg.fp8_quantize(x, Q=Q, S=S, stream=s)
    assert q is Q and sc is S
    s.synchronize()
    want = sg.fp8_quantize(x, dtype=torch.float8_e5m2)
    assert torch.equal(q.float(), want[0].float()) and torch.equal(sc, want[1])
