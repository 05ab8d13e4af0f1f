"""sgemm_fp8_quantize against the definition, bit for bit: every step is one
fp32 operation rounded to nearest, so codes and scales have one right value."""
import numpy as np
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import fp8_plain as fp

pytestmark = pytest.mark.gpu

GROUPS = [(1, 128), (128, 1), (128, 128)]


def _torch_type(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16,
            "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[name]


def _input(rows, cols, xt, seed):
    import torch
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((1, cols)) * 2)
    return torch.from_numpy(x.astype(np.float32)).to(_torch_type(xt))


def _check(x, group, fmt, pad_x=0, off_x=0, pad_q=0, off_q=0, pad_s=0):
    """x: CPU tensor.  Runs on views inside larger buffers; checks nothing else changed."""
    import torch
    rows, cols = x.shape
    want_c, want_s = fp.quantize(x.float().numpy(), group, fmt)
    bx = torch.zeros(rows * (cols + pad_x) + off_x + 8, dtype=x.dtype, device="cuda")
    X = bx[off_x: off_x + rows * (cols + pad_x)].view(rows, cols + pad_x)[:, :cols]
    X.copy_(x.cuda())
    bq = torch.full((rows * (cols + pad_q) + off_q + 16,), 0x55, dtype=torch.uint8, device="cuda")
    Q = bq[off_q: off_q + rows * (cols + pad_q)].view(rows, cols + pad_q)[:, :cols]
    bs = torch.full((want_s.shape[0], want_s.shape[1] + pad_s), -7.0, device="cuda")
    S = bs[:, : want_s.shape[1]]
    st = sg.sgemm_fp8_quantize(rows, cols, X.data_ptr(), sg._type_of(x.dtype), cols + pad_x, *group,
                               Q.data_ptr(), sg._type_of(_torch_type(fmt)), cols + pad_q,
                               S.data_ptr(), want_s.shape[1] + pad_s, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert st == 0
    assert np.array_equal(S.cpu().numpy().view(np.uint32), want_s.view(np.uint32))
    got = Q.cpu().numpy()
    nan = np.isnan(fp.decode(want_c, fmt))
    assert np.array_equal(np.isnan(fp.decode(got, fmt)), nan)
    assert np.array_equal(got[~nan], want_c[~nan])
    # guards: around the codes, in their rows' gaps and in the scales' gaps
    mask = torch.ones_like(bq, dtype=torch.bool)
    mask[off_q: off_q + rows * (cols + pad_q)].view(rows, cols + pad_q)[:, :cols] = False
    assert bool((bq[mask] == 0x55).all())
    if pad_s:
        assert bool((bs[:, want_s.shape[1]:] == -7.0).all())


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 129), (33, 127), (128, 256), (129, 131),
                                       (256, 512), (300, 1000)])
def test_matches_the_definition(group, xt, fmt, rows, cols):
    _check(_input(rows, cols, xt, rows * 1000 + cols), group, fmt)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("xt", ["f32", "bf16"])
@pytest.mark.parametrize("pads", [(4, 0, 4, 0, 0), (4, 4, 12, 4, 3), (1, 0, 0, 0, 0), (0, 1, 0, 0, 5),
                                  (0, 0, 3, 1, 0), (0, 0, 0, 2, 1)])
def test_strides_and_alignment(group, xt, pads):
    px, ox, pq, oq, ps = pads
    _check(_input(137, 260, xt, 5), group, "e4m3", px, ox, pq, oq, ps)


@pytest.mark.parametrize("group", GROUPS)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_special_values(group, fmt):
    x = _input(260, 300, "f32", 9)
    x[:128, :128] = 0.0                      # a group of zeros
    x[128:, 128:256] *= 1e-41                # subnormal inputs: the scale's floor
    x[3, 5] = float("inf")
    x[200, 299] = float("-inf")
    x[7, 130] = float("nan")
    x[130:258, 260] = float("nan")           # a 128 x 1 group without a finite value
    x[9, :] = float("inf")                   # a row without one
    x[11, 140] = 3.4e38                      # the largest magnitudes
    x[12, 141] = -0.0
    _check(x, group, fmt)


def test_ties_go_to_even():
    import torch
    # amax 448: scale 1, so the codes are the roundings of the values themselves
    v = torch.tensor([448.0, 1.0625, 1.1875, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -432.0, -416.0])
    x = torch.zeros(1, 128)
    x[0, : v.numel()] = v
    q, s = sg.fp8_quantize(x.cuda())
    assert s.item() == 1.0
    want = [448.0, 1.0, 1.25, 16.0, 20.0, 0.0, 2.0 ** -8, -448.0, -416.0]
    assert q[0, : v.numel()].float().cpu().tolist() == want


def test_another_stream_and_empty_shapes():
    import torch
    s = torch.cuda.Stream()
    x = _input(64, 256, "f32", 1).cuda()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q, sc = sg.fp8_quantize(x)
    s.synchronize()
    want_c, want_s = fp.quantize(x.cpu().numpy(), (1, 128), "e4m3")
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want_c)
    assert np.array_equal(sc.cpu().numpy(), want_s)
    for shape in ((0, 128), (4, 0)):
        q, sc = sg.fp8_quantize(torch.empty(shape, device="cuda"))
        assert q.shape == shape
