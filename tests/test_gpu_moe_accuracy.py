"""How near sgemm_moe's results are to the 64-bit ones, beyond the worst-case bounds
of test_gpu_moe.py: those leave room for a part too few."""
import numpy as np
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import fp8_plain as fp
from tests.test_gpu_moe import Layer, _x

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,D,F,E,topk", [(16, 2048, 512, 4, 2), (4, 4096, 256, 6, 3), (40, 1000, 300, 2, 1)])
def test_bf16_results_are_rounded_once(T, D, F, E, topk):
    """Nearly every bf16 output is the 64-bit result rounded.

    A bf16 step is 2^-8 .. 2^-7 of a value, so an error of r of it turns the rounding with
    probability r / 2^-7.5.  h is held to 2^-19 of each value or better and the sums are in fp32,
    so r is about 2^-20 where terms do not cancel: one output in 2^12.5.  16 times that are
    allowed for sums that cancel.  (One 8-bit part less gives 32 times the rate.)"""
    import torch
    layer = Layer(D, F, E, seed=T)
    x = _x(T, D, "bfloat16")
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(1)).cuda()
    y = layer.run(x, topk, True, logits=logits)[0]
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    want, _, _, _, _ = fp.moe(x.double().cpu().numpy(), None, layer.val["gate"], layer.val["up"], layer.val["down"],
                              topk, True, logits=logits.double().cpu().numpy())
    # (the step to bf16 in one rounding: torch's conversion from float64 goes through fp32)
    step = np.exp2(np.floor(np.log2(np.abs(want))) - 7)
    rounded = np.rint(want / step) * step
    share = np.mean(y.double().cpu().numpy() != rounded)
    assert share <= 2.0 ** -8.5, share


@pytest.mark.parametrize("exponent,s_down", [(0, 1.0), (-30, 1.0), (-48, 2.0 ** -25), (-54, 2.0 ** -12), (30, 2.0 ** 30)])
def test_small_and_large_tokens_keep_their_bits(exponent, s_down):
    """h is of the order of the square of x, so its blocks' powers of two reach 2^-126 while the
    result is a normal number.  Relative to y's norm: 2^-19 of each h at most, sums in fp32 (2^-23
    each, some tens of them, at random): below 2^-18, whatever the size."""
    import torch
    D, F, E, T = 128, 128, 2, 6
    layer = Layer(D, F, E, seed=3)
    s = torch.full((E, 1, 1), 0.0031 * 1.2345678 * s_down, device="cuda")
    codes = layer.dev["down"].float().double().cpu().numpy()
    layer.dev["s_down"], layer.val["down"] = s, codes * s.double().cpu().numpy()
    x = _x(T, D, "float32", seed=2) * 2.0 ** exponent
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(1)).cuda()
    y = layer.run(x, 1, True, logits=logits)[0].double().cpu().numpy()
    want = fp.moe(x.double().cpu().numpy(), None, layer.val["gate"], layer.val["up"], layer.val["down"], 1, True,
                  logits=logits.double().cpu().numpy())[0]
    assert np.abs(want).mean() > 2.0 ** -122
    assert np.linalg.norm(y - want) <= 2.0 ** -18 * np.linalg.norm(want)


def _split_error(v, of_value, of_largest):
    """The documented error of a row of values held in 8-bit parts."""
    blocks = np.pad(np.abs(v), ((0, 0), (0, -v.shape[1] % 128))).reshape(len(v), -1, 128)
    largest = np.repeat(blocks.max(2), 128, axis=1)[:, : v.shape[1]]
    return np.maximum(np.abs(v) * of_value, largest * of_largest)


@pytest.mark.parametrize("dtype,outlier", [("float32", 2.0 ** 18), ("float32", 2.0 ** 24), ("bfloat16", 2.0 ** 12)])
def test_an_outlier_that_meets_weights_of_zero(dtype, outlier):
    """One value of the token far above the others, with gate and up codes of 0 where it is: the
    result hangs on the small values, whose parts' error is relative to the outlier.

    Bound: the parts' documented errors through both products, and (128 + blocks + 16) roundings
    of 2^-23 of the magnitudes for each sum, 2^-20 of h for its function, one rounding of y."""
    import torch
    D, F, E, T = 256, 192, 2, 5
    layer = Layer(D, F, E, seed=4)
    x = _x(T, D, dtype, seed=3)
    x[:, 77] = outlier
    for name in ("gate", "up"):
        layer.val[name][:, :, 77] = 0
        layer.dev[name].view(torch.uint8)[:, :, 77] = 0
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(1)).cuda()
    y = layer.run(x, 1, True, logits=logits)[0].double().cpu().numpy()
    x, which = x.double().cpu().numpy(), logits.argmax(1).tolist()
    dx = _split_error(x, 2.0 ** -19 if dtype == "float32" else 0.0, 2.0 ** -32 if dtype == "float32" else 2.0 ** -22)
    r1, r2 = (128 + D / 128 + 16) * 2.0 ** -23, (128 + F / 128 + 16) * 2.0 ** -23
    for t, e in enumerate(which):
        W, U, V = (layer.val[n][e] for n in ("gate", "up", "down"))
        g, u = W @ x[t], U @ x[t]
        dg, du = (np.abs(m) @ dx[t] + r1 * (np.abs(m) @ np.abs(x[t])) for m in (W, U))
        s = g / (1 + np.exp(-g))
        h = s * u
        dh = 1.1 * dg * np.abs(u) + np.abs(s) * du + 1.1 * dg * du + 2.0 ** -20 * np.abs(h)
        dh += _split_error((np.abs(h) + dh)[None], 2.0 ** -19, 2.0 ** -32)[0]
        want = V @ h
        tol = np.abs(V) @ dh + r2 * (np.abs(V) @ (np.abs(h) + dh))
        tol += (2.0 ** -24 if dtype == "float32" else 2.0 ** -8) * (np.abs(want) + tol)
        assert np.all(np.abs(y[t] - want) <= tol)
