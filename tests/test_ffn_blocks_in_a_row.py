"""What a block's calls return may be the next block's input: rows on 16 bytes whatever the width."""
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp
from tests.test_fp8_tensor_calls import Tensor, calls  # noqa: F401  (a fixture)

BF16 = torch.bfloat16


def _padded(rows, cols):
    return torch.zeros(rows, -(-cols // 8) * 8, dtype=BF16)[:, :cols]


@pytest.mark.parametrize("D", [1, 7, 40, 1001])
@pytest.mark.parametrize("T", [1, 6])
def test_new_results(calls, monkeypatch, T, D):  # noqa: F811
    F, new = 24, sg._new
    monkeypatch.setattr(sg, "_new", lambda *a, **k: Tensor(new(*a, **k)))
    x, gate, up, down = (Tensor(t) for t in (_padded(T, D), _padded(F, D), _padded(F, D), _padded(D, F)))
    kept = tuple(Tensor(_padded(T, F)) for _ in range(2))
    h, scratch = Tensor(_padded(T, F)), tuple(Tensor(_padded(T, F)) for _ in range(3))
    y, _ = sg.ffn(x, gate, up, down, h=h, kept=kept)
    dx, *_ = sg.ffn_backward(x, x, gate, up, down, kept, scratch=scratch)
    for t in (y, dx):
        assert t.shape == (T, D) and t.stride()[1] == 1 and t.stride()[0] % 8 == 0
        assert D % 8 or t.is_contiguous()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 50])
@pytest.mark.parametrize("D", [39, 64])
def test_two_blocks(T, D):
    """Two blocks forward and backward, each call's input as the last one returned it, against buffers given."""
    F = 100
    gen = torch.Generator(device="cuda").manual_seed(T + D)
    x, dy = (fp.matrix(gen, T, D) for _ in range(2))
    w = [[fp.matrix(gen, *s, 0.2) for s in ((F, D), (F, D), (D, F))] for _ in range(2)]
    y0, k0 = sg.ffn(x, *w[0], keep=BF16)
    y1, k1 = sg.ffn(y0, *w[1], keep=BF16)
    given = sg.ffn(y0, *w[1], y=torch.empty((T, D), device="cuda", dtype=BF16), keep=BF16)[0]
    assert torch.equal(y1, given)
    assert sg.ffn(sg.ffn(x, *w[0])[0], *w[1])[0].shape == (T, D)
    d1 = sg.ffn_backward(dy, y0, *w[1], k1)
    d0 = sg.ffn_backward(d1[0], x, *w[0], k0)
    again = sg.ffn_backward(dy, y0, *w[1], k1, dx=torch.empty((T, D), device="cuda", dtype=BF16))
    assert torch.equal(d1[0], again[0]) and all(bool(t.isfinite().all()) for t in d0)
    fp.close("y", y1, *fp.forward(y0, *w[1], "silu")["y"])
