"""Infinities and NaN in a block of few tokens of which nothing is kept (products of few rows, the second
of which reads what the first made of them), against the definition."""
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp
from tests.test_gpu_ffn import ACT, _inputs

pytestmark = pytest.mark.gpu

SIZES = [(96, 300), (101, 333), (4096, 1000), (200, 9001)]


def _copy(t):
    """With rows on 16 bytes."""
    import torch
    full = torch.zeros((t.shape[0], -(-t.shape[1] // 8) * 8), device="cuda", dtype=t.dtype)[:, :t.shape[1]]
    full.copy_(t)
    return full


def _same_kind(name, got, want):
    """The same infinities and NaN, and nothing else where want has them."""
    import torch
    bad = ~want.isfinite()
    assert torch.equal(bad, ~got.isfinite()), name
    same = (got.double() == want) | (got.isnan() & want.isnan())
    assert bool(same[bad].all()), name


@pytest.mark.parametrize("T", [2, 9, 16])
@pytest.mark.parametrize("D,F", SIZES)
def test_a_bad_token(T, D, F):
    """Its row is bad in y, as the definition has it; the others are bit for bit what they are without it."""
    import torch
    _, x, gate, up, down = _inputs(T, D, F)
    for act in ("silu", "gelu", "relu", "none"):
        clean = sg.ffn(x, gate, up, down, ACT[act])[0]
        for value in ("nan", "inf", "-inf"):
            for at in (0, D - 1):
                bad = _copy(x)
                bad[1, at] = float(value)
                h = torch.zeros((T, -(-F // 8) * 8), device="cuda", dtype=torch.bfloat16)[:, :F]
                y = sg.ffn(bad, gate, up, down, ACT[act], h=h)[0]
                others = [t for t in range(T) if t != 1]
                assert torch.equal(y[others], clean[others])
                g, u = (bad[1:2].double() @ w.double().t() for w in (gate, up))
                a = fp.act(act, g)
                _same_kind("h", h[1:2], a * u)
                _same_kind("y", y[1:2], h[1:2].double() @ down.double().t())
                assert not bool(y[1].isfinite().any())
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0


@pytest.mark.parametrize("T", [1, 5, 16])
@pytest.mark.parametrize("D,F", SIZES)
def test_a_bad_weight(T, D, F):
    """In the last column of gate, up or down, which the sums' ends reach: its own column of h, or of y."""
    import torch
    _, x, gate, up, down = _inputs(T, D, F)
    x[:, D - 1] = 2.0
    clean_h = torch.zeros((T, -(-F // 8) * 8), device="cuda", dtype=torch.bfloat16)[:, :F]
    clean = sg.ffn(x, gate, up, down, h=clean_h)[0]
    for i in range(2):
        for value in ("inf", "-inf", "nan"):
            w = [_copy(t) for t in (gate, up)]
            w[i][7, D - 1] = float(value)
            h = _copy(clean_h)
            sg.ffn(x, *w, down, h=h)
            others = [n for n in range(F) if n != 7]
            assert torch.equal(h[:, others], clean_h[:, others])
            g, u = (x.double() @ t.double().t() for t in w)
            _same_kind("h", h, fp.act("silu", g) * u)
    bad = _copy(down)
    bad[3, F - 1] = float("inf")
    y = sg.ffn(x, gate, up, bad)[0]
    others = [n for n in range(D) if n != 3]
    assert torch.equal(y[:, others], clean[:, others])
    assert torch.equal(y[:, 3].double(), torch.sign(clean_h[:, F - 1].double()) * float("inf"))
