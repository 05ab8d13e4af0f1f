"""GELU's and SiLU's gradients at finite g however far from zero: act' is 0 or 1 there, never NaN."""
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", [sg.ACT_GELU, sg.ACT_SILU])
@pytest.mark.parametrize("T,D,F", [(5, 16, 40), (150, 200, 300), (600, 700, 1500)])
def test_far_from_zero(T, D, F, act):
    """Kept g of -1e10 to the lowest number give the gradients that g = -200 gives; those of 1e10 and
    more dg = dh u."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(T)
    dy, x, gate, up, down = (fp.matrix(gen, *s, 0.2) for s in ((T, D), (T, D), (F, D), (F, D), (D, F)))
    g, u = (torch.randn((T, F), device="cuda", generator=gen).to(torch.bfloat16) for _ in range(2))
    far = torch.tensor([-1e10, -1e30, -1e35, -4e35, -1e36, -1e38, torch.finfo(torch.bfloat16).min], device="cuda")
    where = torch.rand((T, F), device="cuda", generator=gen) < 0.3
    pick = far[torch.randint(0, len(far), (T, F), device="cuda", generator=gen)].to(torch.bfloat16)
    near = torch.where(where, torch.full_like(g, -200.0), g)
    got = sg.ffn_backward(dy, x, gate, up, down, (torch.where(where, pick, g), u), act)
    want = sg.ffn_backward(dy, x, gate, up, down, (near, u), act)
    for a, b in zip(got, want):
        assert bool(a.isfinite().all()) and torch.equal(a, b)
    # the other end: dg = dh u, whatever g is
    scratch = [[torch.zeros((T, F + (-F) % 8), device="cuda", dtype=torch.bfloat16)[:, :F] for _ in range(3)] for _ in range(2)]
    for value, s in zip((200.0, 3e38), scratch):
        sg.ffn_backward(dy, x, gate, up, down, (torch.where(where, torch.full_like(g, value), g), u), act, scratch=tuple(s))
    assert bool(scratch[1][0].isfinite().all()) and torch.equal(scratch[0][0], scratch[1][0])
