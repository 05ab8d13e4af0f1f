"""SiLU and GELU far below zero, where their values are small but normal numbers: in the products of
few rows, on tiles, and in the backward pass' first launch, against 64 bits."""
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp
from tests.test_gpu_q4 import ACT

pytestmark = pytest.mark.gpu

SUBNORMAL = 2.0 ** -149


def _exponent(act, g):
    """v of act(g) = g / (1 + exp(-v))."""
    return g if act == "silu" else 2 * fp.C * (g + fp.A * g ** 3)


def _error(act, g):
    """Of the value, relative: an exponential of v / 2, whose error grows with v, twice; v's own
    roundings; a quotient and three products: 2^-20 (1 + |v|), below -64 cut there."""
    return 2.0 ** -20 * (1 + _exponent(act, g.clamp_min(-64)).abs().clamp_max(200))


def _values(act):
    """bf16 values of g down to where act(g) leaves the normal numbers, and some around zero."""
    import torch
    low = -105.0 if act == "silu" else -11.0
    return torch.cat([torch.linspace(low, 0, 420), torch.linspace(0, 100, 80)]).to(torch.bfloat16).cuda()


def _want(act, g, u, half):
    """(act(g) u, bound) for a result rounded by `half` of it; act itself may be subnormal."""
    c = fp.act(act, g) * u
    return c, (_error(act, g) + 2.0 ** -24 + half) * c.abs() * 1.001 + SUBNORMAL * (4 * u.abs() + 1)


@pytest.mark.parametrize("u", [1.0, -2.0 ** 40])
@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_4_bit_product(act, x, u):
    """g and u are columns of X (of blocks of 128 of their own, so that both are held exactly), by
    matrices whose rows hold one code of one."""
    import torch
    g = _values(act)
    X = torch.zeros((len(g), 192), device="cuda")
    X[:, 0], X[:, 140] = g.float(), u
    X = X.to(torch.bfloat16) if x == "bf16" else X
    q = torch.full((2, 5, 96), 0x88, device="cuda", dtype=torch.uint8)
    q[0, :, 0] = 0x89
    q[1, :, 70] = 0x89
    s = torch.ones((6, 5), device="cuda")
    got = sg.q4_gemm(X, q[0], s, Q2=q[1], S2=s, group=32, activation=ACT[act], dtype=torch.float32)
    want, bound = _want(act, g.double()[:, None].expand(-1, 5), torch.full((len(g), 5), u, device="cuda", dtype=torch.float64), 2.0 ** -24)
    fp.close("c", got, want, bound)


def _block(g, u, D=16, F=40):
    import torch
    x = torch.zeros((len(g), D), device="cuda", dtype=torch.bfloat16)
    x[:, 0], x[:, 9] = g, u
    gate, up = (torch.zeros((F, D), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    gate[:, 0], up[:, 9] = 1.0, 1.0
    return x, gate, up, torch.zeros((D, F), device="cuda", dtype=torch.bfloat16)


@pytest.mark.parametrize("u", [1.0, -2.0 ** 40])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("part", [16, 500])
def test_block(part, act, u):
    """h, which is rounded to bf16, of few tokens and of many."""
    import torch
    for g in _values(act).split(part):
        x, gate, up, down = _block(g, u)
        h = torch.zeros((len(g), 40), device="cuda", dtype=torch.bfloat16)
        y, kept = sg.ffn(x, gate, up, down, ACT[act], h=h, keep=torch.bfloat16 if part > 16 else None)
        want, bound = _want(act, g.double()[:, None].expand(-1, 40), torch.full((len(g), 40), u, device="cuda", dtype=torch.float64), fp.BF16)
        # (bf16's smallest numbers are 2^-133 apart)
        fp.close("h", h, want, bound + 2.0 ** -134)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward(act):
    """h, du and dg of values kept; dh is 1."""
    import torch
    g = _values(act)
    T, D, F = len(g), 16, 40
    kept = (g[:, None].repeat(1, F), torch.full((T, F), 2.0 ** 30, device="cuda", dtype=torch.bfloat16))
    x, gate, up, down = _block(g, 1.0)
    dy = torch.zeros((T, D), device="cuda", dtype=torch.bfloat16)
    dy[:, 0], down[0] = 1.0, 1.0
    dg, du, h = (torch.zeros((T, F), device="cuda", dtype=torch.bfloat16) for _ in range(3))
    sg.ffn_backward(dy, x, gate, up, down, kept, ACT[act], scratch=(dg, du, h))
    g64, one = g.double()[:, None].expand(-1, F), torch.ones((T, F), device="cuda", dtype=torch.float64)
    for name, t, u in (("du", du, one), ("h", h, one * 2.0 ** 30)):
        want, bound = _want(act, g64, u, fp.BF16)
        fp.close(name, t, want, bound + 2.0 ** -134)
    # act' = p + g p (1 - p) v': each of the two to the error above, p off by a subnormal step
    v, dv = _exponent(act, g64), 1.0 if act == "silu" else 2 * fp.C * (1 + 3 * fp.A * g64 * g64)
    p = 1 / (1 + torch.exp(-v))
    size = p + (g64 * p * (1 - p) * dv).abs()
    want = fp.slope(act, g64) * 2.0 ** 30
    bound = (2 * _error(act, g64) * size + SUBNORMAL * 4 * (1 + g64.abs() * dv)) * 2.0 ** 30
    fp.close("dg", dg, want, bound + fp.BF16 * (want.abs() + bound) + 2.0 ** -134)
