"""sgemm_q4 with x near the largest numbers and small scales: sums that are finite with their scales
on, and would not be without them."""
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp
from tests import q4_plain as qp
from tests.test_gpu_q4 import ACT, _dtype

pytestmark = pytest.mark.gpu


def _operands(M, N, K, group, zeros, x, seed=0):
    """Rows of x alternate between numbers about 1 and ones up to 2^127 or 2^128, all of a sign;
    codes that are all 15 or all 0, group by group."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed + M + 3 * N + 7 * K)
    X = torch.rand((M, K), device="cuda", generator=gen) + 0.5
    X[0::2] *= 2.0 ** 127 * 1.3
    X = X.to(_dtype(x))
    groups = -(-K // group)
    high = torch.rand((N, groups), device="cuda", generator=gen) < 0.5
    code = torch.where(high, 15, 0).repeat_interleave(group, 1)[:, :K + K % 2]
    if K % 2:
        code[:, K:] = 0
    half = (K + 1) // 2
    q = torch.zeros((N, -(-half // 16) * 16), device="cuda", dtype=torch.uint8)[:, :half]
    q.copy_(code[:, 0::2] + 16 * code[:, 1::2])
    s = torch.rand((groups, N), device="cuda", generator=gen) + 0.5
    z = torch.where(high.t(), 0, 15).to(torch.uint8).contiguous() if zeros else None
    if z is not None:
        z[:, ::3] = 6
    return X, q, s, z


def _check(X, q, s, z, group, c, more=(), act=None):
    """The product, and that the rows about 1 come out as they do without the large ones."""
    import torch
    K = X.shape[1]
    C = sg.q4_gemm(X, q, s, None, z, *more, group=group, activation=act, dtype=_dtype(c))
    w = qp.values(q, s, z, group, K)
    name = {v: k for k, v in ACT.items()}.get(act)
    want, e = qp.gated(X, w, qp.values(*more, group, K), group, name) if more else qp.product(X, w, group)
    fp.close("c", C, want, e + (2.0 ** -24 if c == "f32" else fp.BF16) * (want.abs() + e) + fp.TINY)
    small = X.clone()
    small[0::2] = 1.0
    again = sg.q4_gemm(small, q, s, None, z, *more, group=group, activation=act, dtype=_dtype(c))
    assert torch.equal(C[1::2], again[1::2])
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0


@pytest.mark.parametrize("x,c", [("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("M", [1, 3, 12, 30, 64, 70])
def test_sums_past_the_largest_number(M, group, zeros, x, c):
    """In every width of columns, with sums cut over warps and clusters, and ends inside a group."""
    for N, K in ((70, 516), (40, 9001)):
        X, q, s, z = _operands(M, N, K, group, zeros, x)
        # a whole row: 9001 * 15 * 1.5 * 2^128.4 at most, times 2^-22
        _check(X, q, s * 2.0 ** -22, z, group, c)


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
def test_gated(act, x):
    X, q, s, z = _operands(5, 50, 700, 64, True, x)
    _, q2, s2, z2 = _operands(5, 50, 700, 64, True, x, 1)
    # (g of a few units at most)
    _check(X, q, s * 2.0 ** -140, z, 64, "f32", (q2, s2 * 2.0 ** -126, z2), ACT[act])


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_largest_numbers(x):
    """Every x the type's largest number, of each sign, and one infinity, which stays one."""
    import torch
    X, q, s, z = _operands(4, 33, 300, 128, False, x)
    X[:] = torch.finfo(_dtype(x)).max
    X[1] = -X[1]
    s = s * 2.0 ** -20
    C = sg.q4_gemm(X, q, s, dtype=torch.float32)
    w = qp.values(q, s, None, 128, 300)
    want, e = qp.product(X, w, 128)
    fp.close("c", C, want, e + 2.0 ** -24 * (want.abs() + e))
    X[2, 140] = float("inf")
    D = sg.q4_gemm(X, q, s, dtype=torch.float32)
    assert torch.equal(D[[0, 1, 3]], C[[0, 1, 3]])
    assert torch.equal(D[2].double(), torch.sign(w[:, 140]) * float("inf"))
