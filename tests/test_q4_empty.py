"""Gated 4-bit products with a size of zero: a tensor without elements has no address, so the second
matrix' absence does not say that there is one matrix (no GPU: nothing is launched)."""
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg
from tests.test_fp8_tensor_calls import Tensor, calls  # noqa: F401  (a fixture)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_fp32_gemm_05_gb300 import build
    build.build()
    sg.load()


P = 1 << 20      # never dereferenced
F32, BF16 = sg.TYPE_F32, sg.TYPE_BF16


@pytest.mark.parametrize("act", [sg.ACT_NONE, sg.ACT_RELU, sg.ACT_SILU, sg.ACT_GELU])
@pytest.mark.parametrize("M,N,X,C", [(0, 20, 0, 0), (3, 0, P, 0), (0, 0, 0, 0)])
def test_of_nothing_is_ok(M, N, X, C, act):
    for codes in (0, P):
        assert sg.sgemm_q4(M, N, 300, X, BF16, 300, codes, codes, codes, codes, codes, codes, 160, 20, 64, act, C, BF16, 20) == 0


def test_one_matrix_with_an_activation_is_refused_whatever_its_size_but_zero():
    args = [3, 20, 300, P, BF16, 300, P, P, P, 0, 0, 0, 160, 20, 64, sg.ACT_SILU, P, BF16, 20]
    assert sg.sgemm_q4(*args) == -16
    args[15] = 4
    assert sg.sgemm_q4(*args) == -16
    args[0] = 0
    assert sg.sgemm_q4(*args) == -16


@pytest.mark.skipif(torch.cuda.is_available(), reason="writes to an address of no buffer")
def test_empty_sums_are_not_refused():
    """(without a GPU the zeros cannot be written: an error of CUDA, not of an argument)"""
    assert sg.sgemm_q4(3, 20, 0, 0, BF16, 1, 0, 0, 0, 0, 0, 0, 1, 20, 64, sg.ACT_SILU, P, BF16, 20) == sg.SGEMM_ERR_CUDA


def test_what_the_library_gets_of_an_empty_gated_product(calls):
    u8 = lambda *s: Tensor(torch.zeros(s, dtype=torch.uint8))  # noqa: E731
    f32 = lambda *s: Tensor(torch.zeros(s))  # noqa: E731
    sg.q4_gemm(f32(3, 64), u8(0, 32), f32(1, 0), f32(3, 0), Q2=u8(0, 32), S2=f32(1, 0))
    name, args = calls.pop()
    assert name == "sgemm_q4" and args[:3] == (3, 0, 64) and not args[9] and args[15] == sg.ACT_SILU


@pytest.mark.gpu
@pytest.mark.parametrize("act", [None, sg.ACT_GELU, sg.ACT_NONE])
def test_gated_products_of_nothing(act):
    e = lambda *s, d=torch.float32: torch.empty(s, device="cuda", dtype=d)  # noqa: E731
    u8 = torch.uint8
    assert sg.q4_gemm(e(0, 64), e(8, 32, d=u8), e(1, 8), Q2=e(8, 32, d=u8), S2=e(1, 8), activation=act).shape == (0, 8)
    assert sg.q4_gemm(e(3, 64), e(0, 32, d=u8), e(1, 0), Z=e(1, 0, d=u8), Q2=e(0, 32, d=u8), S2=e(1, 0), Z2=e(1, 0, d=u8),
                      activation=act).shape == (3, 0)
    for dtype in (torch.float32, torch.bfloat16):
        c = torch.full((3, 8), 7.0, device="cuda", dtype=dtype)
        sg.q4_gemm(e(3, 0), e(8, 0, d=u8), e(0, 8), c, Q2=e(8, 0, d=u8), S2=e(0, 8), activation=act)
        assert bool((c == 0).all())
