"""4-bit matrices without a GPU: refusals (nothing is launched), how the tensor calls check
their arguments, and the plain evaluation against closed forms."""
import numpy as np
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg
from tests import q4_plain as qp


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_fp32_gemm_05_gb300 import build
    build.build()
    sg.load()


P = 1 << 20      # never dereferenced
F32, BF16, E4M3 = sg.TYPE_F32, sg.TYPE_BF16, sg.TYPE_E4M3
BAD = sg.SGEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,want", [
    ({0: -1}, -1), ({0: 2 ** 31}, -1), ({1: 2 ** 31 - 1}, -2), ({2: 0}, -3), ({2: P + 2}, -3), ({3: E4M3}, -4), ({4: 255}, -5),
    ({5: 16}, -6), ({5: 0}, -6), ({6: 0}, -7), ({7: 127}, -8), ({8: 0}, -9), ({8: P + 2}, -9), ({10: 9}, -11), ({11: P + 2}, -12),
    ({12: E4M3}, -13), ({13: 255}, -14)])
def test_quantize_refusals(change, want):
    args = [10, 256, P, F32, 256, 64, P, 128, P, P, 10, P, F32, 256]
    for i, v in change.items():
        args[i] = v
    assert sg.sgemm_q4_quantize(*args) == want


@pytest.mark.parametrize("change,want", [
    ({0: -1}, -1), ({1: 2 ** 31}, -2), ({2: -1}, -3), ({3: 0}, -4), ({3: P + 1}, -4), ({4: E4M3}, -5), ({5: 299}, -6), ({6: 0}, -7),
    ({7: 0}, -8), ({7: P + 2}, -8), ({10: 0}, -11), ({11: 0}, -12), ({8: 0}, -12), ({12: 149}, -13), ({13: 19}, -14), ({14: 16}, -15),
    ({15: 4}, -16), ({9: 0, 10: 0, 11: 0}, -16), ({16: 0}, -17), ({16: P + 1}, -17), ({17: E4M3}, -18), ({18: 19}, -19),
    ({6: P + 8}, BAD), ({9: P + 4}, BAD), ({12: 168}, BAD)])
def test_product_refusals(change, want):
    args = [3, 20, 300, P, BF16, 300, P, P, P, P, P, P, 160, 20, 64, sg.ACT_SILU, P, BF16, 20]
    for i, v in change.items():
        args[i] = v
    assert sg.sgemm_q4(*args) == want


def test_of_nothing_is_ok():
    assert sg.sgemm_q4_quantize(0, 256, 0, F32, 256, 64, 0, 128, 0, 0, 1) == 0
    assert sg.sgemm_q4(0, 20, 300, 0, BF16, 300, 0, 0, 0, 0, 0, 0, 160, 20, 64, 0, 0, BF16, 20) == 0
    assert sg.sgemm_q4(3, 0, 300, 0, F32, 300, 0, 0, 0, 0, 0, 0, 160, 1, 64, 0, 0, F32, 1) == 0


def test_plain_quantize_closed_form():
    w = np.zeros((1, 130), np.float32)
    w[0, 0], w[0, 1], w[0, 129] = 14.0, -3.0, -7.0
    code, s, z, v = qp.quantize(w, 128, True)
    assert s.T.tolist() == [[2.0, 1.0]] and code[0, 0] == 15 and code[0, 1] == 6 and code[0, 129] == 1
    assert v[0, 0] == 14.0 and v[0, 1] == -4.0 and v[0, 129] == -7.0       # (-1.5 goes to even)
    w[0, 0], w[0, 1], w[0, 129] = 10.0, -5.0, -30.0
    code, s, z, v = qp.quantize(w, 128, False)
    assert s.T.tolist()[0][0] == 1.0 and z.T.tolist() == [[5, 15]] and code[0, :3].tolist() == [15, 0, 5] and code[0, 129] == 0
    assert v[0, 0] == 10.0 and v[0, 1] == -5.0 and v[0, 129] == -30.0


def test_plain_values():
    q = torch.tensor([[0x91, 0x0F]], dtype=torch.uint8)
    s = torch.tensor([[2.0]])
    assert qp.values(q, s, None, 32, 3).tolist() == [[-14.0, 2.0, 14.0]]
    assert qp.values(q, s, torch.tensor([[1]], dtype=torch.uint8), 32, 3).tolist() == [[0.0, 16.0, 28.0]]
