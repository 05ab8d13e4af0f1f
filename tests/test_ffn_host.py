"""The gated feed-forward block without a GPU: refusals (nothing is launched), the plan, and
the plain evaluation that the GPU tests compare with, against differences."""
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_fp32_gemm_05_gb300 import build
    build.build()
    sg.load()


P = 1 << 20      # never dereferenced
BF16, E4M3, F32 = sg.TYPE_BF16, sg.TYPE_E4M3, sg.TYPE_F32
BAD = sg.SGEMM_ERR_UNSUPPORTED


@pytest.mark.parametrize("change,want", [
    ({0: -1}, -1), ({0: 2 ** 31}, -1), ({1: -1}, -2), ({2: 2 ** 31 - 1}, -3), ({3: 0}, -4), ({3: P + 1}, -4), ({4: 63}, -5),
    ({5: 0}, -6), ({6: P + 1}, -7), ({7: 63}, -8), ({8: 0}, -9), ({9: 127}, -10), ({10: 4}, -11), ({10: -1}, -11),
    ({11: F32}, -12), ({11: sg.TYPE_E5M2}, -12), ({12: 0}, -13), ({13: 0}, -14), ({12: P + 1}, -13), ({14: 127}, -15),
    ({15: 0}, -16), ({16: P + 1}, -17), ({17: 9}, -18), ({18: 0}, -19), ({19: 127}, -20), ({20: 0}, -21), ({20: P + 1}, -21),
    ({21: 63}, -22), ({1: 0}, BAD), ({3: P + 8}, BAD), ({4: 68}, BAD), ({5: P + 2}, BAD), ({7: 65}, BAD), ({9: 130}, BAD),
    ({18: P + 4}, BAD), ({19: 129}, BAD)])
def test_forward_refusals(change, want):
    codes = any(i in change for i in (15, 16, 17))
    args = [10, 64, 128, P, 64, P, P, 64, P, 128, sg.ACT_SILU, E4M3 if codes else BF16, P, P, 128, P, P, 10, P, 128, P, 64]
    for i, v in change.items():
        args[i] = v
    assert sg.sgemm_ffn(*args) == want


@pytest.mark.parametrize("change,want", [
    ({0: -1}, -1), ({1: 2 ** 31}, -2), ({2: -3}, -3), ({3: 0}, -4), ({4: 63}, -5), ({5: 0}, -6), ({6: 63}, -7), ({7: 0}, -8),
    ({8: P + 1}, -9), ({9: 63}, -10), ({10: 0}, -11), ({11: 127}, -12), ({12: 9}, -13), ({13: F32}, -14), ({14: 0}, -15),
    ({15: 0}, -16), ({16: 127}, -17), ({17: 0}, -18), ({18: P + 1}, -19), ({19: 9}, -20), ({20: 0}, -21), ({21: 0}, -22),
    ({22: P + 1}, -23), ({23: 127}, -24), ({24: 0}, -25), ({25: 63}, -26), ({26: E4M3}, -27), ({28: 0}, -29),
    ({29: P + 2, 26: F32}, -30), ({30: 63}, -31), ({31: 0}, -32), ({32: 127}, -33), ({3: P + 8}, BAD), ({4: 65}, BAD),
    ({6: 66}, BAD), ({9: 68}, BAD), ({11: 129}, BAD), ({20: P + 8}, BAD), ({23: 132}, BAD)])
def test_backward_refusals(change, want):
    codes = any(i in change for i in (17, 18, 19))
    args = [10, 64, 128, P, 64, P, 64, P, P, 64, P, 128, sg.ACT_GELU, E4M3 if codes else BF16, P, P, 128, P, P, 10, P, P, P,
            128, P, 64, BF16, 0, P, P, 64, P, 128]
    for i, v in change.items():
        args[i] = v
    assert sg.sgemm_ffn_backward(*args) == want


def test_of_nothing_is_ok():
    assert sg.sgemm_ffn(0, 64, 128, 0, 64, 0, 0, 64, 0, 128, 1, BF16, 0, 0, 128, 0, 0, 1, 0, 128, 0, 64) == 0
    assert sg.sgemm_ffn(4, 0, 128, 0, 1, 0, 0, 1, 0, 128, 1, BF16, 0, 0, 128, 0, 0, 1, 0, 128, 0, 1) == 0
    assert sg.sgemm_ffn_backward(0, 64, 0, 0, 64, 0, 64, 0, 0, 64, 0, 1, 1, BF16, 0, 0, 1, 0, 0, 1, 0, 0, 0, 1, 0, 64, BF16,
                                 1, 0, 0, 64, 0, 1) == 0


def test_plan():
    tiles = {(256, 256), (128, 128), (128, 64)}
    seen = {}
    for T in (1, 17, 50, 100, 200, 777, 1000, 4000, 20000):
        for D, F in ((64, 64), (300, 2000), (1000, 2500), (2000, 9000), (4096, 8192), (8192, 512), (100, 20000)):
            st, p = sg.sgemm_ffn_plan(T, D, F)
            assert st == 0
            for name, (rows, cols, split) in p.items():
                assert (rows, cols) in tiles
                seen.setdefault(name, set()).add((rows, cols, split))
                if split > 1:                  # whole sums are left, and clusters are resident at once
                    n, k = (D, F) if name == "down" else (D, 2 * F)
                    assert name in ("down", "dx") and (rows, cols) != (256, 256)
                    assert -(-T // rows) * -(-n // cols) * split <= 152 and 4 * split <= -(-k // 64) + 1
            if p["dx"][2] == 0:
                assert p["dx"][:2] == p["weights"][:2]
            # groups of 128 kept columns lie in one tile
            assert sg.sgemm_ffn_plan(T, D, F, E4M3)[1]["gated"] == (256, 256, 1)
    assert {t[:2] for s in seen.values() for t in s} == tiles
    assert {t[2] for t in seen["down"]} == {1, 2, 4, 8} and len({t[2] for t in seen["dx"]}) > 2
    assert {t[2] for n in ("gated", "slope", "weights") for t in seen[n]} == {1}
    assert sg.sgemm_ffn_plan(8192, 4096, 8192)[1]["gated"] == (256, 256, 1)
    for args, want in (((0, 1, 1), -1), ((1, 0, 1), -2), ((1, 1, 0), -3), ((1, 1, 1, BF16, 0), -5)):
        assert sg.sgemm_ffn_plan(*args)[0] == want


@pytest.mark.parametrize("act", fp.ACTS)
def test_plain_gradients_against_differences(act):
    gen = torch.Generator().manual_seed(0)
    T, D, F = 5, 7, 9
    x, gate, up, down, dy = (torch.randn(s, generator=gen, dtype=torch.float64)
                             for s in ((T, D), (F, D), (F, D), (D, F), (T, D)))
    grads = fp.backward(dy, x, gate, up, down, x @ gate.t(), x @ up.t(), act)
    at = {"dx": x, "dgate": gate, "dup": up, "ddown": down}

    def loss():
        return float((dy * ((fp.act(act, x @ gate.t()) * (x @ up.t())) @ down.t())).sum())

    for n, t in at.items():
        for i in range(0, t.numel(), 5):
            flat = t.view(-1)
            old = float(flat[i])
            flat[i] = old + 1e-6
            high = loss()
            flat[i] = old - 1e-6
            low = loss()
            flat[i] = old
            # (relu's corner is not within 1e-6 of these values)
            assert abs((high - low) / 2e-6 - float(grads[n][0].reshape(-1)[i])) < 1e-6 * (1 + abs(high))


def test_plain_activations():
    g = torch.linspace(-8, 8, 101, dtype=torch.float64)
    assert torch.allclose(fp.act("silu", g), torch.nn.functional.silu(g))
    assert torch.allclose(fp.act("gelu", g), torch.nn.functional.gelu(g, approximate="tanh"))
    for a in ("silu", "gelu"):
        assert float(fp.slope(a, g).abs().max()) < 1.13
