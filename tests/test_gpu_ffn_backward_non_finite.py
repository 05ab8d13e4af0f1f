"""Infinities and NaN in the backward pass: what they reach, by the definition, and nothing else."""
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp
from tests.test_gpu_ffn import ACT, _inputs

pytestmark = pytest.mark.gpu

NAMES = ("dx", "dgate", "dup", "ddown")


def _copy(t):
    """With rows on 16 bytes."""
    import torch
    full = torch.zeros((t.shape[0], -(-t.shape[1] // 8) * 8), device="cuda", dtype=t.dtype)[:, :t.shape[1]]
    full.copy_(t)
    return full


@pytest.mark.parametrize("grad", ["bf16", "f32"])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf"])
@pytest.mark.parametrize("where", ["dy", "x", "g", "u", "gate", "down"])
@pytest.mark.parametrize("T,D,F", [(3, 40, 70), (130, 100, 300), (700, 264, 1000)])
def test_one_bad_number(T, D, F, where, value, grad):
    import torch
    dy, x, gate, up, down = (_copy(t) for t in _inputs(T, D, F))
    act = "gelu" if T == 130 else "silu"
    g, u = (t.contiguous() for t in sg.ffn(x, gate, up, down, ACT[act], keep=torch.bfloat16)[1])
    tensors = {"dy": dy, "x": x, "g": g, "u": u, "gate": gate, "down": down}
    kind = torch.bfloat16 if grad == "bf16" else torch.float32
    new = [torch.zeros(s, device="cuda", dtype=kind) for s in ((F, D), (F, D), (D, F))]

    def run():
        out = sg.ffn_backward(dy, x, gate, up, down, (g, u), ACT[act], None, *new)
        return [t.clone() for t in out]

    clean = run()
    rows, cols = tensors[where].shape
    # (the last column is in every tail; row 1 of the tokens or of the matrix)
    tensors[where][1, cols - 1] = float(value)
    got = run()
    want = fp.backward(dy, x, gate, up, down, g.double(), u.double(), act)
    for name, a, b in zip(NAMES, got, clean):
        bad = ~want[name][0].isfinite()
        assert torch.equal(~a.isfinite(), bad), name
        # what the bad number does not reach is what it is without it, bit for bit; with an infinity in a
        # weight or value all of a row or column is bad or changed, so the rest is compared
        if where in ("dy", "x", "down", "gate"):
            changed = (a != b) & ~bad
            allowed = torch.zeros_like(bad)
            if where == "down" and name == "dx":
                allowed[:] = True
            assert not bool((changed & ~allowed).any()), name
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
