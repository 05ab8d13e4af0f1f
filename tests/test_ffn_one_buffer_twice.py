"""One buffer for two results of a feed-forward call is refused (no GPU: nothing is launched)."""
import pytest

import dense_fp32_gemm_05_gb300 as sg


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from dense_fp32_gemm_05_gb300 import build
    build.build()
    sg.load()


BF16, E4M3 = sg.TYPE_BF16, sg.TYPE_E4M3
P = [(1 << 20) + (i << 16) for i in range(40)]      # never dereferenced


@pytest.mark.parametrize("codes,one,other,want", [(False, 13, 12, -14), (True, 13, 12, -14), (True, 16, 15, -17), (False, 20, 18, -21)])
def test_forward(codes, one, other, want):
    args = [10, 64, 128, P[3], 64, P[5], P[6], 64, P[8], 128, sg.ACT_SILU, E4M3 if codes else BF16, P[12], P[13], 128, P[15], P[16], 10,
            P[18], 128, P[20], 64]
    args[one] = args[other]
    assert sg.sgemm_ffn(*args) == want


@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("one,other,want", [(21, 20, -22), (22, 20, -23), (22, 21, -23), (29, 28, -30), (31, 28, -32), (31, 29, -32)])
def test_backward(one, other, want, accumulate):
    args = [10, 64, 128, P[3], 64, P[5], 64, P[7], P[8], 64, P[10], 128, sg.ACT_GELU, BF16, P[14], P[15], 128, P[17], P[18], 10, P[20],
            P[21], P[22], 128, P[24], 64, BF16, accumulate, P[28], P[29], 64, P[31], 128]
    args[one] = args[other]
    assert sg.sgemm_ffn_backward(*args) == want


@pytest.mark.gpu
def test_tied_weights():
    """One tensor for gate and up is an input twice, which is fine; their gradients are two buffers."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, w, down = (torch.randn(s, device="cuda", generator=gen).to(torch.bfloat16) for s in ((40, 64), (128, 64), (64, 128)))
    y, kept = sg.ffn(x, w, w, down, keep=torch.bfloat16)
    again, _ = sg.ffn(x, w, w.clone(), down, keep=torch.bfloat16)
    assert torch.equal(y, again) and torch.equal(kept[0], kept[1])
    new = [torch.zeros(s, device="cuda") for s in ((128, 64), (128, 64), (64, 128))]
    sg.ffn_backward(x, x, w, w, down, kept, dgate=new[0], dup=new[1], ddown=new[2], accumulate=True)
    with pytest.raises(sg.SgemmError):
        sg.ffn_backward(x, x, w, w, down, kept, dgate=new[0], dup=new[0], ddown=new[2], accumulate=True)
    grads = sg.ffn_backward(x, x, w, w.clone(), down, kept)
    for a, b in zip(new, grads[1:]):
        assert torch.equal(a.to(torch.bfloat16), b)
