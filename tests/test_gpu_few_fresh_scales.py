"""Weights, scales and zero codes that the kernel just before rewrites in place, again and again, with
nothing waited for: each product is of the newest."""
import pytest

import dense_fp32_gemm_05_gb300 as sg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 500, 4096), (3, 4001, 1000), (20, 1000, 3000), (64, 700, 2000)])
def test_rewritten_in_place(M, N, K, two):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(M)
    w = [torch.randn((N, K), device="cuda", generator=gen) for _ in range(6)]
    codes = [sg.q4_quantize(t, 32, False) for t in w]
    q, s, z = [torch.empty_strided(t.shape, t.stride(), device="cuda", dtype=t.dtype) for t in codes[0]]
    x = torch.randn((M, K), device="cuda", generator=gen).to(torch.bfloat16)

    def product(a, b, c):
        return sg.q4_gemm(x, a, b, Z=c, group=32, **(dict(Q2=a, S2=b, Z2=c) if two else {}))

    want = [product(*c) for c in codes]
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        for to, t in zip((q, s, z), codes[i % 6]):
            to.copy_(t)
        if i % 3 == 0:
            s.add_(0.0)                        # (read and written by the kernel just before)
        got.append(product(q, s, z))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 6]) for i, g in enumerate(got))
    # quantised in place just before, scales last
    got = []
    for i in range(30):
        sg.q4_quantize(w[i % 6], 32, False, Q=q, S=s, Z=z)
        got.append(product(q, s, z))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 6]) for i, g in enumerate(got))
