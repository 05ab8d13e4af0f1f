"""Matrices of more than 2^31 elements: offsets of rows and experts past 32 bits.  Rows at
the start, in the middle and at the end are compared; a wrong offset gives another row's
values, or the fill's."""
import pytest
import torch

import dense_fp32_gemm_05_gb300 as sg

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _windows(n):
    """Indices at the start, about the middle, and at the end."""
    return torch.cat([torch.arange(max(i, 0), min(i + 300, n), device="cuda") for i in (0, n // 2 - 150, n - 300)]).unique()


@pytest.mark.parametrize("group", [(1, 128), (128, 1), (128, 128)])
def test_quantize(group):
    rows, cols = 70001, 32004                                     # 2.24e9 elements
    x = torch.empty((rows, cols), device="cuda", dtype=torch.bfloat16)
    x.random_(-4, 5, generator=torch.Generator(device="cuda").manual_seed(1))
    x[:, ::128] = 448.0                                           # codes are the values, scales 1
    x[::128] = 448.0
    q, s = sg.fp8_quantize(x, group)
    assert bool((s == 1).all())
    for i in range(0, rows, 10000):
        assert torch.equal(q[i: i + 10000].float(), x[i: i + 10000].float())


@pytest.mark.parametrize("M,N,b_group", [(65600, 33000, 128), (65600, 33003, 1), (3000000, 800, 128), (60, 36000000, 128)])
def test_product(M, N, b_group):
    """C of more than 2^31 elements, on wide tiles and (60 rows) narrow ones."""
    K = 128
    gen = torch.Generator(device="cuda").manual_seed(2)
    a, b = (torch.randint(-2, 3, (n, K), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16).to(E4M3)
            for n in (M, N))
    sa = torch.exp2(torch.randint(-2, 3, (1, M), generator=gen, device="cuda").float())
    sb = torch.exp2(torch.randint(-2, 3, (1, N) if b_group == 1 else (-(-N // 128), 1), generator=gen, device="cuda").float())
    C = torch.full((M, N), float("nan"), device="cuda", dtype=torch.bfloat16)
    assert C.numel() > 2 ** 31
    sg.fp8_gemm(a, sa, b, sb, C, b_group=b_group)
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    i, j = _windows(M), _windows(N)
    A = a[i].double() * sa[0, i, None].double()
    B = b[j].double() * (sb[0, j] if b_group == 1 else sb[j // 128, 0])[:, None].double()
    want = (A @ B.t()).to(torch.float32).to(torch.bfloat16)       # (exact in fp32: integers over 16)
    assert torch.equal(C[i[:, None], j[None, :]], want)
    for k in range(0, M, -(-M // 16)):                            # every element was written
        assert not bool(C[k: k + -(-M // 16)].isnan().any())


def test_layer():
    """512 experts, 2^32 bytes and more of codes for each matrix."""
    T, D, F, E, topk = 6, 4096, 2064, 512, 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = {}
    for name, rows, cols in (("gate", F, D), ("up", F, D), ("down", D, F)):
        c = torch.full((E, rows, cols), 0x7f, device="cuda", dtype=torch.uint8)       # NaN
        assert c.numel() > 2 ** 32
        for e in (0, 255, 256, 509, 511):
            v = torch.randn((rows, cols), generator=gen, device="cuda") * 100
            c[e] = v.clamp(-448, 448).to(E4M3).view(torch.uint8)
        w[name] = c.view(E4M3)
        w["s_" + name] = torch.full((E, -(-rows // 128), -(-cols // 128)), 0.04 / cols ** 0.5, device="cuda")
    x = torch.randn((T, D), generator=gen, device="cuda")
    logits = torch.zeros((T, E), device="cuda")
    for t in range(T):
        for k, e in enumerate(((0, 256, 511), (511, 255, 509))[t % 2]):
            logits[t, e] = 5.0 - k
    y, _, idx, weights = sg.moe(x, None, w["gate"], w["s_gate"], w["up"], w["s_up"], w["down"], w["s_down"], topk,
                                logits=logits)
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    assert idx[0].tolist() == [0, 256, 511] and idx[1].tolist() == [511, 255, 509]
    for t in range(T):
        want = 0
        for p, e in zip(weights[t].double(), idx[t].tolist()):
            g, u, d = (w[n][e].double() * w["s_" + n][e, 0, 0].double() for n in ("gate", "up", "down"))
            g, u = g @ x[t].double(), u @ x[t].double()
            want = want + p * (d @ (g * torch.sigmoid(g) * u))
        assert (y[t].double() - want).norm() <= 2.0 ** -18 * want.norm()
