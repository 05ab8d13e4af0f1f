"""The feed-forward and 4-bit operators on matrices of more than 2^31 elements: offsets past 32
bits.  Rows at the start, in the middle and at the end are compared; a wrong offset gives
another row's values, or the fill's."""
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp
from tests import q4_plain as qp

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    import torch
    yield
    torch.cuda.empty_cache()


def _windows(n, size=200):
    import torch
    return torch.cat([torch.arange(max(i, 0), min(i + size, n), device="cuda") for i in (0, n // 2 - size // 2, n - size)]).unique()


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_block(keep):
    """T x F of 2.2e9 elements: kept values, h, dg and du."""
    import torch
    T, D, F = 270001, 64, 8200
    assert T * F > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, dy = fp.matrix(gen, T, D), fp.matrix(gen, T, D, 0.1)
    gate, up, down = fp.matrix(gen, F, D, 0.15), fp.matrix(gen, F, D, 0.15), fp.matrix(gen, D, F, 0.01)
    y, kept = sg.ffn(x, gate, up, down, keep=torch.bfloat16 if keep == "bf16" else torch.float8_e4m3fn)
    grads = [torch.full(s, float("nan"), device="cuda") for s in ((F, D), (F, D), (D, F))]
    dx = sg.ffn_backward(dy, x, gate, up, down, kept, dgate=grads[0], dup=grads[1], ddown=grads[2])[0]
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    at = _windows(T)
    want = fp.forward(x[at], gate, up, down, "silu")
    fp.close("y", y[at], *want["y"])
    rows = [t[at] if i < 2 else t[:, at] for i, t in enumerate(kept)]
    g, u = fp.kept_values(rows)
    for v, n in ((g, "g"), (u, "u")):
        half = fp.BF16 if keep == "bf16" else 2.0 ** -4 * (1 + 2.0 ** -20)
        least = 0.0 if keep == "bf16" else 2.0 ** -10 * rows[2 + "gu".index(n)].double().t().repeat_interleave(128, 1)[:, :F]
        fp.close(n, v, want[n][0], want[n][1] + half * (want[n][0].abs() + want[n][1]) + least)
    v, e = fp.backward(dy[at], x[at], gate, up, down, g, u, "silu")["dx"]
    fp.close("dx", dx[at], v, e + fp.BF16 * (v.abs() + e))
    # the weights' gradients: every token's share (with bounds, in parts)
    total = [[torch.zeros_like(t, dtype=torch.float64) for t in grads] for _ in range(2)]
    for i in range(0, T, 30000):
        part = slice(i, min(i + 30000, T))
        g, u = fp.kept_values([t[part] if k < 2 else t[:, part] for k, t in enumerate(kept)])
        plain = fp.backward(dy[part], x[part], gate, up, down, g, u, "silu")
        for k, n in enumerate(("dgate", "dup", "ddown")):
            v, e = plain[n]
            # (a sum of T terms, not of the part's)
            total[0][k] += v
            total[1][k] += e * (T + 16) / (part.stop - part.start + 16)
        del g, u, plain
    for k, n in enumerate(("dgate", "dup", "ddown")):
        fp.close(n, grads[k], total[0][k], total[1][k] + 2.0 ** -24 * total[0][k].abs())


def test_block_of_one_token():
    """Matrices of 2.4e9 elements, each read once."""
    import torch
    D, F = 60000, 40000
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = fp.matrix(gen, 1, D)
    w = []
    for shape in ((F, D), (F, D), (D, F)):
        t = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
        t.random_(-3, 4, generator=gen)
        t *= 2.0 ** -8
        w.append(t)
    h = torch.empty((1, F), device="cuda", dtype=torch.bfloat16)
    y = sg.ffn(x, *w, h=h)[0]
    at = _windows(F)
    g, u = (x.double() @ w[i][at].double().t() for i in range(2))
    size = x.double().abs() @ w[0][at].double().abs().t()
    e = 4 * (D + 16) * fp.SUM * size * (1 + u.abs() + g.abs())
    want = fp.act("silu", g) * u
    fp.close("h", h[:, at], want, e + fp.BF16 * want.abs())
    at = _windows(D)
    want = h.double() @ w[2][at].double().t()
    e = (F + 16) * fp.SUM * (h.double().abs() @ w[2][at].double().abs().t())
    fp.close("y", y[:, at], want, e + fp.BF16 * want.abs())


def test_quantize():
    import torch
    rows, cols = 70001, 32004
    w = torch.empty((rows, cols), device="cuda", dtype=torch.bfloat16)
    w.random_(-100, 101, generator=torch.Generator(device="cuda").manual_seed(2))
    v = torch.empty((rows, cols), device="cuda", dtype=torch.bfloat16)
    q, s, z = sg.q4_quantize(w, 64, False, V=v)
    at = _windows(rows, 20)
    code, scale, zero, value = qp.quantize(w[at].float().cpu().numpy(), 64, False)
    assert (qp.unpack(q[at], cols).cpu().numpy() == code).all() and (s[:, at].cpu().numpy() == scale).all()
    assert (z[:, at].cpu().numpy() == zero).all() and torch.equal(v[at].cpu(), torch.from_numpy(value).to(torch.bfloat16))


@pytest.mark.parametrize("M,N,K", [(2, 70000, 65536), (64, 36000000, 32)])
def test_product(M, N, K):
    """Codes of 2.3e9 bytes, and a C of 2.3e9 elements."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.empty((N, K // 2), device="cuda", dtype=torch.uint8).random_(0, 256, generator=gen)
    s = torch.rand((-(-K // 128), N), device="cuda", generator=gen) + 0.5
    x = torch.randn((M, K), device="cuda", generator=gen).to(torch.bfloat16)
    C = torch.full((M, N), float("nan"), device="cuda")
    sg.q4_gemm(x, q, s, C)
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0 and not bool(C.isnan().any())
    at = _windows(N)
    want, e = qp.product(x, qp.values(q[at], s[:, at], None, 128, K), 128)
    fp.close("c", C[:, at], want, e + 2.0 ** -24 * want.abs())


def test_product_past_what_is_addressed_is_refused():
    """(Scales are addressed in 32 bits; nothing is launched, so the pointers are never read.)"""
    import torch
    P = torch.empty(64, device="cuda").data_ptr()
    assert sg.sgemm_q4(1, 2 ** 28, 4096, P, sg.TYPE_BF16, 4096, P, P, 0, 0, 0, 0, 2048, 2 ** 28, 32, 0, P, sg.TYPE_BF16,
                       2 ** 28) == sg.SGEMM_ERR_UNSUPPORTED
