"""sgemm_q4_quantize bit for bit against its steps in numpy, and sgemm_q4 against 64 bits: every
kernel (groups, zero codes, columns), odd sizes, strides, types, and what lies around the outputs."""
import numpy as np
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp
from tests import q4_plain as qp

pytestmark = pytest.mark.gpu

ACT = {"none": sg.ACT_NONE, "relu": sg.ACT_RELU, "silu": sg.ACT_SILU, "gelu": sg.ACT_GELU}


def _dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _quantize(w, group, symmetric, q_step=16, q_off=0, v="f32", gap=0):
    import torch
    rows, cols = w.shape
    half, groups = (cols + 1) // 2, -(-cols // group)
    Q = fp.Band(rows, half, torch.uint8, q_step, q_off)
    S, Z = fp.Band(groups, rows, torch.float32, 1, 0, gap=gap), fp.Band(groups, rows, torch.uint8, 1, 0, gap=gap)
    V = fp.Band(rows, cols, _dtype(v), 1 if gap else 8, gap)
    q, s, z = sg.q4_quantize(w, group, symmetric, Q=Q.t, S=S.t, Z=None if symmetric else Z.t, V=V.t)
    code, scale, zero, value = qp.quantize(w.float().cpu().numpy(), group, symmetric)
    assert np.array_equal(qp.unpack(q, cols).cpu().numpy(), code)
    if cols % 2:
        assert bool((q[:, -1] < 16).all())
    assert np.array_equal(s.cpu().numpy().view(np.uint32), scale.view(np.uint32))
    assert symmetric or np.array_equal(z.cpu().numpy(), zero)
    want = torch.from_numpy(value).to(_dtype(v))
    assert torch.equal(V.t.cpu(), want)
    assert Q.untouched() and S.untouched() and Z.untouched() and V.untouched()
    assert not symmetric or bool((Z.flat == 0x5A).all())


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 31), (5, 129), (4, 256), (33, 500), (130, 1027), (64, 2048)])
def test_quantize(rows, cols, dtype, group, symmetric):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(rows + cols)
    w = (torch.randn((rows, cols), generator=gen, device="cuda") + 0.3).to(_dtype(dtype))
    _quantize(w, group, symmetric)


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("dtype,v", [("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("pad,gap,step,off", [(0, 3, 1, 3), (1, 0, 4, 4), (8, 8, 16, 0)])
def test_quantize_strides(pad, gap, step, off, dtype, v, symmetric):
    import torch
    rows, cols = 37, 301
    full = torch.randn((rows, cols + 1 + pad), device="cuda", generator=torch.Generator(device="cuda").manual_seed(pad))
    _quantize(full.to(_dtype(dtype))[:, 1:cols + 1] if pad == 1 else full.to(_dtype(dtype))[:, :cols], 64, symmetric, step,
              off, v, gap)


@pytest.mark.parametrize("symmetric", [True, False])
def test_quantize_extremes(symmetric):
    import torch
    w = torch.randn((9, 400), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    w[0] = 0.0
    w[1, :200] = 3.4e38
    w[1, 200:] = -3.4e38
    w[2] = 1e-42
    w[3, 7] = float("inf")
    w[4, 9] = float("-inf")
    w[5, 11] = float("nan")
    w[6] = float("nan")
    w[7] = float("inf")
    w[8] = -w[8].abs()
    _quantize(w, 128, symmetric)
    _quantize(w, 32, symmetric)


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_ties(dtype, symmetric):
    """Halves of a step everywhere, and ranges whose both ends round away from 0 (16 steps)."""
    import torch
    w = (torch.arange(256, device="cuda") % 31 - 15).float() / 2
    w = torch.stack([w, w.flip(0), w + 0.5, w - 0.5, w * 0.25, w.abs(), -w.abs(), w.clamp(-7, 7)] * 2)
    _quantize(w.to(_dtype(dtype)), 32, symmetric)
    _quantize(w.to(_dtype(dtype))[:, 1:], 128, symmetric)


def _weights(gen, N, K, group, zeros):
    import torch
    half = (K + 1) // 2
    q = torch.full((N, -(-half // 16) * 16), 0xFF, device="cuda", dtype=torch.uint8)[:, :half]
    q.copy_(torch.randint(0, 256, (N, half), device="cuda", generator=gen, dtype=torch.uint8))
    s = torch.exp2(torch.rand((-(-K // group), N), device="cuda", generator=gen) * 4 - 2) / K ** 0.5
    z = torch.randint(0, 16, s.shape, device="cuda", generator=gen, dtype=torch.uint8) if zeros else None
    return q, s, z


def _product(M, N, K, group=128, zeros=False, two=False, x="bf16", c="f32", act="silu", pad=0, gap=0, off=0, edit=None):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(M + 3 * N + 7 * K)
    X = torch.randn((M, K + pad), device="cuda", generator=gen).to(_dtype(x))[:, :K]
    if edit:
        edit(X)
    q, s, z = _weights(gen, N, K, group, zeros)
    q2, s2, z2 = _weights(gen, N, K, group, zeros) if two else (None, None, None)
    C = fp.Band(M, N, _dtype(c), 1 if gap else 8, off, gap=gap)
    got = sg.q4_gemm(X, q, s, C.t, z, q2, s2, z2, group=group, activation=ACT[act] if two else None)
    assert got is C.t
    w = qp.values(q, s, z, group, K)
    want, e = qp.gated(X, w, qp.values(q2, s2, z2, group, K), group, act) if two else qp.product(X, w, group)
    if edit:
        bad = ~want.isfinite()
        assert torch.equal(bad, ~got.isfinite()) and bool(bad.any())
        same = got.double()[bad]
        assert bool(((same == want[bad]) | (same.isnan() & want[bad].isnan())).all())
        want, e, got = (torch.where(bad, torch.zeros_like(t), t) for t in (want, e, got.double()))
    fp.close("c", got, want, e + (2.0 ** -24 if c == "f32" else fp.BF16) * (want.abs() + e) + fp.TINY)
    assert C.untouched()
    return C.t


@pytest.mark.parametrize("two", [False, True])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 7, 13, 27, 64, 70])
def test_every_kernel(M, group, zeros, two):
    """Each group and width of columns: 1, 1, 2, 4 and 8 tiles of 8, and two blocks of them."""
    for N, K in ((200, 516), (72, 2300)):
        _product(M, N, K, group, zeros, two)


@pytest.mark.parametrize("M,N,K,two", [(1, 24000, 768, False), (4, 11776, 1536, False), (1, 14848, 1280, False),
                                       (4, 9728, 1792, False), (4, 12032, 768, True), (30, 11700, 768, False),
                                       (1, 40000, 300, False), (1, 80000, 520, False)])
def test_clusters_of_any_size(M, N, K, two):
    """Sums cut over 3, 6, 5, 7, 3 and 3 CTAs of a cluster, where 152 SMs have room, and more CTAs than that."""
    _product(M, N, K, 64, True, two, "bf16", "bf16")


SIZES = [(1, 1, 1), (1, 16, 32), (2, 17, 33), (1, 1000, 127), (3, 33, 129), (1, 40, 20000), (5, 5000, 300), (1, 2048, 4096),
         (70, 100, 700), (200, 50, 260), (64, 300, 9000), (1, 5, 300000)]


@pytest.mark.parametrize("x,c", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_products(M, N, K, x, c):
    _product(M, N, K, 128, N % 2 == 1, K % 2 == 1, x, c, "gelu")


@pytest.mark.parametrize("x", ["bf16", "f32"])
@pytest.mark.parametrize("pad,gap,off", [(1, 1, 1), (5, 3, 0), (8, 8, 8)])
def test_strides(pad, gap, off, x):
    _product(7, 130, 515, 64, True, True, x, "bf16", "silu", pad, gap, off)
    _product(2, 130, 512, 32, False, False, x, "f32", "none", pad, gap, off)


@pytest.mark.parametrize("act", fp.ACTS)
def test_activations(act):
    _product(3, 100, 384, 64, False, True, "bf16", "f32", act)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_non_finite(x):
    def edit(X):
        X[0, 3] = float("inf")
        X[1, 200] = float("nan")
        X[2, 299] = float("-inf")
    _product(5, 90, 300, 64, True, False, x, "f32", edit=edit)


@pytest.mark.parametrize("x", ["bf16", "f32"])
def test_x_of_any_size(x):
    """A code of one in each row: what x is held as.  Rows of x from small numbers to the largest,
    and values far below their block's largest."""
    import torch
    K = 128
    gen = torch.Generator(device="cuda").manual_seed(0)
    v = torch.randn((40, K), device="cuda", generator=gen)
    v *= torch.exp2(torch.linspace(-95, 124, 40, device="cuda"))[:, None]
    v[20:] *= torch.exp2(torch.randint(-26, 1, (20, K), device="cuda", generator=gen).float())
    X = v.to(_dtype(x))
    for zero in (8, 0):
        q = torch.full((K, 64), 17 * zero, device="cuda", dtype=torch.uint8)
        for i in range(K):
            q[i, i // 2] += 1 if i % 2 == 0 else 16
        Z = None if zero else torch.zeros((1, K), device="cuda", dtype=torch.uint8)
        got = sg.q4_gemm(X, q, torch.ones((1, K), device="cuda"), Z=Z, dtype=torch.float32).double()
        fp.close("x", got, X.double(), qp.held(X) + fp.SUM * X.double().abs())


def test_x_smaller_than_its_block_can_be():
    """Blocks below 2^-101 are held as if their largest value were that."""
    import torch
    X = torch.full((3, 40), 2.0 ** -100, device="cuda")
    X[1] = 2.0 ** -126
    X[2] = 0.0
    q = torch.full((5, 32), 0x99, device="cuda", dtype=torch.uint8)[:, :20]
    got = sg.q4_gemm(X, q, torch.ones((1, 5), device="cuda"))
    assert bool((got[0] == 40 * 2.0 ** -100).all()) and bool((got[2] == 0).all())
    # (scaled by 2^115 it is 2^-11, exact)
    assert bool((got[1] == 40 * 2.0 ** -126).all())


def test_same_every_time_and_on_another_stream():
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, s, z = _weights(gen, 500, 3000, 128, True)
    x = torch.randn((20, 3000), device="cuda", generator=gen)
    first = sg.q4_gemm(x, q, s, Z=z)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        again = sg.q4_gemm(x, q, s, Z=z, stream=side)
        side.synchronize()
        assert torch.equal(first, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sg.q4_gemm(x, q, s, Z=z)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)


def test_nothing_to_do():
    import torch
    e = lambda *s, d=torch.float32: torch.empty(s, device="cuda", dtype=d)  # noqa: E731
    assert sg.q4_gemm(e(0, 64), e(8, 32, d=torch.uint8), e(1, 8)).shape == (0, 8)
    assert sg.q4_gemm(e(3, 64), e(0, 32, d=torch.uint8), e(1, 0)).shape == (3, 0)
    c = torch.full((3, 8), 7.0, device="cuda")
    sg.q4_gemm(e(3, 0), e(8, 0, d=torch.uint8), e(0, 8), c)
    assert bool((c == 0).all())
    q, s, z = sg.q4_quantize(e(0, 70), 32, False)
    assert q.shape == (0, 35) and s.shape == z.shape == (3, 0)


def test_trained_quantised_and_served():
    """The operators as they are used together: a block trained for some steps (kept codes,
    gradients added over two parts of the batch), quantised, and served a token and a few."""
    import torch
    T, D, F = 256, 128, 320
    gen = torch.Generator(device="cuda").manual_seed(3)
    gate, up = (torch.randn((F, D), device="cuda", generator=gen) / D ** 0.5 for _ in range(2))
    down = torch.randn((D, F), device="cuda", generator=gen) / F ** 0.5
    for _ in range(3):
        low = [w.to(torch.bfloat16) for w in (gate, up, down)]
        grads = [torch.zeros_like(w) for w in (gate, up, down)]
        want = [torch.zeros_like(w, dtype=torch.float64) for w in (gate, up, down)]
        bound = [torch.zeros_like(w, dtype=torch.float64) for w in (gate, up, down)]
        for part in range(2):
            x = torch.randn((T, D), device="cuda", generator=gen).to(torch.bfloat16)
            y, kept = sg.ffn(x, *low, keep=torch.float8_e4m3fn)
            dy = ((y.float() - x.float()) / T).to(torch.bfloat16)
            sg.ffn_backward(dy, x, *low, kept, dgate=grads[0], dup=grads[1], ddown=grads[2], accumulate=True)
            plain = fp.backward(dy, x, *low, *fp.kept_values(kept), "silu")
            for i, n in enumerate(("dgate", "dup", "ddown")):
                want[i] += plain[n][0]
                bound[i] += plain[n][1]
        for g, w, e in zip(grads, want, bound):
            fp.close("gradient", g, w, e + 4 * 2.0 ** -24 * (w.abs() + e) + fp.TINY)
        for w, g in zip((gate, up, down), grads):
            w.sub_(g, alpha=0.1)
    q = {n: sg.q4_quantize(w, 64, symmetric=False) for n, w in (("gate", gate), ("up", up), ("down", down))}
    v = {n: qp.values(*q[n], 64, w.shape[1]) for n, w in (("gate", gate), ("up", up), ("down", down))}
    for M in (1, 5):
        x = torch.randn((M, D), device="cuda", generator=gen).to(torch.bfloat16)
        h = sg.q4_gemm(x, q["gate"][0], q["gate"][1], None, q["gate"][2], *q["up"], group=64, dtype=torch.float32)
        y = sg.q4_gemm(h, q["down"][0], q["down"][1], None, q["down"][2], group=64)
        want, e = qp.gated(x, v["gate"], v["up"], 64, "silu")
        fp.close("h", h, want, e + 2.0 ** -24 * (want.abs() + e))
        exact = want @ v["down"].t()
        fp.close("y", y, exact, qp.product(h, v["down"], 64)[1] + (e + 2.0 ** -24 * want.abs()) @ v["down"].abs().t())


def test_captured_behind_two_streams():
    """A product whose operands come from two streams of a captured graph, replayed with new ones."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    w, a, b = (torch.randn(s, device="cuda", generator=gen) for s in ((600, 1000), (600, 1000), (5, 1000)))
    q, s, _ = sg.q4_quantize(w)
    x, C = torch.zeros((5, 1000), device="cuda"), torch.zeros((5, 600), device="cuda")
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(8):
                w.copy_(a)
            sg.q4_quantize(w, Q=q, S=s)
        for _ in range(8):
            x.copy_(b)
        C.zero_()
        main.wait_stream(side)
        sg.q4_gemm(x, q, s, C)
        x.zero_()
    for _ in range(3):
        a.normal_(generator=gen)
        b.normal_(generator=gen)
        graph.replay()
        torch.cuda.synchronize()
        want, e = qp.product(b, qp.values(*sg.q4_quantize(a), 128, 1000), 128)
        fp.close("c", C, want, e + 2.0 ** -24 * (want.abs() + e) + fp.TINY)
