"""sgemm_moe against the layer's definition in 64 bits.

Error bound: activations enter as 8-bit parts whose sum differs from them by at
most 2^-20 of each value (bf16: 2^-21 of the largest of its block of 128, taken
in the bound as 2^-20 of the magnitudes, which are random); the sums are fp32,
at most (D + F) / 128 + 300 roundings of 2^-23 of the magnitudes, which the
definition's `size` adds up through both products.  One rounding to y's type."""
import numpy as np
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import fp8_plain as fp

pytestmark = pytest.mark.gpu


def _pad(n):
    return (n + 15) // 16 * 16


class Layer:
    def __init__(self, D, F, E, seed=0, pad=0):
        import torch
        rng = np.random.default_rng(seed)
        self.D, self.F, self.E = D, F, E
        self.router = (rng.standard_normal((E, D)) / np.sqrt(D)).astype(np.float32)
        self.val, self.dev = {}, {}
        for name, n, k in (("gate", F, D), ("up", F, D), ("down", D, F)):
            codes = fp.encode(np.clip(rng.standard_normal((E, n, k)) * 112, -448, 448), "e4m3")
            s = (np.exp2(rng.uniform(-1, 1, (E, -(-n // 128), -(-k // 128)))) * 4 / 448 / np.sqrt(k)).astype(np.float32)
            self.val[name] = np.stack([fp.values(codes[e], s[e], "e4m3", 128, False) for e in range(E)])
            buf = np.full((E, n + pad, _pad(k) + 16 * pad), 0x7f, np.uint8)     # gaps hold NaN
            buf[:, :n, :k] = codes
            self.dev[name] = torch.from_numpy(buf).cuda().view(torch.float8_e4m3fn)[:, :n, :k]
            self.dev["s_" + name] = torch.from_numpy(s).cuda()
        self.dev["router"] = torch.from_numpy(self.router).cuda()

    def run(self, x, topk, renormalize, logits=None, **kw):
        d = self.dev
        return sg.moe(x, d["router"] if logits is None else None, d["gate"], d["s_gate"], d["up"], d["s_up"],
                      d["down"], d["s_down"], topk, renormalize, logits=logits, **kw)

    def check(self, x, topk, renormalize, logits=None, **kw):
        import torch
        y, lg, idx, w = self.run(x, topk, renormalize, logits, **kw)
        torch.cuda.synchronize()
        assert sg.sgemm_device_error() == 0
        x64 = x.double().cpu().numpy()
        # routing is compared on the logits that the kernel found (a tie within
        # rounding may fall either way), the logits on their own
        l64 = lg.double().cpu().numpy()
        if logits is None:
            ref = x64 @ self.router.astype(np.float64).T
            size = np.abs(x64) @ np.abs(self.router.astype(np.float64)).T
            assert np.all(np.abs(l64 - ref) <= (self.D / 128 + 40) * 2.0 ** -23 * size)
        want, _, order, w64, size = fp.moe(x64, None, self.val["gate"], self.val["up"], self.val["down"], topk,
                                           renormalize, logits=l64)
        assert np.array_equal(idx.cpu().numpy(), order)
        assert np.all(np.abs(w.cpu().numpy() - w64) <= 64 * 2.0 ** -23 * w64 + 1e-37)
        out = -8 if x.dtype == torch.bfloat16 else -24
        tol = ((self.D + self.F) / 128 + 300) * 2.0 ** -23 * size + 2.0 ** -20 * size + 2.0 ** out * np.abs(want) + 1e-37
        err = np.abs(y.double().cpu().numpy() - want) / tol
        assert err.max() <= 1.0, err.max()
        return y


def _x(T, D, dtype, seed=1):
    import torch
    return torch.randn((T, D), generator=torch.Generator().manual_seed(seed)).to(getattr(torch, dtype)).cuda()


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,D,F,E,topk", [
    (1, 256, 128, 4, 1), (1, 128, 64, 2, 2), (1, 1024, 512, 8, 2), (2, 512, 256, 16, 4), (5, 300, 200, 7, 3),
    (8, 257, 129, 3, 3), (9, 384, 320, 8, 2), (16, 256, 192, 33, 8), (17, 640, 100, 5, 2), (32, 256, 256, 4, 4),
    (33, 320, 160, 6, 3), (64, 256, 128, 2, 1), (64, 512, 384, 40, 8), (100, 200, 130, 3, 2), (128, 256, 128, 64, 16),
    (128, 128, 64, 2, 2), (3, 1, 1, 1, 1), (4, 17, 16, 9, 9), (6, 128, 64, 128, 8), (5, 128, 64, 130, 7),
    (2, 64, 32, 512, 16)])
def test_layer(dtype, T, D, F, E, topk):
    Layer(D, F, E, seed=T).check(_x(T, D, dtype), topk, renormalize=T % 2 == 0)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_larger_layer(dtype):
    layer = Layer(2048, 1408, 16, seed=3)
    for T in (1, 4, 23):
        layer.check(_x(T, 2048, dtype, T), 6, True)


def test_strides_offsets_and_padding():
    import torch
    layer = Layer(200, 136, 5, seed=2, pad=3)
    for dtype in ("bfloat16", "float32"):
        big = torch.full((40, 231), float("nan"), device="cuda", dtype=getattr(torch, dtype))
        x = big[3:10, 7:207]
        x.copy_(_x(7, 200, dtype))
        ybig = torch.full((9, 219), -5.0, device="cuda", dtype=x.dtype)
        y = ybig[1:8, 3:203]
        layer.check(x, 2, True, y=y)
        mask = torch.ones_like(ybig, dtype=torch.bool)
        mask[1:8, 3:203] = False
        assert bool((ybig[mask] == -5.0).all())


def test_every_token_to_one_expert_and_ties():
    import torch
    layer = Layer(256, 192, 6, seed=5)
    for T in (7, 16, 40, 90):
        logits = torch.zeros((T, 6), device="cuda")          # all tied: the lowest indices win
        layer.check(_x(T, 256, "float32"), 2, True, logits=logits)
        logits[:, 4] = 3.0
        layer.check(_x(T, 256, "bfloat16"), 1, False, logits=logits)


def test_masked_experts():
    """-inf logits (experts switched off): never chosen while others are left, weight 0 when they must be."""
    import torch
    layer = Layer(256, 128, 8, seed=6)
    logits = torch.randn((12, 8), generator=torch.Generator().manual_seed(0)).cuda()
    logits[:, ::2] = float("-inf")
    y, _, idx, w = layer.run(_x(12, 256, "float32"), 4, True, logits=logits)
    assert bool((idx % 2 == 1).all())
    layer.check(_x(12, 256, "float32"), 4, True, logits=logits)
    logits[:, 3:] = torch.finfo(torch.float32).min
    _, _, idx, w = layer.run(_x(12, 256, "float32"), 5, False, logits=logits)
    assert idx[0].tolist() == [1, 3, 4, 5, 6] and w[0].tolist() == [1.0, 0.0, 0.0, 0.0, 0.0]


def test_values_of_every_size():
    """Tokens scaled by powers of two from 2^-60 to 2^40, and blocks of one token that differ as much."""
    import torch
    layer = Layer(384, 128, 4, seed=7)
    x = _x(24, 384, "float32")
    x *= torch.exp2(torch.linspace(-60, 8, 24, device="cuda").round())[:, None]
    x[5, :128] *= 2.0 ** -30
    x[6, 128:256] = 0.0
    x[7] = 0.0
    x[8, 100] *= 2.0 ** 12
    logits = torch.randn((24, 4), generator=torch.Generator().manual_seed(3)).cuda()
    layer.check(x, 2, True, logits=logits)


def test_not_a_number():
    """A NaN or infinite token makes its own output NaN and no other's."""
    import torch
    layer = Layer(256, 128, 4, seed=8)
    x = _x(6, 256, "float32")
    logits = torch.randn((6, 4), generator=torch.Generator().manual_seed(3)).cuda()
    good = layer.run(x, 2, True, logits=logits)[0].clone()
    x[1, 7], x[4, 200] = float("nan"), float("inf")
    y = layer.run(x, 2, True, logits=logits)[0]
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[4]).all())
    keep = [0, 2, 3, 5]
    assert torch.equal(y[keep], good[keep])


def test_same_result_every_time_on_any_stream_and_in_a_graph():
    import torch
    layer = Layer(1024, 512, 16, seed=9)
    x = _x(11, 1024, "bfloat16")
    outs = [layer.run(x, 4, True)[0] for _ in range(4)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        outs += [layer.run(x, 4, True)[0] for _ in range(3)]
        y = torch.empty_like(x)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            layer.run(x, 4, True, y=y)
        for _ in range(3):
            g.replay()
    torch.cuda.synchronize()
    assert sg.sgemm_device_error() == 0
    assert all(torch.equal(outs[0], o) for o in outs[1:]) and torch.equal(outs[0], y)


def test_between_other_calls():
    """The kernel's barriers are its own: the GEMM's paths on the same stream, whose
    workspaces hold anything, change nothing."""
    import torch
    layer = Layer(1024, 512, 16, seed=12)
    x = _x(3, 1024, "bfloat16")
    good = layer.run(x, 4, True)[0].clone()
    small, big = torch.randn(16, 4096, device="cuda"), torch.randn(4096, 2048, device="cuda")
    square = torch.randn(700, 700, device="cuda")
    for _ in range(3):
        sg.gemm(small, big, torch.empty(16, 2048, device="cuda"))
        sg.gemm(small[:2], big, torch.empty(2, 2048, device="cuda"))
        sg.gemm(square, square, torch.empty(700, 700, device="cuda"))
        assert torch.equal(layer.run(x, 4, True)[0], good)
    layer.check(x, 4, True)
    sg.sgemm_release_workspace()
    assert torch.equal(layer.run(x, 4, True)[0], good)


def test_two_streams_at_once():
    import torch
    layer = Layer(768, 256, 8, seed=10)
    x = [_x(4, 768, "float32", i) for i in range(2)]
    want = [layer.run(v, 2, True)[0].clone() for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = layer.run(x[i], 2, True)[0]
    torch.cuda.synchronize()
    assert sg.sgemm_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_weights_from_the_quantiser():
    """The whole way: fp32 experts quantised block by block, their products by
    sgemm_fp8 close to the layer's (which keeps its activations in full)."""
    import torch
    D, F, E, T = 384, 256, 4, 9
    g = torch.Generator(device="cuda").manual_seed(4)
    w = {n: torch.randn(s, generator=g, device="cuda") / s[-1] ** 0.5
         for n, s in (("gate", (E, F, D)), ("up", (E, F, D)), ("down", (E, D, F)))}
    q = {}
    for n, t in w.items():
        parts = [sg.fp8_quantize(t[e], (128, 128)) for e in range(E)]
        q[n], q["s_" + n] = torch.stack([a for a, _ in parts]), torch.stack([b for _, b in parts])
    x = torch.randn((T, D), generator=g, device="cuda")
    logits = torch.zeros((T, E), device="cuda")
    logits[:, 2] = 1.0
    y = sg.moe(x, None, q["gate"], q["s_gate"], q["up"], q["s_up"], q["down"], q["s_down"], 1, True, logits=logits)[0]
    qx, sx = sg.fp8_quantize(x)
    a, b = (sg.fp8_gemm(qx, sx, q[n][2], q["s_" + n][2], torch.empty(T, F, device="cuda")) for n in ("gate", "up"))
    qh, sh = sg.fp8_quantize(torch.nn.functional.silu(a) * b)
    z = sg.fp8_gemm(qh, sh, q["down"][2], q["s_down"][2], torch.empty(T, D, device="cuda"))
    assert (y - z).norm() < 0.1 * y.norm()


def test_a_wait_that_runs_out_is_reported():
    import torch
    layer = Layer(1024, 512, 16, seed=11)
    x = _x(5, 1024, "float32")
    good = layer.run(x, 4, True)[0].clone()
    torch.cuda.synchronize()
    try:
        assert sg.sgemm_set_wait_limit(1) == 0
        layer.run(x, 4, True)
        assert sg.sgemm_device_error(torch.cuda.current_stream()) == sg.SGEMM_ERR_TIMEOUT
    finally:
        sg.sgemm_set_wait_limit(0)
    for _ in range(2):
        again = layer.run(x, 4, True)[0]
        assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
        assert torch.equal(again, good)


def test_refusals_of_the_tensor_call():
    import torch
    layer = Layer(128, 64, 4)
    x = _x(2, 128, "float32")
    with pytest.raises(sg.SgemmError):
        layer.run(x, 5, True)
    with pytest.raises(ValueError):
        layer.run(x[:, :100], 2, True)
    with pytest.raises(ValueError):
        layer.run(x.half(), 2, True)
    with pytest.raises(ValueError):
        layer.run(x, 2, True, y=torch.empty(2, 128, device="cuda", dtype=torch.bfloat16))
    odd = torch.zeros((4, 64, 129), device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)[:, :, :128]
    d = layer.dev
    with pytest.raises(sg.SgemmError) as e:
        sg.moe(x, d["router"], odd, d["s_gate"], odd, d["s_up"], d["down"], d["s_down"], 2)
    assert e.value.status == sg.SGEMM_ERR_UNSUPPORTED
    assert sg.moe(x[:0], d["router"], d["gate"], d["s_gate"], d["up"], d["s_up"], d["down"], d["s_down"], 2)[0].shape == (0, 128)
