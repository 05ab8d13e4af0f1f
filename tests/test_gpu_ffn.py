"""sgemm_ffn and sgemm_ffn_backward against the definition in 64 bits: every tile, kept type
and activation, odd sizes, strides, single tokens, empty ones, and what lies around the outputs."""
import pytest

import dense_fp32_gemm_05_gb300 as sg
from tests import ffn_plain as fp

pytestmark = pytest.mark.gpu

ACT = {"none": sg.ACT_NONE, "relu": sg.ACT_RELU, "silu": sg.ACT_SILU, "gelu": sg.ACT_GELU}


def _inputs(T, D, F, seed=0, pad=8):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed + 3 * T + 5 * D + 7 * F)
    x = fp.matrix(gen, T, D, 1.0, pad)
    gate, up = (fp.matrix(gen, F, D, 1.5 / max(D, 1) ** 0.5, pad) for _ in range(2))
    down = fp.matrix(gen, D, F, 1.0 / max(F, 1) ** 0.5, pad)
    dy = fp.matrix(gen, T, D, 0.1, pad)
    return dy, x, gate, up, down


def _kept_bands(T, F, keep, gap=0, offset=0):
    import torch
    if keep is None:
        return []
    if keep == "bf16":
        return [fp.Band(T, F, torch.bfloat16, 8, offset, gap=gap) for _ in range(2)]
    return ([fp.Band(T, F, torch.float8_e4m3fn, 16, offset, gap=gap) for _ in range(2)] +
            [fp.Band(-(-F // 128), T, torch.bfloat16, 1, 0, gap=gap) for _ in range(2)])


def _check_kept(kept, want, keep):
    import torch
    for i, name in enumerate(("g", "u")):
        v, e = want[name]
        if keep == "bf16":
            fp.close(name, kept[i], v, e + fp.BF16 * (v.abs() + e) + fp.TINY)
            continue
        F = v.shape[1]
        groups = torch.nn.functional.pad(v.abs() + e, (0, -F % 128)).view(v.shape[0], -1, 128).amax(2).t()
        low = torch.nn.functional.pad(v.abs() - e, (0, -F % 128)).view(v.shape[0], -1, 128).amax(2).t()
        s = kept[2 + i].double()
        assert bool((s <= groups / 448 * (1 + fp.BF16 + 2 * fp.SUM)).all())
        assert bool((s >= low / 448 * (1 - fp.BF16 - 2 * fp.SUM)).all())
        wide = s.t().repeat_interleave(128, 1)[:, :F]
        # (half a step: 2^-4 of the value, or half of the smallest code, 2^-10)
        fp.close(name, kept[i].double() * wide, v, e + 2.0 ** -4 * (1 + 2.0 ** -20) * (v.abs() + e) + 2.0 ** -10 * wide)


def _forward(T, D, F, act="silu", keep=None, pad=8, gap=0, offset=0, seed=0):
    import torch
    _, x, gate, up, down = _inputs(T, D, F, seed, pad)
    bands = _kept_bands(T, F, keep, gap, offset)
    y, h = fp.Band(T, D, torch.bfloat16, 1 if gap else 8, offset, gap=gap), fp.Band(T, F, torch.bfloat16, 8)
    kept = tuple(b.t for b in bands) or None
    got, back = sg.ffn(x, gate, up, down, ACT[act], kept=kept, y=y.t, h=h.t)
    assert got is y.t and back is kept
    want = fp.forward(x, gate, up, down, act)
    fp.close("y", got, *want["y"])
    if keep:
        _check_kept(kept, want, keep)
    assert y.untouched() and h.untouched() and all(b.untouched() for b in bands)
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0
    return y.t, kept


SIZES = [(1, 64, 64), (1, 1, 1), (2, 7, 3), (5, 40, 129), (33, 100, 31), (64, 129, 255), (127, 65, 300), (130, 250, 1000),
         (257, 512, 640), (300, 8, 2000), (515, 700, 513), (1000, 264, 1288)]


@pytest.mark.parametrize("keep", [None, "bf16", "e4m3"])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_forward(T, D, F, keep):
    _forward(T, D, F, "silu", keep)


@pytest.mark.parametrize("act", fp.ACTS)
@pytest.mark.parametrize("keep", [None, "bf16", "e4m3"])
def test_forward_activations(act, keep):
    _forward(140, 200, 300, act, keep)


@pytest.mark.parametrize("keep,gap,offset", [(None, 1, 1), ("bf16", 3, 1), ("bf16", 8, 8), ("bf16", 2, 2), ("e4m3", 5, 3), ("e4m3", 16, 0),
                                            ("e4m3", 4, 4)])
def test_forward_strides(keep, gap, offset):
    """Outputs with odd strides and starts; inputs with wide rows."""
    for T, D, F in ((70, 90, 140), (300, 260, 520)):
        _forward(T, D, F, "gelu", keep, 64, gap, offset)


def _backward(T, D, F, act="silu", keep="bf16", grad="bf16", add=False, pad=8, gap=0, offset=0, edit=None):
    import torch
    dy, x, gate, up, down = _inputs(T, D, F, 1, pad)
    if edit:
        edit(dy, x, gate, up, down)
    kept = sg.ffn(x, gate, up, down, ACT[act], keep=torch.bfloat16 if keep == "bf16" else torch.float8_e4m3fn)[1]
    g, u = fp.kept_values(kept)
    want = fp.backward(dy, x, gate, up, down, g, u, act)
    kind = torch.bfloat16 if grad == "bf16" else torch.float32
    step = 1 if gap else 8
    bands = {"dx": fp.Band(T, D, torch.bfloat16, step, offset, gap=gap), "dgate": fp.Band(F, D, kind, step, offset, gap=gap),
             "dup": fp.Band(F, D, kind, step, offset, gap=gap), "ddown": fp.Band(D, F, kind, step, offset, gap=gap)}
    scratch = [fp.Band(T, F, torch.bfloat16, 8) for _ in range(3)]
    gen = torch.Generator(device="cuda").manual_seed(9)
    before = {}
    for n, b in bands.items():
        b.t.copy_(torch.randn(b.t.shape, generator=gen, device="cuda"))
        before[n] = b.t.double().clone()
    out = sg.ffn_backward(dy, x, gate, up, down, kept, ACT[act], accumulate=add, scratch=tuple(b.t for b in scratch),
                          **{n: b.t for n, b in bands.items()})
    for n, got in zip(bands, out):
        assert got is bands[n].t
        v, e = want[n]
        if add and n != "dx":
            v, e = v + before[n], e + 2.0 ** -24 * (v + before[n]).abs()
        half = 2.0 ** -24 if grad == "f32" and n != "dx" else fp.BF16
        fp.close(n, got, v, e + half * (v.abs() + e) + fp.TINY)
    assert all(b.untouched() for b in list(bands.values()) + scratch)
    assert sg.sgemm_device_error(torch.cuda.current_stream()) == 0


@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_backward(T, D, F, keep):
    _backward(T, D, F, "silu", keep)


@pytest.mark.parametrize("act", fp.ACTS)
@pytest.mark.parametrize("keep", ["bf16", "e4m3"])
def test_backward_activations(act, keep):
    _backward(140, 200, 300, act, keep)


@pytest.mark.parametrize("grad,add", [("f32", False), ("f32", True), ("bf16", True)])
@pytest.mark.parametrize("gap,offset", [(0, 0), (3, 1), (2, 2)])
def test_backward_types_strides_and_sums(grad, add, gap, offset):
    for T, D, F in ((70, 90, 140), (300, 260, 520)):
        _backward(T, D, F, "gelu", "e4m3", grad, add, 64, gap, offset)


def test_every_cut():
    """Each launch of a block in each way that the plan cuts it, by sizes that it cuts so."""
    seen = {n: set() for n in ("gated", "down", "slope", "dx", "weights")}
    sizes = [(T, D, F) for T in (17, 100, 300, 777, 2000, 4000) for D, F in ((64, 96), (200, 1500), (500, 4000), (1000, 2501),
                                                                          (2000, 300), (900, 9000), (3000, 200))]
    sizes.append((2500, 2000, 4000))
    for T, D, F in sizes:
        new = False
        for n, cut in sg.sgemm_ffn_plan(T, D, F)[1].items():
            new = new or cut not in seen[n]
            seen[n].add(cut)
        if new:
            for keep in ("bf16", "e4m3"):
                _forward(T, D, F, "silu", keep)
                _backward(T, D, F, "silu", keep)
            _forward(T, D, F, "silu", None, gap=1)
    assert {c[:2] for c in seen["gated"]} == {c[:2] for c in seen["slope"]} == {(256, 256), (128, 128), (128, 64)}
    assert {c[2] for c in seen["down"]} == {1, 2, 4, 8} and len({c[2] for c in seen["dx"]}) > 2, seen


def test_new_buffers_and_another_stream():
    import torch
    dy, x, gate, up, down = _inputs(200, 96, 160)
    want, kept = sg.ffn(x, gate, up, down, keep=torch.float8_e4m3fn)
    grads = sg.ffn_backward(dy, x, gate, up, down, kept)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, kept2 = sg.ffn(x, gate, up, down, keep=torch.float8_e4m3fn, stream=side)
    grads2 = sg.ffn_backward(dy, x, gate, up, down, kept2, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(kept, kept2))
    assert all(torch.equal(a, b) for a, b in zip(grads, grads2))


@pytest.mark.parametrize("T", [1, 40, 700])
def test_among_other_work(T):
    """Calls in a row with nothing waited for, their inputs and weights written just before them by
    other kernels, and their outputs read just after: the same as one at a time."""
    import torch
    D, F = 544, 1568
    _, x, gate, up, down = _inputs(T, D, F)
    q4 = [sg.q4_quantize(w.float(), 64, False) for w in (gate, down)]

    def steps(wait):
        w = [t.clone() for t in (gate, up, down)]
        codes = [[t.clone() for t in q] for q in q4]
        h = x.clone()
        out = []
        for i in range(12):
            def then(v):
                if wait:
                    torch.cuda.synchronize()
                return v
            y, kept = then(sg.ffn(h, *w, keep=torch.bfloat16 if i % 3 else None))
            if kept is not None:
                grads = then(sg.ffn_backward((y * (0.5 / T)).contiguous(), h, *w, kept))
                for a, g in zip(w, grads[1:]):
                    a.add_(g, alpha=-0.01)
            z = then(sg.q4_gemm(h, codes[0][0], codes[0][1], Z=codes[0][2], group=64))
            z = then(sg.q4_gemm(z, codes[1][0], codes[1][1], Z=codes[1][2], group=64))
            codes[0][1].mul_(1.01)
            codes[1][0].bitwise_xor_(i)
            h = torch.tanh(y.float() + z.float()).to(torch.bfloat16)
            out.append(h)
        torch.cuda.synchronize()
        return out

    want = steps(True)
    assert all(bool(t.isfinite().all()) for t in want)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(steps(False), want))


def test_two_at_a_time():
    """Calls on two streams at once, forward, backward and with 4 bits, as alone."""
    import torch
    sets = []
    for seed, (T, D, F) in enumerate(((900, 256, 1000), (5, 512, 2048))):
        dy, x, gate, up, down = _inputs(T, D, F, seed)
        q = sg.q4_quantize(gate.float())
        y, kept = sg.ffn(x, gate, up, down, keep=torch.bfloat16)
        alone = [sg.ffn(x, gate, up, down)[0], *sg.ffn_backward(dy, x, gate, up, down, kept), sg.q4_gemm(x[:20], *q[:2])]
        sets.append((dy, x, gate, up, down, q, kept, alone, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (dy, x, gate, up, down, q, kept, _, stream) in enumerate(sets):
            with torch.cuda.stream(stream):
                got[i].append([sg.ffn(x, gate, up, down)[0], *sg.ffn_backward(dy, x, gate, up, down, kept),
                               sg.q4_gemm(x[:20], *q[:2])])
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, sets[i][7]))


def test_one_token_captured_and_replayed():
    """Two graphs of a block's decode step, one after the other and with new inputs."""
    import torch
    _, x, gate, up, down = _inputs(1, 520, 2056)
    want = sg.ffn(x, gate, up, down)[0].clone()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            y = x
            for _ in range(3):
                y = sg.ffn(x, gate, up, down)[0]
            outs.append(y)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in outs)
    x.copy_(_inputs(1, 520, 2056, seed=9)[1])
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    want = sg.ffn(x, gate, up, down)[0]
    assert all(torch.equal(y, want) for y in outs)


def test_few_tokens_in_clusters_of_three():
    """A width for which 152 SMs have room for three CTAs a cluster, and one of more CTAs than that."""
    _forward(5, 192, 12032)
    _forward(3, 16, 50000)


def test_captured_behind_two_streams():
    """A block whose operands come from two streams of a captured graph, replayed with new ones."""
    import torch
    for T in (3, 200):
        dy, x, gate, up, down = _inputs(T, 256, 512)
        sources = [t.clone() for t in (x, gate, down)]
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        y = sg.ffn(x, gate, up, down)[0]
        with torch.cuda.graph(graph):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                for _ in range(8):
                    gate.copy_(sources[1])
                    down.copy_(sources[2])
            for _ in range(8):
                x.copy_(sources[0])
            y.zero_()
            main.wait_stream(side)
            sg.ffn(x, gate, up, down, y=y)
            for t in (x, gate, down):
                t.zero_()
        for seed in (5, 6):
            _, *new = _inputs(T, 256, 512, seed)
            for to, t in zip(sources, (new[0], new[1], new[3])):
                to.copy_(t)
            graph.replay()
            torch.cuda.synchronize()
            fp.close("y", y, *fp.forward(new[0], new[1], up, new[3], "silu")["y"])


def test_captured_and_replayed():
    import torch
    dy, x, gate, up, down = _inputs(300, 136, 264)
    y, kept = sg.ffn(x, gate, up, down, keep=torch.bfloat16)
    first = [y.clone()] + [g.clone() for g in sg.ffn_backward(dy, x, gate, up, down, kept)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, kept = sg.ffn(x, gate, up, down, keep=torch.bfloat16)
        grads = sg.ffn_backward(dy, x, gate, up, down, kept)
    for _ in range(3):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first[0]) and all(torch.equal(a, b) for a, b in zip(grads, first[1:]))
    x2 = _inputs(300, 136, 264, seed=50)[1]
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, sg.ffn(x2, gate, up, down)[0])


def test_nothing_to_do():
    import torch
    dy, x, gate, up, down = _inputs(0, 32, 64)
    assert sg.ffn(x, gate, up, down)[0].shape == (0, 32)
    dgate, dup, ddown = (torch.full(s, 7.0, device="cuda") for s in ((64, 32), (64, 32), (32, 64)))
    kept = tuple(torch.empty((0, 64), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    sg.ffn_backward(dy, x, gate, up, down, kept, dgate=dgate, dup=dup, ddown=ddown, accumulate=True)
    assert all(bool((t == 7.0).all()) for t in (dgate, dup, ddown))
    sg.ffn_backward(dy, x, gate, up, down, kept, dgate=dgate, dup=dup, ddown=ddown)
    assert all(bool((t == 0.0).all()) for t in (dgate, dup, ddown))
    dy, x, gate, up, down = _inputs(5, 32, 0)
    y = torch.full((5, 32), 7.0, device="cuda", dtype=torch.bfloat16)
    assert bool((sg.ffn(x, gate, up, down, y=y)[0] == 0).all())
    dx = torch.full((5, 32), 7.0, device="cuda", dtype=torch.bfloat16)
    kept = tuple(torch.empty((5, 0), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    assert bool((sg.ffn_backward(dy, x, gate, up, down, kept, dx=dx)[0] == 0).all())


@pytest.mark.parametrize("T", [3, 200])
def test_non_finite(T):
    """Infinities and NaN reach the rows and groups that they belong to, and no others."""
    import torch
    dy, x, gate, up, down = _inputs(T, 96, 300)
    clean, kept0 = sg.ffn(x, gate, up, down, keep=torch.float8_e4m3fn)
    x = x.clone()
    x[1, 5] = float("nan")
    y, kept = sg.ffn(x, gate, up, down, keep=torch.float8_e4m3fn)
    assert bool(y[1].isnan().all()) and bool(kept[0][1].float().isnan().all())
    assert bool((kept[2][:, 1].float() == 2.0 ** -126).all())            # no finite value in the group
    others = [t for t in range(T) if t != 1]
    assert torch.equal(y[others], clean[others]) and torch.equal(kept[2][:, others], kept0[2][:, others])
    gate = gate.clone()
    gate[7] = 0
    gate[7, 0] = float("inf")
    x[1, 5], x[:, 0] = 1.0, 2.0
    y, kept = sg.ffn(x, gate, up, down, keep=torch.float8_e4m3fn)
    assert bool(kept[0][:, 7].float().isnan().all()) and not bool(kept[0][:, 8:].float().isnan().any())
    assert bool(kept[2].float().isfinite().all())
    y, kept = sg.ffn(x, gate, up, down, keep=torch.bfloat16)
    assert bool((kept[0][:, 7].float() == float("inf")).all())


def test_gradients_against_differences():
    """The 64-bit block's difference quotient along a direction is what the kernels' gradients give."""
    import torch
    T, D, F = 200, 64, 160
    dy, x, gate, up, down = _inputs(T, D, F)
    kept = sg.ffn(x, gate, up, down, ACT["gelu"], keep=torch.bfloat16)[1]
    new = [torch.empty(s, device="cuda") for s in ((F, D), (F, D), (D, F))]
    grads = sg.ffn_backward(dy, x, gate, up, down, kept, ACT["gelu"], dgate=new[0], dup=new[1], ddown=new[2])
    gen = torch.Generator(device="cuda").manual_seed(4)
    at = [t.double() for t in (x, gate, up, down)]
    along = [torch.randn(t.shape, generator=gen, device="cuda", dtype=torch.float64) for t in at]

    def loss(eps):
        x_, g_, u_, d_ = (a + eps * b for a, b in zip(at, along))
        return float((dy.double() * ((fp.act("gelu", x_ @ g_.t()) * (x_ @ u_.t())) @ d_.t())).sum())

    eps = 1e-5
    slope = (loss(eps) - loss(-eps)) / (2 * eps)
    mine = sum(float((g.double() * b).sum()) for g, b in zip(grads, along))
    # the kept values, dg, du, h and dx are rounded to bf16: each term of the sum is off by at most
    # a few 2^-8; the terms' size bounds the sum's error (their signs are as good as random)
    size = sum(float((g.double() * b).square().sum()) for g, b in zip(grads, along)) ** 0.5
    assert abs(mine - slope) <= 8 * fp.BF16 * size, (mine, slope, size)
