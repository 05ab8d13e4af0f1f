"""The 8-bit floating-point operators: quantisation with a scale for each group of
128, the matrix product of two such operands, and a mixture-of-experts layer over
such weights for a few tokens.

A quantised matrix is held as codes (float8_e4m3fn or float8_e5m2) and fp32
scales; the value is code * scale.  Groups are 128 long along the dimension
that a product sums over:

  rows    1 x 128   scales[col // 128][row]
  cols    128 x 1   scales[row // 128][col]
  blocks  128 x 128 scales[row // 128][col // 128]

`own` false: the operators in elementary torch operations in 32 bits.
`own` true: the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
GROUPS = {"rows": (1, 128), "cols": (128, 1), "blocks": (128, 128)}
SMALLEST_SCALE = 2.0 ** -126


def _blocks(n):
    return (n + 127) // 128


def listed():
    return [
        # a decode step's activations for a batch of 16 (latency)
        {"name": "quantize_decode", "op": "quantize", "rows": 16, "cols": 8192, "x": "bf16",
         "group": "rows", "q": "e4m3"},
        # an output gradient with odd sizes, in groups along the tokens for the weight gradient
        {"name": "quantize_grad_ragged", "op": "quantize", "rows": 4095, "cols": 1537, "x": "f32",
         "group": "cols", "q": "e5m2"},
        # a weight matrix after an optimiser step
        {"name": "quantize_weight", "op": "quantize", "rows": 16384, "cols": 8192, "x": "f32",
         "group": "blocks", "q": "e4m3"},
        # the smallest layer: one launch's latency
        {"name": "product_256", "op": "product", "M": 256, "N": 256, "K": 256, "ta": "N", "tb": "T",
         "a": "e4m3", "b": "e4m3", "ga": 1, "gb": 128, "c": "bf16", "beta": 0.0},
        # one token against a large weight matrix
        {"name": "product_decode_m1", "op": "product", "M": 1, "N": 16384, "K": 8192, "ta": "N",
         "tb": "T", "a": "e4m3", "b": "e4m3", "ga": 1, "gb": 128, "c": "bf16", "beta": 0.0},
        # a decode batch of 16, fp32 result
        {"name": "product_decode_m16", "op": "product", "M": 16, "N": 16384, "K": 8192, "ta": "N",
         "tb": "T", "a": "e4m3", "b": "e4m3", "ga": 1, "gb": 128, "c": "f32", "beta": 0.0},
        # input gradient (weights read along their rows), odd sizes and odd leading dimensions
        {"name": "product_dgrad_ragged", "op": "product", "M": 4095, "N": 3073, "K": 1537, "ta": "N",
         "tb": "N", "a": "e5m2", "b": "e4m3", "ga": 1, "gb": 128, "c": "f32", "beta": 0.0},
        # weight gradient added to an fp32 accumulator: both operands summed along the tokens
        {"name": "product_wgrad", "op": "product", "M": 4096, "N": 4096, "K": 8192, "ta": "T",
         "tb": "N", "a": "e5m2", "b": "e4m3", "ga": 1, "gb": 1, "c": "f32", "beta": 1.0},
        # a large forward product (training or prefill)
        {"name": "product_8192", "op": "product", "M": 8192, "N": 8192, "K": 8192, "ta": "N",
         "tb": "T", "a": "e4m3", "b": "e4m3", "ga": 1, "gb": 128, "c": "bf16", "beta": 0.0},
        # one token through a small layer (latency)
        {"name": "moe_t1_small", "op": "moe", "T": 1, "D": 1024, "F": 512, "E": 8, "topk": 2,
         "x": "bf16", "renorm": True},
        # a few tokens through a large layer: most of the time is the experts' weights
        {"name": "moe_t4", "op": "moe", "T": 4, "D": 4096, "F": 2048, "E": 64, "topk": 8,
         "x": "bf16", "renorm": True},
        # a decode batch of 64 in fp32, every expert in use
        {"name": "moe_t64", "op": "moe", "T": 64, "D": 2048, "F": 1024, "E": 32, "topk": 4,
         "x": "f32", "renorm": False},
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of the range; half of them multiples of 16."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5:
        n = (n + 15) // 16 * 16
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "moe"])
    if op == "quantize":
        while True:
            rows, cols = _size(rng, 1, 16384), _size(rng, 16, 16384)
            if rows * cols <= 16384 * 8192:
                return {"op": op, "rows": rows, "cols": cols, "x": rng.choice(["f32", "bf16"]),
                        "group": rng.choice(["rows", "cols", "blocks"]),
                        "q": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "product":
        while True:
            M, N, K = _size(rng, 1, 16384), _size(rng, 16, 16384), _size(rng, 16, 16384)
            if M * N * K <= 8192 ** 3 and max(M * N, M * K, N * K) <= 16384 * 8192:
                break
        ta, tb = rng.choice([("N", "T"), ("N", "T"), ("N", "N"), ("T", "N"), ("T", "T")])
        return {"op": op, "M": M, "N": N, "K": K, "ta": ta, "tb": tb,
                "a": rng.choice(["e4m3", "e4m3", "e5m2"]), "b": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "ga": rng.choice([1, 1, 128]), "gb": rng.choice([1, 128, 128]),
                "c": rng.choice(["f32", "bf16"]), "beta": rng.choice([0.0, 0.0, 1.0])}
    while True:
        T, E = _size(rng, 1, 64), rng.randint(2, 96)
        topk = rng.randint(1, min(8, E))
        D, F = _size(rng, 256, 4096), _size(rng, 128, 4096)
        if T * topk * D * F <= 64 * 4 * 2048 * 1024 and E * D * F <= 64 * 4096 * 2048:
            return {"op": op, "T": T, "D": D, "F": F, "E": E, "topk": topk,
                    "x": rng.choice(["f32", "bf16"]), "renorm": rng.random() < 0.5}


# ----------------------------------------------------------------- the inputs
def _codes(gen, shape, q, ld=None):
    """Codes as the quantiser leaves them: a normal distribution whose largest
    value in a group is near the format's largest.  `ld`: elements from row to row."""
    full = list(shape[:-1]) + [ld or shape[-1]]
    v = torch.randn(full, generator=gen, device=DEV, dtype=torch.float32)
    v *= LARGEST[q] / 4.0
    return v.clamp_(-LARGEST[q], LARGEST[q]).to(TYPES[q])[..., : shape[-1]]


def _scales(gen, shape, typical):
    """Scales within a factor of 4 of a typical one (groups differ in their largest value)."""
    return torch.exp2(torch.rand(shape, generator=gen, device=DEV) * 4.0 - 2.0) * typical


def _scale_shape(mn, k, trans_k_first, group):
    """Scales of an operand with `mn` rows or columns and a sum of length `k`."""
    if group == 1:
        return (_blocks(k), mn)
    return (_blocks(k), _blocks(mn)) if trans_k_first else (_blocks(mn), _blocks(k))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        # activations and gradients: some channels are much larger than others
        x = torch.randn((rows, cols), generator=gen, device=DEV)
        x *= torch.exp(torch.randn((1, cols), generator=gen, device=DEV))
        gr, gc = GROUPS[case["group"]]
        shape = (_blocks(cols), rows) if (gr, gc) == (1, 128) else (_blocks(rows), -(-cols // gc))
        return {"case": case, "x": x.to(TYPES[case["x"]]),
                "q": torch.empty((rows, cols), device=DEV, dtype=TYPES[case["q"]]),
                "s": torch.empty(shape, device=DEV, dtype=torch.float32)}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        a = _codes(gen, (M, K) if case["ta"] == "N" else (K, M), case["a"])
        b = _codes(gen, (K, N) if case["tb"] == "N" else (N, K), case["b"])
        sa = _scales(gen, _scale_shape(M, K, case["ta"] == "T", case["ga"]), 4.0 / LARGEST[case["a"]])
        sb = _scales(gen, _scale_shape(N, K, case["tb"] == "N", case["gb"]),
                     4.0 / LARGEST[case["b"]] / math.sqrt(K))
        if case["beta"]:
            c = torch.randn((M, N), generator=gen, device=DEV).to(TYPES[case["c"]])
        else:
            c = torch.empty((M, N), device=DEV, dtype=TYPES[case["c"]])
        return {"case": case, "a": a, "sa": sa, "b": b, "sb": sb, "c": c}
    T, D, F, E, topk = case["T"], case["D"], case["F"], case["E"], case["topk"]
    pad = lambda n: (n + 15) // 16 * 16  # noqa: E731  (rows of the weights start on 16 bytes)
    s = {"case": case, "x": torch.randn((T, D), generator=gen, device=DEV).to(TYPES[case["x"]]),
         "router": torch.randn((E, D), generator=gen, device=DEV) / math.sqrt(D)}
    for name, n, k in (("gate", F, D), ("up", F, D), ("down", D, F)):
        s[name] = _codes(gen, (E, n, k), "e4m3", pad(k))
        s["s_" + name] = _scales(gen, (E, _blocks(n), _blocks(k)), 4.0 / 448.0 / math.sqrt(k))
    s["y"] = torch.empty((T, D), device=DEV, dtype=s["x"].dtype)
    s["logits"] = torch.empty((T, E), device=DEV)
    s["indices"] = torch.empty((T, topk), device=DEV, dtype=torch.int32)
    s["weights"] = torch.empty((T, topk), device=DEV)
    return s


# ----------------------------------------------------------- the plain forms
def _spread(s, rows, cols, gr, gc):
    """The scale of each value of a rows x cols matrix."""
    if gr == 128:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :cols] if gc == 128 else s


def _plain_quantize(x, group, q):
    gr, gc = GROUPS[group]
    rows, cols = x.shape
    x = x.float()
    up = lambda n, g: -(-n // g) * g  # noqa: E731
    size = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    size = torch.nn.functional.pad(size, (0, up(cols, gc) - cols, 0, up(rows, gr) - rows))
    amax = size.view(up(rows, gr) // gr, gr, up(cols, gc) // gc, gc).amax((1, 3))
    # (a division by a tensor: one by a number is taken as a product with its reciprocal)
    s = (amax / torch.full_like(amax, LARGEST[q])).clamp_min(SMALLEST_SCALE)
    inverse = torch.ones_like(s) / s
    codes = (x * _spread(inverse, rows, cols, gr, gc)).to(TYPES[q])
    return codes, s.t().contiguous() if group == "rows" else s


def _plain_values(codes, s, group, k_first):
    """The values of an operand, 32 bits, as stored."""
    rows, cols = codes.shape
    if group == 128:
        return codes.float() * _spread(s, rows, cols, 128, 128)
    return codes.float() * (_spread(s, rows, cols, 128, 1) if k_first
                            else _spread(s.t(), rows, cols, 1, 128))


def _plain_product(s):
    case = s["case"]
    a = _plain_values(s["a"], s["sa"], case["ga"], case["ta"] == "T")
    b = _plain_values(s["b"], s["sb"], case["gb"], case["tb"] == "N")
    c = (a.t() if case["ta"] == "T" else a) @ (b.t() if case["tb"] == "T" else b)
    if case["beta"]:
        c = c + case["beta"] * s["c"].float()
    s["c"].copy_(c)
    return s["c"]


def _plain_experts(codes, s, which):
    """The chosen experts' matrices in 32 bits: one for each token's each choice."""
    n, k = codes.shape[1:]
    v = codes.view(torch.uint8)[which].view(codes.dtype).float()
    sc = s[which].repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]
    return v.mul_(sc)


def _plain_moe(s):
    case, x = s["case"], s["x"].float()
    T, topk = case["T"], case["topk"]
    logits = x @ s["router"].t()
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices
    chosen = order[:, :topk]
    p = torch.softmax(logits, 1).gather(1, chosen)
    if case["renorm"]:
        p = p / p.sum(1, keepdim=True)
    which = chosen.reshape(-1)
    rows = x.repeat_interleave(topk, 0).unsqueeze(2)
    gate = torch.bmm(_plain_experts(s["gate"], s["s_gate"], which), rows)
    up = torch.bmm(_plain_experts(s["up"], s["s_up"], which), rows)
    h = gate / (1.0 + torch.exp(-gate)) * up
    out = torch.bmm(_plain_experts(s["down"], s["s_down"], which), h).view(T, topk, -1)
    y = (out * p.unsqueeze(2)).sum(1)
    return {"y": y.to(s["x"].dtype), "logits": logits, "indices": chosen.to(torch.int32), "weights": p}


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import dense_fp32_gemm_05_gb300 as sg

        if op == "quantize":
            return sg.fp8_quantize(state["x"], GROUPS[case["group"]], Q=state["q"], S=state["s"])
        if op == "product":
            return sg.fp8_gemm(state["a"], state["sa"], state["b"], state["sb"], state["c"],
                               case["ta"], case["tb"], beta=case["beta"], a_group=case["ga"],
                               b_group=case["gb"])
        y, logits, indices, weights = sg.moe(
            state["x"], state["router"], state["gate"], state["s_gate"], state["up"],
            state["s_up"], state["down"], state["s_down"], case["topk"],
            renormalize=case["renorm"], y=state["y"], logits=state["logits"],
            indices=state["indices"], weights=state["weights"])
        return {"y": y, "logits": logits, "indices": indices, "weights": weights}
    if op == "quantize":
        return _plain_quantize(state["x"], case["group"], case["q"])
    if op == "product":
        return _plain_product(state)
    return _plain_moe(state)


# ---------------------------------------------------------------- the floors
def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op == "quantize":
        rows, cols = case["rows"], case["cols"]
        gr, gc = GROUPS[case["group"]]
        return {"bytes": rows * cols * (size[case["x"]] + 1) + 4 * (-(-rows // gr)) * (-(-cols // gc)),
                "flops": 3 * rows * cols}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        scales = _blocks(K) * (-(-M // case["ga"]) + -(-N // case["gb"]))
        return {"bytes": M * K + N * K + 4 * scales +
                M * N * size[case["c"]] * (2 if case["beta"] else 1),
                "flops": 2 * M * N * K}
    T, D, F, E, topk = case["T"], case["D"], case["F"], case["E"], case["topk"]
    used = E * (1.0 - (1.0 - topk / E) ** T)      # experts that some token chose, on average
    return {"bytes": used * 3 * D * F * (1 + 4 / 128 / 128) + 4 * E * D + 2 * T * D * size[case["x"]] +
            4 * T * (E + 2 * topk),
            "flops": 2 * T * topk * 3 * D * F + 2 * T * E * D}


# ------------------------------------------- the definitions, evaluated in 64 bits
def _exact_scales_of(index_mn, index_k, s, group, k_first):
    if group == 1:
        return s.double()[(index_k // 128)[:, None], index_mn[None, :]]
    if k_first:
        return s.double()[(index_k // 128)[:, None], (index_mn // 128)[None, :]]
    return s.double()[(index_mn // 128)[None, :], (index_k // 128)[:, None]]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].double()
        rows, cols = x.shape
        gr, gc = GROUPS[case["group"]]
        scales = torch.zeros((-(-rows // gr), -(-cols // gc)), dtype=torch.float64, device=DEV)
        r, c = torch.arange(rows, device=DEV) // gr, torch.arange(cols, device=DEV) // gc
        where = (r[:, None] * scales.shape[1] + c[None, :]).reshape(-1)
        scales.view(-1).scatter_reduce_(0, where, x.abs().reshape(-1), "amax")
        scales = torch.clamp(scales / LARGEST[case["q"]], min=SMALLEST_SCALE)
        codes = (x / scales[r[:, None], c[None, :]]).to(TYPES[case["q"]])
        return codes, scales.t().contiguous() if case["group"] == "rows" else scales
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        k = torch.arange(K, device=DEV)
        a = s["a"].double() if case["ta"] == "T" else s["a"].double().t()     # K x M
        a = a * _exact_scales_of(torch.arange(M, device=DEV), k, s["sa"], case["ga"], case["ta"] == "T")
        b = s["b"].double() if case["tb"] == "N" else s["b"].double().t()     # K x N
        b = b * _exact_scales_of(torch.arange(N, device=DEV), k, s["sb"], case["gb"], case["tb"] == "N")
        c = torch.mm(a.t(), b)
        return c + case["beta"] * s["c"].double() if case["beta"] else c
    T, D, E, topk = case["T"], case["D"], case["E"], case["topk"]
    x = s["x"].double()
    logits = x.mm(s["router"].double().t())
    p = torch.exp(logits - logits.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True)
    chosen = torch.argsort(-logits, dim=1, stable=True)[:, :topk]
    weights = torch.stack([p[t, chosen[t]] for t in range(T)])
    if case["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    y = torch.zeros((T, D), dtype=torch.float64, device=DEV)
    for e in range(E):
        tokens, place = torch.nonzero(chosen == e, as_tuple=True)
        if len(tokens) == 0:
            continue
        m = {}
        for name in ("gate", "up", "down"):
            w = s[name][e].double()
            i, j = torch.arange(w.shape[0], device=DEV) // 128, torch.arange(w.shape[1], device=DEV) // 128
            m[name] = w * s["s_" + name][e].double()[i[:, None], j[None, :]]
        g, u = x[tokens].mm(m["gate"].t()), x[tokens].mm(m["up"].t())
        y.index_add_(0, tokens, (g * torch.sigmoid(g) * u).mm(m["down"].t()) * weights[tokens, place][:, None])
    return {"y": y, "logits": logits, "indices": None, "weights": weights}
