"""Feed-forward layers: a gated block trained in bf16, with its intermediate values kept
for the backward pass in 16 or 8 bits, and matrices of 4-bit weights for serving.

  ffn           g = x gate^T, u = x up^T, y = (act(g) * u) down^T, and g and u kept
  ffn_backward  the gradients of x, gate, up and down from dy and what was kept
  q4_quantize   codes of 4 bits with a scale (and a zero code) for each group of a row
  q4_gemm       x W^T, or act(x gate^T) * (x up^T), with such matrices, for few rows of x

Kept in 8 bits, g and u are codes (float8_e4m3fn) and bf16 scales, one for each 128
neighbours in a row, scales[column // 128][row]; the value is code * scale.  A 4-bit matrix
is two codes in a byte, the even column's in the low half, and scales[column // group][row];
the value is (code - zero) * scale, zero 8 where no zero codes are given.

`own` false: the operators in elementary torch operations in 32 bits.
`own` true: the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SMALLEST_SCALE = 2.0 ** -126
LARGEST = 448.0                      # of float8_e4m3fn


def _groups(n, group=128):
    return (n + group - 1) // group


def listed():
    return [
        # one token through a block: its weights are read once
        {"name": "ffn_t1", "op": "ffn", "T": 1, "D": 4096, "F": 8192, "act": "silu", "save": "none"},
        # a short prompt, odd sizes, rows of the matrices apart
        {"name": "ffn_t100_ragged", "op": "ffn", "T": 100, "D": 1001, "F": 2731, "act": "gelu", "save": "none"},
        # a training step's forward pass, values kept in 16 bits
        {"name": "ffn_train_bf16", "op": "ffn", "T": 4096, "D": 2048, "F": 8192, "act": "silu", "save": "bf16"},
        # a large training step's, kept in 8 bits
        {"name": "ffn_train_e4m3", "op": "ffn", "T": 8192, "D": 4096, "F": 8192, "act": "silu", "save": "e4m3"},
        # the backward pass of a small batch, odd sizes
        {"name": "backward_ragged_bf16", "op": "ffn_backward", "T": 777, "D": 1000, "F": 2501, "act": "gelu",
         "save": "bf16"},
        # the backward pass of a large step from values kept in 8 bits
        {"name": "backward_e4m3", "op": "ffn_backward", "T": 4096, "D": 4096, "F": 8192, "act": "silu",
         "save": "e4m3"},
        # a trained matrix made ready for serving
        {"name": "q4_quantize_weight", "op": "q4_quantize", "rows": 8192, "cols": 4096, "w": "f32", "group": 128,
         "symmetric": True},
        # odd sizes, short groups with zero codes
        {"name": "q4_quantize_ragged", "op": "q4_quantize", "rows": 1537, "cols": 4095, "w": "bf16", "group": 32,
         "symmetric": False},
        # a small matrix and one token (latency)
        {"name": "q4_small", "op": "q4_gemm", "M": 1, "N": 1024, "K": 1024, "group": 128, "zeros": False,
         "gated": False, "x": "bf16", "c": "bf16", "act": "none"},
        # one token against a large matrix
        {"name": "q4_m1", "op": "q4_gemm", "M": 1, "N": 16384, "K": 8192, "group": 128, "zeros": False,
         "gated": False, "x": "bf16", "c": "bf16", "act": "none"},
        # four tokens through both input matrices of a gated block, short groups with zero codes
        {"name": "q4_gated_m4", "op": "q4_gemm", "M": 4, "N": 8192, "K": 4096, "group": 64, "zeros": True,
         "gated": True, "x": "bf16", "c": "bf16", "act": "silu"},
        # a decode batch in fp32
        {"name": "q4_m16_f32", "op": "q4_gemm", "M": 16, "N": 4096, "K": 8192, "group": 128, "zeros": True,
         "gated": False, "x": "f32", "c": "f32", "act": "none"},
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of the range; half of them multiples of 16."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5:
        n = (n + 15) // 16 * 16
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_backward", "ffn_backward", "q4_quantize", "q4_gemm", "q4_gemm"])
    if op in ("ffn", "ffn_backward"):
        most = 8192 * 4096 * 8192 // (1 if op == "ffn" else 2)
        while True:
            T, D, F = _size(rng, 1, 8192), _size(rng, 64, 4096), _size(rng, 64, 8192)
            if T * D * F <= most:
                break
        return {"op": op, "T": T, "D": D, "F": F, "act": rng.choice(["silu", "silu", "gelu", "relu"]),
                "save": rng.choice(["none", "bf16", "e4m3"] if op == "ffn" else ["bf16", "e4m3"])}
    if op == "q4_quantize":
        return {"op": op, "rows": _size(rng, 1, 8192), "cols": _size(rng, 16, 4096),
                "w": rng.choice(["f32", "bf16"]), "group": rng.choice([32, 64, 128]),
                "symmetric": rng.random() < 0.5}
    while True:
        M, N, K = _size(rng, 1, 64), _size(rng, 16, 16384), _size(rng, 32, 8192)
        gated = rng.random() < 0.5
        if (2 if gated else 1) * N * K <= 16384 * 8192:
            break
    return {"op": op, "M": M, "N": N, "K": K, "group": rng.choice([32, 64, 128, 128]),
            "zeros": rng.random() < 0.5, "gated": gated, "x": rng.choice(["bf16", "bf16", "f32"]),
            "c": rng.choice(["bf16", "f32"]), "act": rng.choice(["silu", "gelu"]) if gated else "none"}


# ----------------------------------------------------------------- the inputs
def _rows(shape, step, dtype):
    """An empty matrix whose rows start `step` elements or a multiple apart."""
    rows, cols = shape
    return torch.empty((rows, (cols + step - 1) // step * step), device=DEV, dtype=dtype)[:, :cols]


def _matrix(gen, shape, size, spread=0.0):
    """bf16 values of a normal distribution, some columns larger than others by exp(spread * normal)."""
    v = torch.randn(shape, generator=gen, device=DEV)
    if spread:
        v *= torch.exp(torch.randn((1, shape[1]), generator=gen, device=DEV) * spread)
    return _rows(shape, 8, torch.bfloat16).copy_(v.mul_(size))


def _kept_buffers(T, F, save):
    if save == "bf16":
        return [torch.empty((T, F), device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    return ([torch.empty((T, F), device=DEV, dtype=torch.float8_e4m3fn) for _ in range(2)] +
            [torch.empty((_groups(F), T), device=DEV, dtype=torch.bfloat16) for _ in range(2)])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op = case["op"]
    if op in ("ffn", "ffn_backward"):
        T, D, F = case["T"], case["D"], case["F"]
        s = {"case": case, "x": _matrix(gen, (T, D), 1.0, 0.5)}
        s["gate"], s["up"] = (_matrix(gen, (F, D), 1.0 / math.sqrt(D)) for _ in range(2))
        s["down"] = _matrix(gen, (D, F), 1.0 / math.sqrt(F))
        s["h"] = _rows((T, F), 8, torch.bfloat16)
        if op == "ffn":
            s["y"] = torch.empty((T, D), device=DEV, dtype=torch.bfloat16)
            s["kept"] = None if case["save"] == "none" else _kept_buffers(T, F, case["save"])
            return s
        # what a forward pass kept
        g, u = (s["x"].float() @ s[n].float().t() for n in ("gate", "up"))
        if case["save"] == "bf16":
            s["kept"] = [g.to(torch.bfloat16), u.to(torch.bfloat16)]
        else:
            (qg, sg), (qu, su) = _plain_keep(g), _plain_keep(u)
            s["kept"] = [qg, qu, sg, su]
        s["dy"] = _matrix(gen, (T, D), 0.01, 0.5)
        s["dg"], s["du"] = (_rows((T, F), 8, torch.bfloat16) for _ in range(2))
        for name, like in (("dx", "x"), ("dgate", "gate"), ("dup", "up"), ("ddown", "down")):
            s[name] = torch.empty(s[like].shape, device=DEV, dtype=torch.bfloat16)
        return s
    if op == "q4_quantize":
        rows, cols = case["rows"], case["cols"]
        w = torch.randn((rows, cols), generator=gen, device=DEV) / math.sqrt(cols)
        w *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device=DEV))
        if not case["symmetric"]:
            w += 0.5 / math.sqrt(cols)
        groups = _groups(cols, case["group"])
        return {"case": case, "w": w.to(TYPES[case["w"]]), "q": _rows((rows, (cols + 1) // 2), 16, torch.uint8),
                "s": torch.empty((groups, rows), device=DEV),
                "z": None if case["symmetric"] else torch.empty((groups, rows), device=DEV, dtype=torch.uint8),
                "v": torch.empty((rows, cols), device=DEV)}
    M, N, K, group = case["M"], case["N"], case["K"], case["group"]
    s = {"case": case, "x": torch.randn((M, K), generator=gen, device=DEV).to(TYPES[case["x"]]),
         "c": torch.empty((M, N), device=DEV, dtype=TYPES[case["c"]])}
    for name in ("w", "up") if case["gated"] else ("w",):
        q = _rows((N, (K + 1) // 2), 16, torch.uint8)
        q.copy_(torch.randint(0, 256, q.shape, generator=gen, device=DEV, dtype=torch.uint8))
        if K % 2:
            q[:, -1] &= 15               # no code past the last column
        s[name] = q
        # scales within a factor of 4 of one another
        s["s_" + name] = (torch.exp2(torch.rand((_groups(K, group), N), generator=gen, device=DEV) * 2.0 - 1.0) *
                          (0.25 / math.sqrt(K)))
        s["z_" + name] = (torch.randint(4, 12, (_groups(K, group), N), generator=gen, device=DEV, dtype=torch.uint8)
                          if case["zeros"] else None)
    return s


# ----------------------------------------------------------- the plain forms
def _plain_gate(act, g):
    """The factor of g in act(g), and the derivative of act."""
    if act == "none":
        return torch.ones_like(g), torch.ones_like(g)
    if act == "relu":
        step = (g > 0).float()
        return step, step
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return p, p * (1.0 + g * (1.0 - p))
    # gelu in its tanh form, g (1 + tanh(v)) / 2 = g / (1 + exp(-2 v))
    c, a = 2.0 * math.sqrt(2.0 / math.pi), 0.044715
    p = 1.0 / (1.0 + torch.exp(-c * (g + a * g * g * g)))
    return p, p * (1.0 + g * (1.0 - p) * c * (1.0 + 3.0 * a * g * g))


def _plain_keep(v):
    """Codes and scales, a scale for each 128 of a row."""
    T, F = v.shape
    n = _groups(F)
    full = torch.nn.functional.pad(v, (0, n * 128 - F)).view(T, n, 128)
    amax = full.abs().amax(2)
    s = (amax / torch.full_like(amax, LARGEST)).clamp_min(SMALLEST_SCALE).to(torch.bfloat16)
    inverse = torch.ones_like(amax) / s.float()
    codes = (full * inverse.unsqueeze(2)).clamp(-LARGEST, LARGEST).to(torch.float8_e4m3fn)
    return codes.view(T, n * 128)[:, :F].contiguous(), s.t().contiguous()


def _plain_kept(kept):
    if len(kept) == 2:
        return [v.float() for v in kept]
    F = kept[0].shape[1]
    return [q.float() * s.float().t().repeat_interleave(128, 1)[:, :F] for q, s in zip(kept[:2], kept[2:])]


def _plain_ffn(s):
    case, x = s["case"], s["x"].float()
    g, u = x @ s["gate"].float().t(), x @ s["up"].float().t()
    out = {"y": ((g * _plain_gate(case["act"], g)[0] * u) @ s["down"].float().t()).to(torch.bfloat16)}
    if case["save"] == "bf16":
        out["g"], out["u"] = g.to(torch.bfloat16), u.to(torch.bfloat16)
    elif case["save"] == "e4m3":
        (out["g"], out["sg"]), (out["u"], out["su"]) = _plain_keep(g), _plain_keep(u)
    return out


def _plain_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    g, u = _plain_kept(s["kept"])
    p, slope = _plain_gate(s["case"]["act"], g)
    dh = dy @ s["down"].float()
    a = g * p
    dg, du = dh * u * slope, dh * a
    out = {"dx": dg @ s["gate"].float() + du @ s["up"].float(), "dgate": dg.t() @ x, "dup": du.t() @ x,
           "ddown": dy.t() @ (a * u)}
    return {n: v.to(torch.bfloat16) for n, v in out.items()}


def _plain_q4_quantize(s):
    case = s["case"]
    rows, cols, group = case["rows"], case["cols"], case["group"]
    n = _groups(cols, group)
    w = torch.nn.functional.pad(s["w"].float(), (0, n * group - cols)).view(rows, n, group)
    if case["symmetric"]:
        amax = w.abs().amax(2)
        scale = (amax / torch.full_like(amax, 7.0)).clamp_min(SMALLEST_SCALE)
        zero = torch.full_like(scale, 8.0)
    else:
        high, low = w.amax(2).clamp_min(0.0), w.amin(2).clamp_max(0.0)
        fifteen = torch.full_like(high, 15.0)
        scale = (high / fifteen - low / fifteen).clamp_min(SMALLEST_SCALE)
        zero = torch.round(-low * (torch.ones_like(scale) / scale)).clamp(0.0, 15.0)
    inverse = torch.ones_like(scale) / scale
    code = (torch.round(w * inverse.unsqueeze(2)) + zero.unsqueeze(2)).clamp(0.0, 15.0)
    value = ((code - zero.unsqueeze(2)) * scale.unsqueeze(2)).view(rows, n * group)[:, :cols]
    code = code.view(rows, n * group)[:, :cols].to(torch.uint8)
    code = torch.nn.functional.pad(code, (0, cols % 2))
    return {"q": code[:, 0::2] | (code[:, 1::2] << 4), "s": scale.t().contiguous(),
            "z": None if case["symmetric"] else zero.t().to(torch.uint8), "v": value.contiguous()}


def _plain_q4_values(q, scale, zero, K, group):
    code = torch.stack([q & 15, q >> 4], 2).view(q.shape[0], -1)[:, :K].float()
    code -= 8.0 if zero is None else zero.t().float().repeat_interleave(group, 1)[:, :K]
    return code * scale.t().repeat_interleave(group, 1)[:, :K]


def _plain_q4_gemm(s):
    case, x = s["case"], s["x"].float()
    K, group = case["K"], case["group"]
    c = x @ _plain_q4_values(s["w"], s["s_w"], s["z_w"], K, group).t()
    if case["gated"]:
        c = c * _plain_gate(case["act"], c)[0] * (x @ _plain_q4_values(s["up"], s["s_up"], s["z_up"], K, group).t())
    return c.to(TYPES[case["c"]])


# -------------------------------------------------------------------- one pass
def _own(s):
    import dense_fp32_gemm_05_gb300 as sg

    case = s["case"]
    act = {"none": sg.ACT_NONE, "relu": sg.ACT_RELU, "silu": sg.ACT_SILU, "gelu": sg.ACT_GELU}.get(case.get("act"))
    if case["op"] == "ffn":
        y, kept = sg.ffn(s["x"], s["gate"], s["up"], s["down"], act, kept=s["kept"], y=s["y"], h=s["h"])
        return {"y": y, **dict(zip(("g", "u", "sg", "su"), kept or ()))}
    if case["op"] == "ffn_backward":
        grads = sg.ffn_backward(s["dy"], s["x"], s["gate"], s["up"], s["down"], s["kept"], act, dx=s["dx"],
                                dgate=s["dgate"], dup=s["dup"], ddown=s["ddown"],
                                scratch=(s["dg"], s["du"], s["h"]))
        return dict(zip(("dx", "dgate", "dup", "ddown"), grads))
    if case["op"] == "q4_quantize":
        q, scale, zero = sg.q4_quantize(s["w"], case["group"], case["symmetric"], Q=s["q"], S=s["s"], Z=s["z"],
                                        V=s["v"])
        return {"q": q, "s": scale, "z": zero, "v": s["v"]}
    up = {"Q2": s["up"], "S2": s["s_up"], "Z2": s["z_up"]} if case["gated"] else {}
    return sg.q4_gemm(s["x"], s["w"], s["s_w"], s["c"], s["z_w"], group=case["group"], activation=act, **up)


def run(state):
    if own:
        return _own(state)
    return {"ffn": _plain_ffn, "ffn_backward": _plain_backward, "q4_quantize": _plain_q4_quantize,
            "q4_gemm": _plain_q4_gemm}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the floors
def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op in ("ffn", "ffn_backward"):
        T, D, F = case["T"], case["D"], case["F"]
        kept = 2 * T * {"none": 0, "bf16": 2 * F, "e4m3": F + 2 * _groups(F)}[case["save"]]
        if op == "ffn":
            return {"bytes": 2 * (3 * D * F + 2 * T * D) + kept, "flops": 6 * T * D * F}
        return {"bytes": 2 * (6 * D * F + 3 * T * D) + kept, "flops": 12 * T * D * F}
    if op == "q4_quantize":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": rows * (cols * (size[case["w"]] + 4) + (cols + 1) // 2 +
                                 _groups(cols, case["group"]) * (4 if case["symmetric"] else 5)),
                "flops": 5 * rows * cols}
    M, N, K = case["M"], case["N"], case["K"]
    two = 2 if case["gated"] else 1
    return {"bytes": two * N * ((K + 1) // 2 + _groups(K, case["group"]) * (5 if case["zeros"] else 4)) +
            M * K * size[case["x"]] + M * N * size[case["c"]],
            "flops": two * 2 * M * N * K}


# ------------------------------------------- the definitions, evaluated in 64 bits
def _exact_act(act, g):
    if act == "silu":
        return g * torch.sigmoid(g)
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3)))
    return torch.relu(g) if act == "relu" else g


def _exact_slope(act, g):
    if act == "silu":
        p = torch.sigmoid(g)
        return p + g * p * (1.0 - p)
    if act == "gelu":
        t = torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 0.134145 * g * g)
    return torch.heaviside(g, torch.zeros_like(g)) if act == "relu" else torch.ones_like(g)


def _exact_keep(v):
    """What the codes of v round, and the scales before their rounding."""
    T, F = v.shape
    s = torch.zeros((T, _groups(F)), dtype=torch.float64, device=DEV)
    column = (torch.arange(F, device=DEV) // 128).expand(T, F)
    s.scatter_reduce_(1, column, v.abs(), "amax")
    s = torch.clamp(s / LARGEST, min=SMALLEST_SCALE)
    rounded = s.to(torch.bfloat16).double()
    return v / rounded.gather(1, column), s.t().contiguous()


def _exact_kept(kept, T, F):
    if len(kept) == 2:
        return kept[0].double(), kept[1].double()
    column = torch.arange(F, device=DEV) // 128
    return tuple(kept[i].double() * kept[i + 2].double()[column].t() for i in range(2))


def _exact_weight(s, name, case):
    K, group = case["K"], case["group"]
    k = torch.arange(K, device=DEV)
    code = (s[name].long()[:, k // 2] >> (4 * (k % 2))) & 15
    zero = s["z_" + name].long()[k // group].t() if case["zeros"] else 8
    return (code - zero).double() * s["s_" + name].double()[k // group].t()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "ffn":
        x = s["x"].double()
        g, u = x.mm(s["gate"].double().t()), x.mm(s["up"].double().t())
        out = {"y": (_exact_act(case["act"], g) * u).mm(s["down"].double().t())}
        if case["save"] == "bf16":
            out["g"], out["u"] = g, u
        elif case["save"] == "e4m3":
            (out["g"], out["sg"]), (out["u"], out["su"]) = _exact_keep(g), _exact_keep(u)
        return out
    if op == "ffn_backward":
        g, u = _exact_kept(s["kept"], case["T"], case["F"])
        x, dy = s["x"].double(), s["dy"].double()
        dh = dy.mm(s["down"].double())
        dg = dh * u * _exact_slope(case["act"], g)
        du = dh * _exact_act(case["act"], g)
        return {"dx": torch.addmm(dg.mm(s["gate"].double()), du, s["up"].double()), "dgate": dg.t().mm(x),
                "dup": du.t().mm(x), "ddown": dy.t().mm(_exact_act(case["act"], g) * u)}
    if op == "q4_quantize":
        w, group = s["w"].double(), case["group"]
        rows, cols = w.shape
        column = (torch.arange(cols, device=DEV) // group).expand(rows, cols)
        empty = torch.zeros((rows, _groups(cols, group)), dtype=torch.float64, device=DEV)
        if case["symmetric"]:
            scale = empty.scatter_reduce(1, column, w.abs(), "amax") / 7.0
        else:
            scale = (empty.scatter_reduce(1, column, w, "amax") - empty.scatter_reduce(1, column, w, "amin")) / 15.0
        # (codes and their values next to a border are as the 32-bit steps have them)
        return {"q": None, "s": torch.clamp(scale, min=SMALLEST_SCALE).t().contiguous(), "z": None, "v": None}
    x = s["x"].double()
    c = x.mm(_exact_weight(s, "w", case).t())
    return _exact_act(case["act"], c) * x.mm(_exact_weight(s, "up", case).t()) if case["gated"] else c
