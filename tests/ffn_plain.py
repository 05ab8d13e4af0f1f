"""The gated feed-forward block in 64 bits, with bounds on the error that the kernels'
arithmetic may make, and buffers whose surroundings are checked.

Bounds, from the arithmetic (half steps of a rounding: bf16 2^-8, fp32 2^-24, E4M3 2^-4):
a sum of K exact products in fp32 is off by at most (K + 16) 2^-23 sum |terms| (a
rounding or truncation for each); the activation and its derivative, an exponential, a
quotient and a few products in fp32, by 2^-19 (1 + |g|) of 1 (the exponential's relative
error grows with its argument); each rounding to bf16 by 2^-8 of the value."""
import math

import torch

BF16 = 2.0 ** -8
SUM = 2.0 ** -23
TINY = 2.0 ** -120                 # below what is told apart from zero
ACTS = ("none", "relu", "silu", "gelu")
C, A = math.sqrt(2 / math.pi), 0.044715


def act(name, g):
    if name == "none":
        return g
    if name == "relu":
        return torch.where(g < 0, torch.zeros_like(g), g)
    if name == "silu":
        return g / (1 + torch.exp(-g))
    return g / (1 + torch.exp(-2 * C * (g + A * g ** 3)))


def slope(name, g):
    if name == "none":
        return torch.ones_like(g)
    if name == "relu":
        return (g > 0).to(g.dtype)
    v, dv = (g, 1.0) if name == "silu" else (2 * C * (g + A * g ** 3), 2 * C * (1 + 3 * A * g * g))
    p = 1 / (1 + torch.exp(-v))
    return p + g * p * (1 - p) * dv


def product(a, b, ea=None):
    """(a b, bound): b exact, a off by at most ea."""
    c = a @ b
    e = (a.shape[1] + 16) * SUM * (a.abs() @ b.abs())
    return c, e if ea is None else e + ea @ b.abs()


def act_error(name, g):
    return torch.zeros_like(g) if name in ("none", "relu") else 2.0 ** -19 * (1 + g.abs())


def forward(x, gate, up, down, name):
    """{value: (exact, bound)} of g, u and y; g and u as fp32 sums, before they are rounded."""
    x, gate, up, down = (t.double() for t in (x, gate, up, down))
    (g, eg), (u, eu) = product(x, gate.t()), product(x, up.t())
    a = act(name, g)
    # |act'| is at most 1.13
    ea = 1.13 * eg + act_error(name, g) * a.abs()
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu
    eh = eh + (BF16 + SUM) * (h.abs() + eh) + TINY
    y, ey = product(h, down.t(), eh)
    return {"g": (g, eg), "u": (u, eu), "y": (y, ey + BF16 * (y.abs() + ey) + TINY)}


def kept_values(kept):
    """g and u as the backward pass takes them."""
    if len(kept) == 2:
        return [t.double() for t in kept]
    F = kept[0].shape[1]
    return [q.double() * s.double().t().repeat_interleave(128, 1)[:, :F] for q, s in zip(kept[:2], kept[2:])]


def backward(dy, x, gate, up, down, g, u, name):
    """{gradient: (exact, bound before its last rounding)}."""
    dy, x, gate, up, down = (t.double() for t in (dy, x, gate, up, down))
    dh, edh = product(dy, down)
    a, s = act(name, g), slope(name, g)
    ea, es = act_error(name, g) * a.abs(), act_error(name, g) * (1 + g.abs())

    def rounded(v, e):
        return v, e + (BF16 + 2 * SUM) * (v.abs() + e) + TINY

    dg, edg = rounded(dh * u * s, (edh * (s.abs() + es) + dh.abs() * es) * u.abs())
    du, edu = rounded(dh * a, edh * (a.abs() + ea) + dh.abs() * ea)
    h, eh = rounded(a * u, ea * u.abs())
    dx0, e0 = product(dg, gate, edg)
    dx1, e1 = product(du, up, edu)
    both = SUM * (2 * g.shape[1] + 16) * (dg.abs() @ gate.abs() + du.abs() @ up.abs())

    def weight(v, ev, w):
        return v.t() @ w, ev.t() @ w.abs() + (v.shape[0] + 16) * SUM * (v.abs().t() @ w.abs())

    ddown, edown = weight(h, eh, dy)
    return {"dx": (dx0 + dx1, e0 + e1 + both), "dgate": weight(dg, edg, x), "dup": weight(du, edu, x),
            "ddown": (ddown.t(), edown.t())}


def matrix(gen, rows, cols, size=1.0, pad=8, device="cuda"):
    """bf16 values; rows start `pad` elements or a multiple apart, with NaN in the gaps."""
    full = torch.full((rows, -(-cols // pad) * pad), float("nan"), device=device, dtype=torch.bfloat16)
    full[:, :cols] = torch.randn((rows, cols), generator=gen, device=device) * size
    return full[:, :cols]


class Band:
    """A rows x cols matrix inside a buffer of a byte that shows; `untouched` says whether what
    lies around it still holds it."""

    def __init__(self, rows, cols, dtype, step=8, offset=0, device="cuda", gap=0):
        ld = -(-cols // step) * step + gap
        size = torch.empty(0, dtype=dtype).element_size()
        self.flat = torch.full(((rows * ld + 64 + offset) * size,), 0x5A, device=device, dtype=torch.uint8)
        typed = self.flat.view(dtype)
        at = 32 + offset
        self.t = typed[at: at + rows * ld].view(rows, ld)[:, :cols]
        inside = torch.zeros(self.flat.numel() // size, device=device, dtype=torch.bool)
        inside[at: at + rows * ld].view(rows, ld)[:, :cols] = True
        self.outside = ~inside.repeat_interleave(size)

    def untouched(self):
        return bool((self.flat[self.outside] == 0x5A).all())


def close(name, got, want, bound):
    """Every element of got within its bound of want."""
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        worst = float((off / bound.clamp_min(1e-300)).nan_to_num(float("inf")).max())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside, the first at {i}: {float(got[i])} not "
                             f"{float(want[i])} within {float(bound[i])}; worst {worst:.3g} of its bound")
