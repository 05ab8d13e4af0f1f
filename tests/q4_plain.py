"""4-bit matrices in plain operations: the quantiser's fp32 steps one by one, the values in 64
bits, and products with a bound on the error that the kernel's arithmetic may make."""
import numpy as np
import torch

from tests import ffn_plain as fp


def unpack(q, cols):
    return torch.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)[:, :cols]


def spread(t, group, cols):
    """Of each element: its group's scale or zero code."""
    return t.t().repeat_interleave(group, 1)[:, :cols]


def values(q, s, z, group, cols):
    zero = 8.0 if z is None else spread(z.double(), group, cols)
    return (unpack(q, cols).double() - zero) * spread(s.double(), group, cols)


def quantize(w, group, symmetric):
    """(codes unpacked, scales, zero codes, values), numpy fp32 in the operator's own steps."""
    f = np.float32
    w = np.asarray(w, dtype=f)
    rows, cols = w.shape
    n = -(-cols // group)
    full = np.zeros((rows, n * group), f)
    full[:, :cols] = w
    g = full.reshape(rows, n, group)
    fin = np.where(np.isfinite(g), g, f(0))
    with np.errstate(all="ignore"):
        if symmetric:
            scale = np.maximum(np.abs(fin).max(2) / f(7), f(2.0 ** -126))
            zero = np.full_like(scale, 8)
        else:
            high, low = np.maximum(fin.max(2), f(0)), np.minimum(fin.min(2), f(0))
            scale = np.maximum(high / f(15) - low / f(15), f(2.0 ** -126))
            zero = np.minimum(np.rint(-low * (f(1) / scale)), f(15))
        inverse = f(1) / scale
        code = np.clip(np.rint(g * inverse[:, :, None]) + zero[:, :, None], f(0), f(15))
        code = np.where(np.isnan(g), zero[:, :, None], code)
        value = (code - zero[:, :, None]) * scale[:, :, None]
    assert scale.dtype == f and value.dtype == f
    flat = lambda a: a.reshape(rows, n * group)[:, :cols]  # noqa: E731
    return flat(code).astype(np.uint8), scale.T, zero.T.astype(np.uint8), flat(value)


def product(x, w, group):
    """(x w^T, bound): the terms of a group are added in fp32, its sum scaled and added in fp32
    (a rounding or truncation each, 2^-23), then up to 64 partial sums; parts of an
    fp32 x add up to no more than (1 + 2^-7) of its size."""
    x = x.double()
    c = x @ w.t()
    steps = 3 * group + w.shape[1] // group + 160
    return c, steps * fp.SUM * 1.01 * (x.abs() @ w.abs().t())


def gated(x, w, w2, group, act):
    (g, eg), (u, eu) = product(x, w, group), product(x, w2, group)
    a = fp.act(act, g)
    ea = 1.13 * eg + fp.act_error(act, g) * a.abs()
    c = a * u
    return c, ea * (u.abs() + eu) + a.abs() * eu + 2 * fp.SUM * c.abs()
