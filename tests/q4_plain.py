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


def held(x):
    """How far what x is held as may be from it.  A block of 128 is scaled to 2^14 .. 2^15 at its
    largest, where fp16's smallest half step, 2^-25 (16 times that where codes are 16
    times larger), is 2^-35 of the largest; bf16 has no more bits than fp16.  Of fp32 a
    first part leaves half a step, 2^-11 of its binade, and the second, 2^11 times larger,
    half a step of that: 2^-23, and 2^-46 of the largest."""
    M, K = x.shape
    most = torch.nn.functional.pad(x.double().abs(), (0, -K % 128)).view(M, -1, 128).amax(2).repeat_interleave(128, 1)[:, :K]
    if x.dtype == torch.bfloat16:
        return 2.0 ** -35 * most
    return 2.0 ** -23 * x.double().abs() + 2.0 ** -46 * most


def product(x, w, group):
    """(x w^T, bound): the terms of a group (of two parts at most, together 1 + 2^-10 of x's
    size) are added in fp32, its sum is scaled twice and added in fp32 (a rounding or
    truncation each, 2^-23), then up to 64 partial sums; and x is held to held(x)."""
    c = x.double() @ w.t()
    steps = 2 * group + 4 * (w.shape[1] // group) + 160
    return c, 1.01 * steps * fp.SUM * (x.double().abs() @ w.abs().t()) + held(x) @ w.abs().t()


def gated(x, w, w2, group, act):
    (g, eg), (u, eu) = product(x, w, group), product(x, w2, group)
    a = fp.act(act, g)
    ea = 1.13 * eg + fp.act_error(act, g) * a.abs()
    c = a * u
    return c, ea * (u.abs() + eu) + a.abs() * eu + 2 * fp.SUM * c.abs()
