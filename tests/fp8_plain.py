"""The 8-bit operators evaluated in 64 bits with numpy, from the formats'
definitions: decoding tables, rounding to a format, group scales, the
block-scaled product and the mixture-of-experts layer.  Shares no code with the
library."""
import numpy as np

LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


def table(fmt):
    """The 256 values of a format (sign, exponent, mantissa)."""
    e_bits, m_bits, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    v = np.zeros(256)
    for c in range(256):
        sign = -1.0 if c & 0x80 else 1.0
        e, m = (c & 0x7f) >> m_bits, c & ((1 << m_bits) - 1)
        if fmt == "e5m2" and e == 31:
            v[c] = sign * (np.inf if m == 0 else np.nan)
        elif fmt == "e4m3" and (c & 0x7f) == 0x7f:
            v[c] = np.nan
        elif e == 0:
            v[c] = sign * m * 2.0 ** (1 - bias - m_bits)
        else:
            v[c] = sign * (1 + m / (1 << m_bits)) * 2.0 ** (e - bias)
    return v


TABLE = {f: table(f) for f in ("e4m3", "e5m2")}


def decode(codes, fmt):
    return TABLE[fmt][np.asarray(codes, dtype=np.uint8)]


def encode(x, fmt):
    """Codes of |x| <= largest (a hair above rounds down to it), ties to even;
    infinities to infinity (e5m2) or NaN (e4m3)."""
    x = np.asarray(x, dtype=np.float64)
    n = 0x7f if fmt == "e4m3" else 0x7c          # codes 0..n-1: the finite magnitudes, ascending
    mags = TABLE[fmt][:n]
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(mags, a), 1, n - 1)
    lo = hi - 1
    dl, dh = a - mags[lo], mags[hi] - a
    pick_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    c = np.where(pick_hi, hi, lo).astype(np.uint8)
    c = np.where(np.isinf(x), 0x7c if fmt == "e5m2" else 0x7f, c)
    c = np.where(np.isnan(x), 0x7f, c)
    return (c | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def spread(s, rows, cols, gr, gc):
    """The scale of each element; s as the library lays it out for the group."""
    r, c = np.arange(rows), np.arange(cols)
    if (gr, gc) == (1, 128):
        return s[(c // 128)[None, :], r[:, None]]
    if (gr, gc) == (128, 1):
        return s[(r // 128)[:, None], c[None, :]]
    return s[(r // 128)[:, None], (c // 128)[None, :]]


def quantize(x, group, fmt):
    """(codes, scales): each step one fp32 operation, rounded to nearest, as documented."""
    gr, gc = group
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    rb, cb = -(-rows // gr), -(-cols // gc)
    a = np.zeros((rb * gr, cb * gc), dtype=np.float32)
    a[:rows, :cols] = np.where(np.isfinite(x), np.abs(x), np.float32(0))
    amax = a.reshape(rb, gr, cb, gc).max((1, 3))
    s = np.maximum(amax / np.float32(LARGEST[fmt]), np.float32(2.0 ** -126)).astype(np.float32)
    inv = (np.float32(1) / s).astype(np.float32)
    if gr == 1:
        s, inv = np.ascontiguousarray(s.T), np.ascontiguousarray(inv.T)
    with np.errstate(invalid="ignore", over="ignore"):
        y = (x * spread(inv, rows, cols, gr, gc)).astype(np.float32)
    return encode(y, fmt), s


def values(codes, s, fmt, group, k_first):
    """The values of an operand as stored; `k_first`: its rows run across the sum."""
    rows, cols = codes.shape
    shape = (128, 128) if group == 128 else ((128, 1) if k_first else (1, 128))
    return decode(codes, fmt) * spread(np.asarray(s, np.float64), rows, cols, *shape)


def product(a, b, alpha=1.0, beta=0.0, c=None):
    """alpha a b + beta c in 64 bits, and the sum of the terms' magnitudes (for error bounds)."""
    with np.errstate(invalid="ignore", over="ignore"):
        out, size = alpha * (a @ b), abs(alpha) * (np.abs(a) @ np.abs(b))
        if beta != 0:
            out, size = out + beta * c, size + np.abs(beta * c)
    return out, size


def moe(x, router, gate, up, down, topk, renormalize, logits=None):
    """(y, logits, indices, weights) in 64 bits; gate, up, down: E matrices of values."""
    logits = x @ router.T if logits is None else logits
    order = np.argsort(-logits, axis=1, kind="stable")[:, :topk]
    p = np.exp(logits - logits.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    w = np.take_along_axis(p, order, 1)
    if renormalize:
        w = w / w.sum(1, keepdims=True)
    y = np.zeros(x.shape)
    size = np.zeros(x.shape)                   # what errors of the products are measured against
    for t in range(x.shape[0]):
        for j, e in enumerate(order[t]):
            g, u = gate[e] @ x[t], up[e] @ x[t]
            with np.errstate(over="ignore"):
                h = g / (1 + np.exp(-g)) * u
            y[t] += w[t, j] * (down[e] @ h)
            gs, us = np.abs(gate[e]) @ np.abs(x[t]), np.abs(up[e]) @ np.abs(x[t])
            # |dh| <= |silu'| |dg| |u| + |silu| |du|, |silu'| < 1.1
            size[t] += w[t, j] * (np.abs(down[e]) @ (1.1 * gs * np.abs(u) + np.abs(h / np.where(u == 0, 1, u)) * us + np.abs(h)))
    return y, logits, order, w, size
