"""The int8 operators from their definitions, in float64 numpy on the host, with
the error bounds the tests use.

Quantisation has none: scales and codes are exact.  A product's sum is an exact
integer; rounded to fp32 and multiplied by the row's scale and the channel's it
takes three roundings of half a unit, 2^-24 each, in that order, so the fp32
result can be computed bit for bit (``product_f32``).  In a layer each of those,
silu and the weighted sum adds its own roundings (``expert``).
"""
import numpy as np

MIN_SCALE = 2.0 ** -120
U = 2.0 ** -24  # half a unit of fp32, relative


def quantize(x):
    """(codes int64 [rows, cols], scales float32 [rows]) of finite float64 rows (values that fp32 holds)."""
    top = np.abs(x).max(1)
    s = np.maximum((top / 127.0).astype(np.float32), np.float32(MIN_SCALE))
    s = np.where(top == 0, np.float32(1.0), s)
    return np.rint(x / s.astype(np.float64)[:, None]).astype(np.int64), s


def dequant(q, s):
    return q.astype(np.float64) * s.astype(np.float64)[:, None]


def int_sums(q, w):
    """Exact sums of products of codes (float64 holds them: below 2^31)."""
    return q.astype(np.float64) @ w.astype(np.float64).T


def product_f32(q, s, w, ws):
    """The library's fp32 product, bit for bit."""
    with np.errstate(over="ignore", invalid="ignore"):
        return (int_sums(q, w).astype(np.float32) * s.astype(np.float32)[:, None]) * ws.astype(np.float32)[None]


def to_bf16(v):
    """fp32 values rounded to bf16 (nearest, ties to even), as fp32."""
    import torch
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).bfloat16().float().numpy()


def silu(g):
    return g / (1.0 + np.exp(-g))


def quantize_interval(h, eh):
    """Dequantised quantisation of rows h, and how far from it the result can be if every value is off by at most
    eh: the row's scale lies between those of the smallest and the largest maximum, a code between those of the
    interval's ends over either scale, and the value between the products of these ends."""
    q, s = quantize(h)
    mid = dequant(q, s)
    up = (np.abs(h) + eh).max(1)
    down = np.maximum(np.abs(h) - eh, 0.0).max(1)
    # (an fp32 maximum's quotient by 127 is rounded once more)
    hi = np.maximum(up / 127.0 * (1 + U), MIN_SCALE)[:, None]
    lo = np.maximum(down / 127.0 * (1 - U), MIN_SCALE)[:, None]
    ends = [np.rint((h + sg * eh) / sc) for sg in (-1.0, 1.0) for sc in (lo, hi)]
    nmin, nmax = np.minimum.reduce(ends), np.maximum.reduce(ends)
    far = np.zeros_like(h)
    for n in (nmin, nmax):
        for sc in (lo, hi):
            far = np.maximum(far, np.abs(n * sc - mid))
    return mid, far


def expert(x, gate, up, down):
    """(SwiGLU expert output, bound): x dequantised rows, matrices dequantised (float64)."""
    g, u = x @ gate.T, x @ up.T
    eg, eu = 3.01 * U * np.abs(g), 3.01 * U * np.abs(u)
    h = silu(g) * u
    # |silu'| <= 1.1; silu in fp32 with the hardware's exponential and reciprocal, whose argument's product with
    # log2 e is rounded too: (16 + |g|) 2^-23 covers them and the two products
    eh = 1.1 * eg * (np.abs(u) + eu) + (np.abs(silu(g)) + 1.1 * eg) * eu + (16 + np.abs(g)) * 2.0 ** -23 * np.abs(h)
    hd, far = quantize_interval(h, eh)
    y = hd @ down.T
    ey = far @ np.abs(down).T
    return y, ey + 4.01 * U * (np.abs(y) + ey)  # (the fourth: the routing weight's product)


def bf16_bound(y, err):
    return err + 2.0 ** -8 * (np.abs(y) + err)
