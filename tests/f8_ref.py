"""The 8-bit operators and the grouped selection from their definitions, in
float64 numpy on the host, with the error bounds the tests use.

Bounds.  A product's sum runs over blocks of 128 columns.  In a block the
products of two e4m3 codes are exact and the matrix instruction adds them in
fp32: 128 additions, each off by at most one unit in the last place (2^-23
relative) of a partial sum no larger than the sum of magnitudes.  The row scale
is a power of two (exact); the weight scale is one fused multiply-add per block
(half a unit each), and up to 8 partial sums are added at the end.  So
|error| <= (128 + blocks + 8) 2^-23 * sum |terms|.  bf16 outputs add half a
step, 2^-8 of the value.

Results that are rounded to 16 or 8 bits next may come from the 8-bit matrix
instruction.  It cuts (towards zero) each product of 8 consecutive columns
below 2^-13 of the largest one's power of two before it adds them: the other
seven lose less than 2^-13 of the largest each.  ``cut`` adds that,
7 * 2^-13 * max |x| max |w| for each group of 8 columns.
"""
import numpy as np

B = 128


def e4m3_decode(codes):
    """float64 values of e4m3 codes (uint8)."""
    c = codes.astype(np.int64)
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(s == 1, -v, v)


def e4m3_round(v):
    """float64 values rounded to the e4m3 grid (nearest, ties to even); |v| <= 448."""
    _, e = np.frexp(v)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.rint(v / step) * step


def pad(x):
    k = x.shape[-1]
    n = -(-k // B) * B
    return np.pad(x, [(0, 0)] * (x.ndim - 1) + [(0, n - k)])


def block_scale(amax):
    """The smallest power of two s >= 2^-126 with amax <= 448 s (1 for 0)."""
    m, e = np.frexp(amax)
    return np.where(amax > 0, np.ldexp(1.0, np.maximum(e - 9 + (m > 0.875), -126)), 1.0)


def quantize(x):
    """(values / scale on the e4m3 grid [rows, cols], scales [rows, blocks]) of finite float64 rows."""
    rows, cols = x.shape
    p = pad(x).reshape(rows, -1, B)
    s = block_scale(np.abs(p).max(2))
    return e4m3_round(p / s[:, :, None]).reshape(rows, -1)[:, :cols], s


def dequant_rows(q, s):
    return q * np.repeat(s, B, axis=1)[:, :q.shape[1]]


def dequant_weight(q, s):
    """q [rows, cols] float64 values, s [ceil(rows/128), ceil(cols/128)]."""
    return q * np.repeat(np.repeat(s, B, axis=0), B, axis=1)[:q.shape[0], :q.shape[1]]


def matmul(xd, wd, cut=False):
    """(product, bound on the library's sum) of dequantised float64 operands."""
    k = xd.shape[1]
    blocks = -(-k // B)
    err = (128 + blocks + 8) * 2.0 ** -23 * (np.abs(xd) @ np.abs(wd).T)
    if cut:
        top = [np.abs(pad(a)).reshape(len(a), -1, 8).max(2) for a in (xd, wd)]
        err = err + 7 * 2.0 ** -13 * (top[0] @ top[1].T)
    return xd @ wd.T, err


def bf16_bound(y, err):
    return err + 2.0 ** -8 * (np.abs(y) + err)


def quantize_interval(h, eh):
    """Dequantised quantisation of rows h, and how far from it the result can be
    if every value is off by at most eh (a code moves if the interval crosses a
    rounding boundary, a scale if the block's maximum crosses one)."""
    rows, cols = h.shape
    lo, hi = pad(h - eh).reshape(rows, -1, B), pad(h + eh).reshape(rows, -1, B)
    p = pad(h).reshape(rows, -1, B)
    a = np.abs(p)
    up = np.maximum(np.abs(lo), np.abs(hi)).max(2)
    down = np.maximum(a - pad(eh).reshape(rows, -1, B), 0.0).max(2)
    s = block_scale(a.max(2))
    mid = e4m3_round(p / s[:, :, None]) * s[:, :, None]
    far = np.zeros_like(p)
    for sc in (block_scale(up), block_scale(down), s):
        for end in (lo, hi):
            v = np.clip(end / sc[:, :, None], -448.0, 448.0)
            far = np.maximum(far, np.abs(e4m3_round(v) * sc[:, :, None] - mid))
    return mid.reshape(rows, -1)[:, :cols], far.reshape(rows, -1)[:, :cols]


def silu(g):
    return g / (1.0 + np.exp(-g))


def expert(xd, wg, wu, wd, cut=False):
    """(SwiGLU expert output, bound) of dequantised rows through dequantised weights."""
    g, eg = matmul(xd, wg, cut)
    u, eu = matmul(xd, wu, cut)
    h = silu(g) * u
    # |silu'| <= 1.1; silu itself in fp32: a few units (16 * 2^-23 covers exp, reciprocal and products)
    eh = 1.1 * eg * (np.abs(u) + eu) + (np.abs(silu(g)) + 1.1 * eg) * eu + 16 * 2.0 ** -23 * np.abs(h)
    hd, far = quantize_interval(h, eh)
    y, ey = matmul(hd, wd, cut)
    return y, ey + far @ np.abs(wd).T * (1 + 2.0 ** -10)


def scores(logits, kind):
    l = logits.astype(np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "softmax":
            finite = np.where(np.isnan(l), -np.inf, l)
            e = np.exp(l - finite.max(1, keepdims=True))
            s = e / e.sum(1, keepdims=True)
        elif kind == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.sqrt(np.maximum(l, 0) + np.log1p(np.exp(-np.abs(l))))
    return s.astype(np.float32)


def _order(key):
    """Indices by (larger key, lower index), NaN after every number."""
    nan = np.isnan(key)
    k = np.where(nan, 0.0, key.astype(np.float64))
    return np.lexsort((np.arange(len(key)), -k, nan))


def select(logits, bias, k, kind, scale, n_group=1, topk_group=1, group_top=1, normalise=True):
    """(indices [T, k], weights float64 [T, k])."""
    T, E = logits.shape
    s = scores(logits, kind)
    key = s if bias is None else (s + bias.astype(np.float32)).astype(np.float32)
    idx = np.zeros((T, k), np.int32)
    w = np.zeros((T, k))
    S = E // n_group
    for t in range(T):
        allowed = np.arange(E)
        if topk_group < n_group:
            gs = np.zeros(n_group, np.float32)
            for g in range(n_group):
                kg = key[t, g * S:(g + 1) * S]
                best = kg[_order(kg)[:group_top]]
                gs[g] = best[0] if len(best) == 1 else np.float32(best[0]) + np.float32(best[1])
            keep = np.sort(_order(gs)[:topk_group])
            allowed = (keep[:, None] * S + np.arange(S)).reshape(-1)
        pick = allowed[_order(key[t, allowed])[:k]]
        sel = s[t, pick].astype(np.float64)
        idx[t] = pick
        if normalise:
            tot = sel.sum()
            w[t] = scale * (sel / tot) if tot > 0 else 0.0
        else:
            w[t] = scale * sel
    return idx, w
