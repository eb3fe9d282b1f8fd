"""The balance loss and the routing's gradient from their definitions, in float64 numpy, with the bounds of the
library's fp32 arithmetic that the tests use.

Bounds.  U = 2^-24.  A score takes an exponential of an fp32 argument (softmax: a difference of logits, rounded: off by
|l - max| U, which is the exponential's relative error too), and a few operations of at most two units each: relative
error below (R + 16) 2 U, R the largest |l - max| (0 for the other scores, whose argument is the logit itself).  The sum
over E experts adds at most 21 additions on a path through the tree, the reciprocal and its product three more units: p
is off by ``eps_p`` = (2 R + 64) U relative.  prob adds non-negative fp32 numbers: at most ceil(T / 4096) + 16 on a path
(a workgroup's wavefronts go round its range of tokens, then their sums are added), fp64 beyond.

The gradient's terms are differences, so its bound goes by magnitudes: for ds the sum of the magnitudes of its parts,
(|f - 1| + sum |f - 1| p) and (|dw| + sum |dw| s / S), each made of numbers with the errors above and of up to 21
additions: 4 eps_p + 64 U of it in all.
"""
import numpy as np

U = 2.0 ** -24


def seq_index(T, off, mask):
    """Sequence of each token, -1 for none."""
    if off is None:
        q = np.zeros(T, np.int64)
    else:
        off = np.asarray(off, np.int64)
        q = np.searchsorted(off, np.arange(T), side="right") - 1
        q[q >= len(off) - 1] = -1
    return q if mask is None else np.where(np.asarray(mask) != 0, q, -1)


def score(l, kind):
    """(s, s'(l)): softmax's second is None (it is no function of one logit)."""
    l = l.astype(np.float64)
    with np.errstate(over="ignore"):
        if kind == "softmax":
            e = np.exp(l - l.max(1, keepdims=True))
            return e / e.sum(1, keepdims=True), None
        sg = 1.0 / (1.0 + np.exp(-l))
        if kind == "sigmoid":
            return sg, sg / (1.0 + np.exp(l))
        s = np.sqrt(np.maximum(l, 0) + np.log1p(np.exp(-np.abs(l))))
        return s, np.where(s > 0, 0.5 * sg / np.where(s > 0, s, 1.0), 0.0)  # (below e^-745 both vanish)


def eps_p(l, kind):
    R = (l.max(1) - l.min(1)).max() if kind == "softmax" and l.size else 0.0
    return (2 * float(R) + 64) * U


def balance(l, idx, kind, off=None, mask=None, n_seq=1):
    """counts, tokens, prob, loss (float64) and the relative bound of the last two."""
    T, E = l.shape
    q = seq_index(T, off, mask)
    counts, tokens, prob = np.zeros((n_seq, E), np.int64), np.zeros(n_seq, np.int64), np.zeros((n_seq, E))
    for t in np.nonzero(q >= 0)[0]:
        tokens[q[t]] += 1
        for x in idx[t]:
            if 0 <= x < E:
                counts[q[t], x] += 1
    live = q >= 0
    s, _ = score(l[live], kind)
    p = s / s.sum(1, keepdims=True)
    np.add.at(prob, q[live], p)
    n = np.maximum(tokens, 1)[:, None]
    prob /= n
    f = E * counts / (idx.shape[1] * n)
    rel = eps_p(l[live], kind) + (-(-T // 4096) + 16 + 2) * U
    return counts, tokens, prob, (f * prob).sum(1), rel


def backward(l, idx, kind, scale=1.0, normalise=True, d_w=None, counts=None, tokens=None, d_loss=None, off=None,
             mask=None, eps=None):
    """(d_logits, bound), float64; eps: a relative error of p that stands for eps_p."""
    T, E = l.shape
    k = idx.shape[1]
    q = seq_index(T, off, mask)
    out, err = np.zeros((T, E)), np.zeros((T, E))
    live = np.nonzero(q >= 0)[0]
    if not len(live):
        return out, err
    s, slope = score(l[live], kind)
    ds, mag = np.zeros_like(s), np.zeros_like(s)
    if d_loss is not None:
        n = np.maximum(tokens, 1).astype(np.float64)[:, None]
        f1 = (E * counts / (k * n) - 1.0)[q[live]]
        rate = (d_loss.astype(np.float64) / n[:, 0])[q[live]][:, None]
        S = s.sum(1, keepdims=True)
        p = s / S
        ds += rate * (f1 - (f1 * p).sum(1, keepdims=True)) / S
        mag += np.abs(rate) * (np.abs(f1) + (np.abs(f1) * p).sum(1, keepdims=True)) / S
    if d_w is not None:
        for i, t in enumerate(live):
            ok = (idx[t] >= 0) & (idx[t] < E)
            x, dw = idx[t][ok], scale * d_w[t][ok].astype(np.float64)
            m = np.abs(dw)
            if normalise:
                sel = s[i, x]
                S = sel.sum()
                if S > 0:
                    m = (m + (m * sel).sum() / S) / S
                    dw = (dw - (dw * sel).sum() / S) / S
                else:
                    dw = m = np.zeros_like(dw)
            np.add.at(ds[i], x, dw)
            np.add.at(mag[i], x, m)
    if kind == "softmax":
        out[live] = s * (ds - (ds * s).sum(1, keepdims=True))
        err[live] = s * (mag + (mag * s).sum(1, keepdims=True))
    else:
        out[live] = ds * slope
        err[live] = mag * slope
    return out, err * (4 * (eps_p(l[live], kind) if eps is None else eps) + 64 * U)


def objective(l, idx, kind, scale, normalise, d_w, counts, tokens, d_loss, off, mask):
    """What ``backward`` is the gradient of, with the counts held."""
    T, E = l.shape
    q = seq_index(T, off, mask)
    s, _ = score(l, kind)
    p = s / s.sum(1, keepdims=True)
    total = 0.0
    for t in np.nonzero(q >= 0)[0]:
        n = max(int(tokens[q[t]]), 1)
        total += float(d_loss[q[t]]) * float((E * counts[q[t]] / (idx.shape[1] * n) * p[t]).sum()) / n
        ok = (idx[t] >= 0) & (idx[t] < E)
        sel = s[t, idx[t][ok]]
        w = scale * sel / sel.sum() if normalise else scale * sel
        total += float((d_w[t][ok] * w).sum())
    return total
