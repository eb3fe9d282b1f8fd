"""Workloads of the layer's 8-bit and grouped-routing operators, with their plain forms.

Four operators, each with a plain form of elementary torch operations in 32
bits (64 for the router, as the layer defines it) and the library's own call:

* ``select``  top-k of given logits with expert groups (softmax or sigmoid
  scores, a balance bias, the best groups, renormalised weights), and
  ``route``, the same behind the router product;
* ``quant``   rows to e4m3 codes with one power-of-two scale (its e8m0
  exponent byte; a row's bytes are padded to a multiple of 4) per 128 columns;
* ``matmul``  x W^T of e4m3 rows and e4m3 weights in blocks of 128 x 128;
* ``layer``   the whole sparse MoE layer over such weights: grouped routing,
  routed and shared SwiGLU experts, weighted sum, y in bf16.

``run`` takes the library's kernels where ``own`` is true.
"""
import math

import torch

own = False

DEV = "cuda"
B = 128          # columns (and weight rows) that share a scale
F8_MAX = 448.0   # largest finite e4m3 value


def listed():
    return [
        # one generated token's routing: router product, 8 groups of 32 experts, the best 4 groups, top-8
        dict(name="route_1", op="route", T=1, d=4096, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, normalise=True, scale=2.5, act="bf16"),
        # selection of a 4096-token prompt over 192 experts: softmax scores, no groups
        dict(name="select_4096_softmax", op="select", T=4096, E=192, k=8, score="softmax", bias=False, n_group=1,
             topk_group=1, group_top=1, normalise=False, scale=1.0),
        # selection of a batch of long prompts, 256 experts in 8 groups with a balance bias
        dict(name="select_65536", op="select", T=65536, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, normalise=True, scale=2.5),
        # activations of a small ragged batch, rows inside a wider buffer
        dict(name="quant_33", op="quant", rows=33, cols=4096, ld=4224, x="bf16"),
        # activations of a long prompt
        dict(name="quant_4096", op="quant", rows=4096, cols=6144, ld=6144, x="bf16"),
        # one token through a projection (gate and up of a shared expert)
        dict(name="matmul_1", op="matmul", m=1, n=4096, k=6144, x="bf16", out="bf16"),
        # a verification batch through a down projection, odd row count
        dict(name="matmul_77", op="matmul", m=77, n=6144, k=2048, x="bf16", out="f32"),
        # a long prompt through a projection, rows already quantised
        dict(name="matmul_4096", op="matmul", m=4096, n=4096, k=6144, x="f8", out="bf16"),
        # single-token decode
        dict(name="layer_1", op="layer", T=1, d=4096, F=2048, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, normalise=True, scale=2.5, skew=0.0),
        # decode of eight sequences, 192 experts, flat softmax routing
        dict(name="layer_8", op="layer", T=8, d=4096, F=1536, E=192, k=8, score="softmax", bias=False, n_group=1,
             topk_group=1, group_top=1, normalise=True, scale=1.0, skew=0.0),
        # a prompt chunk: about 16 rows for each expert
        dict(name="layer_512", op="layer", T=512, d=6144, F=2048, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, normalise=True, scale=2.5, skew=0.0),
        # a long prompt with unevenly loaded experts
        dict(name="layer_4096", op="layer", T=4096, d=6144, F=2048, E=256, k=8, score="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, normalise=True, scale=2.5, skew=0.07),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_routing(rng, Es):
    E = rng.choice(Es)
    g = rng.choice([n for n in (1, 2, 4, 8) if E % n == 0 and E // n >= 4])
    tg = rng.randint(1, g)
    k = rng.randint(1, min(12, tg * (E // g)))
    return dict(E=E, k=k, score=rng.choice(["softmax", "sigmoid", "sqrt_softplus"]), bias=rng.random() < 0.5, n_group=g,
                topk_group=tg, group_top=rng.choice([1, 2]), normalise=rng.random() < 0.7,
                scale=rng.choice([1.0, 1.5, 2.5]))


def draw(rng):
    op = rng.choice(["route", "select", "quant", "matmul", "layer", "layer"])
    if op == "route":
        return dict(op=op, T=_log_int(rng, 1, 2048), d=64 * _log_int(rng, 4, 96), act=rng.choice(["bf16", "f32"]),
                    **_draw_routing(rng, [32, 60, 128, 192, 256]))
    if op == "select":
        return dict(op=op, T=_log_int(rng, 1, 65536), **_draw_routing(rng, [8, 40, 64, 100, 160, 192, 256]))
    if op == "quant":
        cols = 16 * _log_int(rng, 1, 384)
        return dict(op=op, rows=_log_int(rng, 1, 4096), cols=cols, ld=cols + rng.choice([0, 0, 16, 128]),
                    x=rng.choice(["bf16", "f32"]))
    if op == "matmul":
        return dict(op=op, m=_log_int(rng, 1, 4096), n=_log_int(rng, 16, 4096), k=16 * _log_int(rng, 4, 384),
                    x=rng.choice(["bf16", "f32", "f8"]), out=rng.choice(["bf16", "f32"]))
    r = _draw_routing(rng, [16, 32, 64, 128])
    return dict(op=op, T=_log_int(rng, 1, 4096), d=64 * _log_int(rng, 4, 96), F=64 * _log_int(rng, 2, 32),
                skew=rng.choice([0.0, 0.05]), **r)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _weights(gen, n, rows, cols):
    """e4m3 codes [n, rows, cols] of a normal matrix and fp32 scales per 128 x 128 block."""
    q = torch.empty((n, rows, cols), dtype=torch.float8_e4m3fn, device=DEV)
    flat, step = q.view(-1), 1 << 28
    for i in range(0, flat.numel(), step):
        m = min(step, flat.numel() - i)
        flat[i:i + m] = torch.randn(m, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(64).clamp_(-F8_MAX, F8_MAX).to(
            torch.float8_e4m3fn)
    s = torch.rand((n, -(-rows // B), -(-cols // B)), generator=gen, device=DEV) + 0.5
    return q, s * (0.02 / 64)


def _scale_ld(cols):
    """Bytes of a row's scales: one per 128 columns, padded to a multiple of 4."""
    return -(-cols // (4 * B)) * 4


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    op = c["op"]
    s = dict(c=c)
    if op == "quant":
        dt = torch.bfloat16 if c["x"] == "bf16" else torch.float32
        # a few large columns, as the activations of trained networks have
        col = torch.where(torch.rand(c["ld"], generator=gen, device=DEV) < 0.01, 30.0, 1.0)
        s["x"] = (torch.randn((c["rows"], c["ld"]), generator=gen, device=DEV) * col).to(dt)[:, :c["cols"]]
        s["q"] = torch.empty((c["rows"], c["cols"]), dtype=torch.float8_e4m3fn, device=DEV)
        s["s"] = torch.empty((c["rows"], _scale_ld(c["cols"])), dtype=torch.uint8, device=DEV)
        return s
    if op == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        w, ws = _weights(gen, 1, n, k)
        s["w"], s["ws"] = w[0], ws[0]
        x = torch.randn((m, k), generator=gen, device=DEV)
        if c["x"] == "f8":
            s["x"] = (x * 64).clamp_(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn)
            s["xs"] = torch.randint(119, 124, (m, _scale_ld(k)), generator=gen, device=DEV, dtype=torch.uint8)
        else:
            s["x"], s["xs"] = x.to(torch.bfloat16 if c["x"] == "bf16" else torch.float32), None
        s["out"] = torch.empty((m, n), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
        if own:
            import sparse_moe_layer_02_amd as moe
            s["wk"] = moe.block_matmul_workspace(s["x"], n)
        return s
    T, E, k = c["T"], c["E"], c["k"]
    s["bias"] = None
    if c["bias"]:
        s["bias"] = torch.rand(E, generator=gen, device=DEV) * 0.02 - 0.01
        if c.get("skew"):
            rank = torch.randperm(E, generator=gen, device=DEV) + 1
            s["bias"] -= c["skew"] * torch.log(rank.float())
    s["idx"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
    s["wt"] = torch.empty((T, k), device=DEV)
    if op == "select":
        s["logits"] = torch.randn((T, E), generator=gen, device=DEV)
        if own:
            import sparse_moe_layer_02_amd as moe
            s["cfg"] = moe.make_config(T, 64, E, k, 64, n_shared=0, score=c["score"], route_scale=c["scale"])
            s["grp"] = moe.make_groups(c["n_group"], c["topk_group"], c["group_top"], c["normalise"])
        return s
    d = c["d"]
    act = c.get("act", "bf16")
    s["x"] = torch.randn((T, d), generator=gen, device=DEV).to(torch.bfloat16 if act == "bf16" else torch.float32)
    s["w_router"] = torch.randn((E, d), generator=gen, device=DEV) / math.sqrt(d)
    if op == "route":
        s["logits"] = torch.empty((T, E), device=DEV)
        if own:
            import sparse_moe_layer_02_amd as moe
            s["cfg"] = moe.make_config(T, d, E, k, 64, n_shared=0, score=c["score"], route_scale=c["scale"], act=act,
                                       w=act)
            s["grp"] = moe.make_groups(c["n_group"], c["topk_group"], c["group_top"], c["normalise"])
        return s
    F = c["F"]
    s["gate"], s["up"], s["down"] = _weights(gen, E, F, d), _weights(gen, E, F, d), _weights(gen, E, d, F)
    s["s_gate"], s["s_up"], s["s_down"] = _weights(gen, 1, F, d), _weights(gen, 1, F, d), _weights(gen, 1, d, F)
    s["y"] = torch.empty((T, d), dtype=torch.bfloat16, device=DEV)
    if own:
        import sparse_moe_layer_02_amd as moe
        s["cfg"] = moe.make_config(T, d, E, k, F, score=c["score"], route_scale=c["scale"], act="bf16", w="f8b128")
        s["grp"] = moe.make_groups(c["n_group"], c["topk_group"], c["group_top"], c["normalise"])
        s["W"] = moe.make_weights({key: s[key] for key in ("w_router", "bias", "gate", "up", "down", "s_gate", "s_up",
                                                           "s_down")})
        s["wk"] = moe.workspace(s["cfg"])
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _select(c, logits, bias):
    """Indices [T, k] and weights [T, k] from fp32 logits, scores in 64 bits rounded once."""
    E, k, G = c["E"], c["k"], c["n_group"]
    l = logits.double()
    if c["score"] == "softmax":
        e = torch.exp(l - l.max(1, keepdim=True).values)
        s = e / e.sum(1, keepdim=True)
    elif c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        s = torch.sqrt(torch.clamp(l, min=0.0) + torch.log1p(torch.exp(-l.abs())))
    s = s.float()
    key = s if bias is None else s + bias
    if G > 1:
        best = key.view(-1, G, E // G).topk(min(c["group_top"], E // G), dim=2).values
        gs = best[..., 0] if best.shape[2] == 1 else best[..., 0] + best[..., 1]
        order = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, order, True)
        key = torch.where(keep.repeat_interleave(E // G, dim=1), key, -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = torch.gather(s, 1, idx).double()
    if c["normalise"]:
        tot = w.sum(1, keepdim=True)
        w = torch.where(tot > 0, w / tot, 0.0)
    return idx.int(), (w * c["scale"]).float()


def _logits(x, w_router):
    return (x.double() @ w_router.double().t()).float()


def _blocks(a, rows):
    """Scales [.., rb, cb] spread over 128 columns (and 128 rows)."""
    a = a.repeat_interleave(B, dim=-1)
    return a.repeat_interleave(B, dim=-2) if rows else a


def _quant(x):
    """e4m3 codes and the power-of-two scale of every 128 columns, in 32 bits."""
    x = x.float()
    rows, cols = x.shape
    kb = -(-cols // B)
    b = torch.nn.functional.pad(x, (0, kb * B - cols)).view(rows, kb, B)
    m, e = torch.frexp(b.abs().amax(2))
    # amax = m 2^e with m in [0.5, 1); 448 = 0.875 2^9
    p2 = torch.clamp(e - 9 + (m > 0.875), min=-126)
    s = torch.where(m > 0, ((p2 + 127) << 23).view(torch.float32), 1.0)  # 2^p2 by its exponent bits
    q = (b / s.unsqueeze(2)).to(torch.float8_e4m3fn).view(rows, kb * B)[:, :cols]
    return q, s


def _dequant(q, s, rows=False):
    n, k = q.shape[-2:]
    return q.float() * _blocks(s, rows)[..., :n, :k] if rows else q.float() * _blocks(s, False)[..., :k]


def _matmul(xq, xs, wq, ws):
    return _dequant(xq, xs) @ _dequant(wq, ws, True).t()


def _ffn(xd, gate, up, down):
    """SwiGLU of dequantised rows xd through one expert's dequantised weights."""
    g, u = xd @ gate.t(), xd @ up.t()
    return _dequant(*_quant(g / (1.0 + torch.exp(-g)) * u)) @ down.t()


def _layer(s):
    c = s["c"]
    idx, wt = _select(c, _logits(s["x"], s["w_router"]), s["bias"])
    xd = _dequant(*_quant(s["x"]))
    mats = [s["gate"], s["up"], s["down"]]
    y = _ffn(xd, *(_dequant(q[0], a[0], True) for q, a in (s["s_gate"], s["s_up"], s["s_down"])))
    e_of = idx.flatten().long()
    order = torch.sort(e_of, stable=True).indices
    count = torch.bincount(e_of, minlength=c["E"]).tolist()
    at = 0
    for e, n in enumerate(count):  # only the experts that have rows are read
        if n:
            f = order[at:at + n]
            t = torch.div(f, c["k"], rounding_mode="floor")
            r = _ffn(xd[t], *(_dequant(q[e], a[e], True) for q, a in mats))
            y.index_add_(0, t, r * wt.flatten()[f].unsqueeze(1))
            at += n
    return dict(y=y.to(torch.bfloat16), idx=idx, wt=wt)


def run(s):
    c = s["c"]
    op = c["op"]
    if own:
        import sparse_moe_layer_02_amd as moe
        if op == "quant":
            moe.moe_quantize_rows(s["x"], s["q"], s["s"])
            return dict(q=s["q"], s=s["s"][:, :-(-c["cols"] // B)].view(torch.float8_e8m0fnu))
        if op == "matmul":
            moe.moe_block_matmul(s["x"], s["xs"], s["w"], s["ws"], s["out"], s["wk"])
            return dict(out=s["out"])
        if op == "select":
            moe.moe_select_grouped(s["cfg"], s["grp"], s["logits"], s["bias"], s["idx"], s["wt"])
            return dict(idx=s["idx"], wt=s["wt"])
        if op == "route":
            moe.moe_route_grouped(s["cfg"], s["grp"], s["x"], s["w_router"], s["bias"], s["logits"], s["idx"], s["wt"],
                                  None)
            return dict(idx=s["idx"], wt=s["wt"], logits=s["logits"])
        moe.moe_layer_forward_grouped(s["cfg"], s["grp"], s["x"], s["W"], s["y"], s["wk"],
                                      debug=dict(topk_idx=s["idx"], topk_w=s["wt"]))
        return dict(y=s["y"], idx=s["idx"], wt=s["wt"])
    if op == "quant":
        q, a = _quant(s["x"])
        return dict(q=q.contiguous(), s=a.to(torch.float8_e8m0fnu))
    if op == "matmul":
        xq, xs = (s["x"], (s["xs"].int() << 23).view(torch.float32)) if s["xs"] is not None else _quant(s["x"])
        return dict(out=_matmul(xq, xs, s["w"], s["ws"]).to(s["out"].dtype))
    if op == "select":
        idx, wt = _select(c, s["logits"], s["bias"])
        return dict(idx=idx, wt=wt)
    if op == "route":
        logits = _logits(s["x"], s["w_router"])
        idx, wt = _select(c, logits, s["bias"])
        return dict(idx=idx, wt=wt, logits=logits)
    return _layer(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    op = c["op"]
    xb = {"bf16": 2, "f32": 4, "f8": 1}
    if op == "quant":
        return dict(bytes=c["rows"] * (c["cols"] * (xb[c["x"]] + 1) + 4 * -(-c["cols"] // B)),
                    flops=2 * c["rows"] * c["cols"])
    if op == "matmul":
        m, n, k = c["m"], c["n"], c["k"]
        return dict(bytes=m * k * xb[c["x"]] + n * k + m * n * xb[c["out"]], flops=2 * m * n * k)
    T, E, k = c["T"], c["E"], c["k"]
    sel = 8 * T * k + 4 * E
    if op == "select":
        return dict(bytes=4 * T * E + sel, flops=8 * T * E)
    if op == "route":
        return dict(bytes=T * c["d"] * xb[c["act"]] + 4 * E * c["d"] + 4 * T * E + sel, flops=2 * T * E * c["d"])
    d, F = c["d"], c["F"]
    touched = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token selects
    return dict(bytes=(touched + 1) * 3 * F * d + 4 * E * d + 4 * T * d + sel,
                flops=2 * T * E * d + 6 * T * (k + 1) * F * d)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _wide(a):
    return a.to(torch.float32).double()


def _two_to(p):
    """2^p for whole p in float64, exactly (the exponent field set)."""
    return ((p.long() + 1023) << 52).view(torch.float64)


def _quant64(x):
    """(values, scales) [rows, cols], [rows, blocks] of rows x: the smallest power of two s with amax <= 448 s
    (1 for a block of zeros), and x / s on the grid of 8-bit floats with 3 fraction bits, ties to even."""
    rows, cols = x.shape
    vals, scales = torch.empty_like(x), []
    for b in range(0, cols, B):
        blk = x[:, b:b + B]
        top = blk.abs().max(dim=1).values
        p = torch.ceil(torch.log2(torch.clamp(top, min=1e-45) / F8_MAX))
        p = torch.where(_two_to(p - 1) * F8_MAX >= top, p - 1, p)  # logarithms next to a whole number
        p = torch.where(_two_to(p) * F8_MAX < top, p + 1, p)
        s = torch.where(top > 0, _two_to(torch.clamp(p, min=-126.0)), 1.0)
        v = blk / s[:, None]
        e = torch.clamp(torch.frexp(v).exponent - 1, min=-6)  # v = f 2^e with f in [1, 2), or subnormal
        grid = _two_to(e - 3)
        vals[:, b:b + B] = torch.round(v / grid) * grid
        scales.append(s)
    return vals, torch.stack(scales, 1)


def _times(vals, s):
    out = vals.clone()
    for b in range(s.shape[1]):
        out[:, b * B:(b + 1) * B] *= s[:, b:b + 1]
    return out


def _weight64(q, s):
    out = _wide(q)
    for b in range(s.shape[0]):
        out[b * B:(b + 1) * B] = _times(out[b * B:(b + 1) * B], s[b:b + 1].double().expand(out[b * B:(b + 1) * B].shape[0], -1))
    return out


def _route64(c, logits, bias):
    E, k, G = c["E"], c["k"], c["n_group"]
    l = logits.double()
    if c["score"] == "softmax":
        s = torch.softmax(l, dim=1)
    elif c["score"] == "sigmoid":
        s = torch.sigmoid(l)
    else:
        s = torch.logaddexp(l, torch.zeros_like(l)).sqrt()
    s = s.float()  # scores are kept in fp32
    key = (s if bias is None else s + bias).double()
    if G > 1:
        g = key.reshape(-1, G, E // G).sort(dim=2, descending=True).values[:, :, :c["group_top"]].float()
        g = (g[:, :, 0] + g[:, :, 1] if g.shape[2] > 1 else g[:, :, 0]).double()
        # rank of a group: how many come before it (larger, or equal and lower)
        before = (g[:, None, :] > g[:, :, None]) | ((g[:, None, :] == g[:, :, None]) & torch.ones(
            (G, G), device=g.device).tril(-1).bool())
        out = before.sum(2) >= c["topk_group"]
        key = key.masked_fill(out.repeat_interleave(E // G, 1), -math.inf)
    idx, left = [], key.clone()
    pos = torch.arange(E, device=key.device)
    for _ in range(k):
        top = left.max(dim=1, keepdim=True).values
        e = torch.where(left == top, pos, E).min(dim=1, keepdim=True).values
        left.scatter_(1, e, -math.inf)
        idx.append(e)
    idx = torch.cat(idx, 1)
    w = torch.gather(s.double(), 1, idx)
    if c["normalise"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.int(), w * c["scale"]


def _expert64(x, gate, up, down):
    g, u = x @ gate.mT, x @ up.mT
    return _times(*_quant64(torch.nn.functional.silu(g) * u)) @ down.mT


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    op = c["op"]
    if op == "quant":
        q, a = _quant64(_wide(s["x"]))
        return dict(q=q, s=a)
    if op == "matmul":
        x = _times(_wide(s["x"]), _two_to(s["xs"].long() - 127)) if s["xs"] is not None else _times(*_quant64(_wide(s["x"])))
        return dict(out=x @ _weight64(s["w"], s["ws"]).mT)
    if op == "select":
        idx, wt = _route64(c, s["logits"], s["bias"])
        return dict(idx=idx, wt=wt)
    logits = _wide(s["x"]) @ s["w_router"].double().mT
    idx, wt = _route64(c, logits.float(), s["bias"])
    if op == "route":
        return dict(idx=idx, wt=wt, logits=logits)
    x = _times(*_quant64(_wide(s["x"])))
    y = _expert64(x, *(_weight64(s[m][0][0], s[m][1][0]) for m in ("s_gate", "s_up", "s_down")))
    for e in idx.unique().tolist():
        t, j = (idx == e).nonzero(as_tuple=True)
        y[t] += wt[t, j, None] * _expert64(x[t], *(_weight64(s[m][0][e], s[m][1][e]) for m in ("gate", "up", "down")))
    return dict(y=y, idx=idx, wt=wt)
