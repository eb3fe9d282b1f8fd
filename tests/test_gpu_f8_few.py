"""e4m3 layers of few tokens: their fused routing (selection with and without groups, grouping, quantisation
of x) against the definitions and against the separate calls, at every token count where the path changes;
rows that are not finite; activations of more than 2^31 values."""
import sys

import numpy as np
import pytest

import f8_ref as R
import gpu_harness as H

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def dev():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import sparse_moe_layer_02_amd as moe
    moe.load()
    return torch, moe


def make_weights(torch, E, d, F, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = dict(w_router=torch.randn((E, d), generator=g, device="cuda") / d ** 0.5,
             bias=torch.rand(E, generator=g, device="cuda") * 0.1 - 0.05)
    for key, n, rows, cols in (("gate", E, F, d), ("up", E, F, d), ("down", E, d, F), ("s_gate", 1, F, d),
                               ("s_up", 1, F, d), ("s_down", 1, d, F)):
        c = torch.randint(0, 0x70, (n, rows, cols), generator=g, device="cuda", dtype=torch.uint8)
        c |= torch.randint(0, 2, c.shape, generator=g, device="cuda", dtype=torch.uint8) << 7
        s = torch.rand((n, -(-rows // 128), -(-cols // 128)), generator=g, device="cuda") + 0.5
        W[key] = (c, s * (0.5 / 64 / cols ** 0.5))
    return W


# (d, E, F, k, kind, (n_group, topk_group, group_top, normalise) or None, bias): E below, at and above 256 and at its
# limit, no power of two, k up to 32, d over 4096 (the router's second pass) and of many scale blocks
ROUTING = [(128, 8, 64, 2, "softmax", None, False), (192, 60, 64, 6, "sqrt_softplus", (12, 5, 2, 1), True),
           (256, 256, 64, 8, "sigmoid", (8, 4, 2, 1), True), (128, 256, 64, 32, "softmax", (16, 9, 1, 0), True),
           (64, 320, 64, 8, "sigmoid", None, True), (64, 320, 64, 9, "softmax", (10, 3, 2, 1), False),
           (64, 1024, 64, 32, "sqrt_softplus", (32, 8, 2, 0), True), (64, 1024, 64, 8, "softmax", (1, 1, 1, 1), True),
           (4160, 12, 64, 3, "sigmoid", (4, 2, 1, 1), True), (8256, 9, 64, 4, "softmax", (3, 2, 2, 0), False)]


@pytest.mark.parametrize("T", [1, 3, 8, 9, 12, 16, 17])
@pytest.mark.parametrize("d,E,F,k,kind,groups,biased", ROUTING)
def test_routing(dev, T, d, E, F, k, kind, groups, biased):
    torch, moe = dev
    say("T=%d d=%d E=%d k=%d %s %s" % (T, d, E, k, kind, groups))
    W = make_weights(torch, E, d, F, seed=d + E)
    if not biased:
        W["bias"] = None
    x = torch.randn((T, d), device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)).bfloat16()
    if T > 1:
        x[1] = 0.0  # equal logits: every tie goes to the lower index
    c = moe.make_config(T, d, E, k, F, score=kind, route_scale=1.5, act="bf16", w="f8b128")
    g = None if groups is None else moe.make_groups(*groups)
    n, Wm = T * k, moe.make_weights(W)
    out = dict(logits=torch.empty((T, E), device="cuda"), topk_idx=torch.empty((T, k), dtype=torch.int32, device="cuda"),
               topk_w=torch.empty((T, k), device="cuda"), offsets=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
               perm_rows=torch.empty(n, dtype=torch.int32, device="cuda"),
               inv_perm=torch.empty(n, dtype=torch.int32, device="cuda"))
    ws = moe.workspace(c)
    ws.fill_(0xA5)
    y, yb = torch.full((T, d), float("nan"), device="cuda"), torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    moe.moe_layer_forward_grouped(c, g, x, Wm, y, ws, debug=out)
    torch.cuda.synchronize()
    lg = out["logits"].cpu().numpy()
    assert H.ulp_diff_f32(lg, (x.double() @ W["w_router"].double().t()).float().cpu().numpy()).max() <= 1
    bias = None if W["bias"] is None else W["bias"].cpu().numpy()
    G = (1, 1, 1, 1) if groups is None else groups
    idx, w = R.select(lg, bias, k, kind, 1.5, G[0], G[1], G[2], bool(G[3]))
    assert np.array_equal(out["topk_idx"].cpu().numpy(), idx)
    assert H.ulp_diff_f32(out["topk_w"].cpu().numpy(), w.astype(np.float32)).max() <= 1
    # the same layer by separate calls: equal lists, equal bits
    off, perm, inv = (torch.empty_like(out[key]) for key in ("offsets", "perm_rows", "inv_perm"))
    moe.moe_permute(c, out["topk_idx"], off, perm, inv, ws)
    slot, sh, want = torch.empty((n, d), device="cuda"), torch.empty((T, d), device="cuda"), torch.empty((T, d), device="cuda")
    moe.moe_expert_ffn(c, x, Wm, off, perm, out["topk_w"], slot, sh, ws)
    moe.moe_combine(c, slot, sh, want)
    moe.moe_layer_forward_grouped(c, g, x, Wm, yb, ws)
    torch.cuda.synchronize()
    for key, v in (("offsets", off), ("perm_rows", perm), ("inv_perm", inv)):
        assert torch.equal(out[key], v), key
    assert torch.isfinite(y).all() and torch.equal(y, want) and torch.equal(yb, want.bfloat16())


@pytest.mark.parametrize("T,E,d,F", [(3, 4, 192, 128), (16, 2, 320, 192), (60, 8, 256, 192), (200, 2, 448, 192)])
def test_rows_that_are_not_finite(dev, T, E, d, F):
    """A row of x with one infinity or NaN is NaN in y; the others are what they are without it."""
    torch, moe = dev
    say("not finite", T, E, d, F)
    W = make_weights(torch, E, d, F, seed=T)
    x = torch.randn((T, d), device="cuda", generator=torch.Generator(device="cuda").manual_seed(T)).bfloat16()
    x[T // 2] = 0.0
    c = moe.make_config(T, d, E, 1, F, score="sigmoid", act="bf16", w="f8b128")
    Wm, ws = moe.make_weights(W), moe.workspace(c)
    want, y = torch.empty((T, d), device="cuda"), torch.empty((T, d), device="cuda")
    moe.moe_layer_forward_grouped(c, None, x, Wm, want, ws)
    others = torch.arange(T, device="cuda") != T // 2
    for value, at in ((float("inf"), d - 1), (float("-inf"), 0), (float("nan"), d // 2)):
        x[T // 2] = 0.0
        x[T // 2, at] = value
        moe.moe_layer_forward_grouped(c, None, x, Wm, y, ws)
        torch.cuda.synchronize()
        assert torch.isnan(y[T // 2]).all() and torch.equal(y[others], want[others]), (value, at)


def test_activations_beyond_2_31(dev):
    """n_tokens * d_model between 2^31 and 2^32: the last rows are what a small batch makes of them."""
    torch, moe = dev
    T, d, E, F, few = 1 << 20, 2112, 2, 64, 200
    W = make_weights(torch, E, d, F, seed=7)
    Wm = moe.make_weights(W)
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    y = torch.full((T, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    c = moe.make_config(T, d, E, 1, F, score="sigmoid", act="bf16", w="f8b128")
    say("T", T, "d", d)
    ws = torch.empty(moe.moe_workspace_bytes(c), dtype=torch.uint8, device="cuda")
    moe.moe_layer_forward_grouped(c, None, x, Wm, y, ws)
    torch.cuda.synchronize()
    small = moe.make_config(few, d, E, 1, F, score="sigmoid", act="bf16", w="f8b128")
    sw, want = moe.workspace(small), torch.empty((few, d), dtype=torch.bfloat16, device="cuda")
    for at in (0, (1 << 31) // d - few // 2, T - few):
        moe.moe_layer_forward_grouped(small, None, x[at:at + few].contiguous(), Wm, want, sw)
        torch.cuda.synchronize()
        assert torch.isfinite(want).all() and torch.equal(y[at:at + few], want), at
