"""Grouped selection in the decode path of more than 256 experts (fp32, bf16 and int8 weights): routing against
the definition, permutation exact, y against the separate calls."""
import sys

import numpy as np
import pytest

import f8_ref as R
import gpu_harness as H
from synth import configs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wt,act", [("bf16", "bf16"), ("q8b32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("T,E,k,kind,groups", [(1, 320, 8, "softmax", None), (2, 320, 6, "sigmoid", (10, 3, 2, 1)),
                                               (5, 1024, 4, "sqrt_softplus", (32, 5, 1, 0)), (8, 600, 3, "softmax", (12, 4, 2, 1))])
def test_decode(T, E, k, kind, groups, wt, act):
    import torch
    import sparse_moe_layer_02_amd as moe
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    moe.load()
    d, F, n = 128, 64, T * k
    print("decode", T, E, k, kind, groups, wt, flush=True)
    sys.stdout.flush()
    cfg = configs.custom(T=T, d=d, E=E, k=k, F=F, Fs=F, n_shared=1, act=act, w=wt, x_sigma=1.0, w_sigma=0.05,
                         wr_sigma=1 / 16.0, score="sigmoid", bias="uniform")
    L = configs.make_layer(cfg)
    W, x = H.upload_layer(L), H.to_dev(L["x"])
    Wm = moe.make_weights(W)
    c = moe.make_config(T, d, E, k, F, score=kind, route_scale=1.5, act=act, w=wt)
    g = None if groups is None else moe.make_groups(*groups)
    out = dict(logits=torch.empty((T, E), device="cuda"), topk_idx=torch.empty((T, k), dtype=torch.int32, device="cuda"),
               topk_w=torch.empty((T, k), device="cuda"), offsets=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
               perm_rows=torch.empty(n, dtype=torch.int32, device="cuda"),
               inv_perm=torch.empty(n, dtype=torch.int32, device="cuda"))
    y, want = torch.full((T, d), float("nan"), device="cuda"), torch.empty((T, d), device="cuda")
    ws = moe.workspace(c)
    ws.fill_(0xA5)
    moe.moe_layer_forward_grouped(c, g, x, Wm, y, ws, debug=out)
    torch.cuda.synchronize()
    G = (1, 1, 1, 1) if groups is None else groups
    idx, w = R.select(out["logits"].cpu().numpy(), L["bias"], k, kind, 1.5, G[0], G[1], G[2], bool(G[3]))
    assert np.array_equal(out["topk_idx"].cpu().numpy(), idx)
    assert H.ulp_diff_f32(out["topk_w"].cpu().numpy(), w.astype(np.float32)).max() <= 1
    off, perm, inv = (torch.empty_like(out[key]) for key in ("offsets", "perm_rows", "inv_perm"))
    moe.moe_permute(c, out["topk_idx"], off, perm, inv, ws)
    slot, sh = torch.empty((n, d), device="cuda"), torch.empty((T, d), device="cuda")
    moe.moe_expert_ffn(c, x, Wm, off, perm, out["topk_w"], slot, sh, ws)
    moe.moe_combine(c, slot, sh, want)
    torch.cuda.synchronize()
    for key, v in (("offsets", off), ("perm_rows", perm), ("inv_perm", inv)):
        assert torch.equal(out[key], v), key
    H.check_y(y.cpu().numpy(), want.double().cpu().numpy(), cfg, "decode")
