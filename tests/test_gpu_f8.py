"""The 8-bit operators on the GPU against their float64 definitions (f8_ref,
which derives the bounds): codes and scales exact, products within the fp32
summation bound, the layer within that bound carried through the quantised
SwiGLU intermediate, and bit for bit on layers whose arithmetic is exact."""
import sys

import numpy as np
import pytest

import f8_ref as R
import gpu_harness as H
from synth import configs

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


def codes_of(rng, shape, sigma=64.0):
    """Random e4m3 codes of a normal distribution (float64 values, uint8 codes)."""
    import torch
    v = torch.from_numpy(np.clip(rng.standard_normal(shape) * sigma, -448, 448)).to(torch.float32).to(torch.float8_e4m3fn)
    c = v.view(torch.uint8).numpy()
    return R.e4m3_decode(c), c


def weights_of(rng, rows, cols, n=None):
    shape = (rows, cols) if n is None else (n, rows, cols)
    v, c = codes_of(rng, shape)
    s = (rng.random(shape[:-2] + (-(-rows // 128), -(-cols // 128))) + 0.5).astype(np.float32) * np.float32(0.03 / 64)
    return v, c, s


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

def quant_rows(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * 4)
    x[:, ::17] *= 30
    for i, v in enumerate([0.0, 448.0, 449.0, 3e38, 1e-38, 2.0 ** -130, -0.0, 224.0 * 2 ** -20]):
        if i < rows:
            x[i] = 0.0
            x[i, i % cols] = v
    if rows > 9:
        x[9] = rng.integers(-32, 33, cols)  # many ties
    return x


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,ld", [(1, 16, 16), (1, 4096, 4096), (3, 112, 128), (33, 128, 128), (17, 144, 160),
                                          (10, 1040, 1040), (129, 512, 640), (1000, 6144, 6144)])
def test_quantize(dev, rows, cols, ld, dt):
    torch, moe = dev
    say("quantize", rows, cols, ld, dt)
    rng = np.random.default_rng(rows + cols)
    buf = torch.full((rows, ld), 7.0, dtype=torch.float32)
    buf[:, :cols] = torch.from_numpy(quant_rows(rng, rows, cols).astype(np.float32))
    buf = buf.bfloat16() if dt == "bf16" else buf
    x = buf.cuda()[:, :cols]
    q = torch.full((rows, cols), 0xAA, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, moe.scale_ld(cols)), 0xAA, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_rows(x, q, s)
    torch.cuda.synchronize()
    want_q, want_s = R.quantize(buf[:, :cols].double().numpy())
    nb = want_s.shape[1]
    sb = s.cpu().numpy()
    assert np.array_equal(np.ldexp(1.0, sb[:, :nb].astype(int) - 127), want_s)
    assert (sb[:, nb:] == 127).all()
    assert np.array_equal(R.e4m3_decode(q.cpu().numpy()), want_q)


def test_quantize_poisoned_blocks(dev):
    torch, moe = dev
    x = torch.ones((6, 272), device="cuda")
    x[0, 5], x[1, 130], x[2, 271], x[3, 0] = float("nan"), float("inf"), float("-inf"), float("inf")
    x[3, 1] = float("nan")
    for t in (x, x.bfloat16()):
        q, s = torch.empty((6, 272), dtype=torch.uint8, device="cuda"), torch.empty((6, 4), dtype=torch.uint8, device="cuda")
        moe.moe_quantize_rows(t, q, s)
        torch.cuda.synchronize()
        assert s[:, :3].cpu().tolist() == [[255, 119, 119], [119, 255, 119], [119, 119, 255], [255, 119, 119],
                                           [119, 119, 119], [119, 119, 119]]
        assert (q[0, :128] == 0x7F).all() and (q[1, 128:256] == 0x7F).all() and (q[2, 256:] == 0x7F).all()
        assert (q[4:] == 0x78).all() and (q[0, 128:] == 0x78).all()  # 1 / 2^-8 = 256


def test_quantize_leaves_other_rows(dev):
    torch, moe = dev
    x = torch.randn((5, 256), device="cuda").bfloat16()
    q, s = torch.full((7, 256), 9, dtype=torch.uint8, device="cuda"), torch.full((7, 4), 9, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_rows(x, q[1:6], s[1:6])
    torch.cuda.synchronize()
    assert (q[[0, 6]] == 9).all() and (s[[0, 6]] == 9).all()


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

SIZES = [(1, 16, 16), (1, 4096, 6144), (1, 1, 128), (2, 130, 144), (5, 67, 1040), (15, 256, 128), (16, 96, 272),
         (17, 200, 512), (32, 129, 2048), (33, 48, 640), (64, 1000, 1152), (65, 256, 256), (77, 640, 2048),
         (128, 384, 896), (200, 130, 304), (257, 512, 512), (300, 1037, 1296), (513, 256, 2048), (1030, 770, 400)]


@pytest.mark.parametrize("xdt", ["f8", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_matmul(dev, m, n, k, xdt):
    torch, moe = dev
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    wv, wc, wsc = weights_of(rng, n, k)
    wd = R.dequant_weight(wv, wsc.astype(np.float64))
    w, wscale = torch.from_numpy(wc).cuda(), torch.from_numpy(wsc).cuda()
    if xdt == "f8":
        xv, xc = codes_of(rng, (m, k))
        nb = -(-k // 128)
        e = np.full((m, moe.scale_ld(k)), 255, np.uint8)  # bytes past the last block are not read as scales
        e[:, :nb] = rng.integers(110, 140, (m, nb))
        xd = R.dequant_rows(xv, np.ldexp(1.0, e[:, :nb].astype(int) - 127))
        x, xs = torch.from_numpy(xc).cuda(), torch.from_numpy(e).cuda()
    else:
        x = torch.from_numpy((rng.standard_normal((m, k)) * 3).astype(np.float32))
        x = x.bfloat16() if xdt == "bf16" else x
        xd = R.dequant_rows(*R.quantize(x.double().numpy()))
        x, xs = x.cuda(), None
    for odt in (torch.float32, torch.bfloat16):
        ref, err = R.matmul(xd, wd, cut=odt == torch.bfloat16)
        say("matmul m=%d n=%d k=%d %s -> %s" % (m, n, k, xdt, odt))
        out = torch.full((m + 1, n), 123.0, dtype=odt, device="cuda")
        wk = moe.block_matmul_workspace(x, n)
        if wk is not None:
            wk.fill_(0xFF)  # the workspace needs no initialisation
        moe.moe_block_matmul(x, xs, w, wscale, out[:m], wk)
        torch.cuda.synchronize()
        got = out[:m].double().cpu().numpy()
        lim = err if odt == torch.float32 else R.bf16_bound(ref, err)
        worst = np.max(np.abs(got - ref) - lim)
        assert np.isfinite(got).all() and worst <= 0, (worst, np.argwhere(np.abs(got - ref) > lim)[:4])
        assert (out[m] == 123.0).all()  # the row behind the last is left alone


# sizes whose tiles are the larger ones (128 x 128; 256 x 256 and, for fp32 results, 128 x 256), with ends in
# rows, columns and K; K below one block; K of more blocks than a wavefront has lanes
LARGE = [(1600, 2000, 272), (3500, 3600, 400), (70, 200, 16), (300, 70, 112), (1600, 2000, 48), (3500, 3600, 80),
         (90, 150, 8464), (600, 1000, 8464), (1600, 2000, 8320), (250, 1000, 2064), (8000, 20, 1040), (70, 132, 144), (70, 133, 144), (70, 134, 144), (70, 136, 144)]


@pytest.mark.parametrize("odt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", LARGE)
def test_matmul_large(dev, m, n, k, odt):
    """On a spread of rows and columns, the first and last among them: the definition needs not every one."""
    torch, moe = dev
    rng = np.random.default_rng(m + n + k)
    wv, wc, wsc = weights_of(rng, n, k)
    xv, xc = codes_of(rng, (m, k))
    e = np.full((m, moe.scale_ld(k)), 127, np.uint8)
    e[:, :-(-k // 128)] = rng.integers(110, 140, (m, -(-k // 128)))
    odt = torch.bfloat16 if odt == "bf16" else torch.float32
    out = torch.full((m + 1, n), 123.0, dtype=odt, device="cuda")
    say("matmul", m, n, k, odt)
    moe.moe_block_matmul(torch.from_numpy(xc).cuda(), torch.from_numpy(e).cuda(), torch.from_numpy(wc).cuda(),
                         torch.from_numpy(wsc).cuda(), out[:m])
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([np.arange(0, m, 29), np.arange(max(0, m - 40), m)]))
    cols = np.unique(np.concatenate([np.arange(0, n, 13), np.arange(max(0, n - 40), n)]))
    xd = R.dequant_rows(xv, np.ldexp(1.0, e[:, :-(-k // 128)].astype(int) - 127))[rows]
    wd = R.dequant_weight(wv, wsc.astype(np.float64))[cols]
    ref, err = R.matmul(xd, wd, cut=odt == torch.bfloat16)
    got = out[:m].double().cpu().numpy()
    assert np.isfinite(got).all() and (out[m] == 123.0).all()
    lim = err if odt == torch.float32 else R.bf16_bound(ref, err)
    assert (np.abs(got[np.ix_(rows, cols)] - ref) <= lim).all()


@pytest.mark.parametrize("m,n,k", [(1, 640, 2048), (4, 33, 1040), (5, 640, 272), (16, 200, 6144), (16, 9000, 144), (17, 64, 256)])
def test_matmul_rows_quantised_first(dev, m, n, k):
    """Rows handed in as bf16 or fp32 give what their quantised codes give, bit for bit, with the scales
    of zero blocks, tiny, huge and non-finite ones."""
    torch, moe = dev
    rng = np.random.default_rng(m * n + k)
    _, wc, wsc = weights_of(rng, n, k)
    w, ws = torch.from_numpy(wc).cuda(), torch.from_numpy(wsc).cuda()
    x = torch.randn((m, k), device="cuda") * torch.exp(torch.randn((m, 1), device="cuda") * 4)
    for i, v in enumerate((0.0, 1e-37, 2.0 ** -140, 1e30, float("inf"), float("nan"))):
        x[i % m, min(16 * i, k - 16):][:16] = v
    for dt in (torch.bfloat16, torch.float32):
        xr = x.to(dt)
        q, s = torch.empty((m, k), dtype=torch.uint8, device="cuda"), torch.empty((m, moe.scale_ld(k)), dtype=torch.uint8, device="cuda")
        moe.moe_quantize_rows(xr, q, s)
        for odt in (torch.bfloat16, torch.float32):
            say("rows", m, n, k, dt, odt)
            a, b = (torch.full((m, n), 7.0, dtype=odt, device="cuda") for _ in range(2))
            moe.moe_block_matmul(xr, None, w, ws, a, moe.block_matmul_workspace(xr, n))
            moe.moe_block_matmul(q, s, w, ws, b)
            torch.cuda.synchronize()
            ints = torch.int16 if odt == torch.bfloat16 else torch.int32
            same = (a.view(ints) == b.view(ints)) | (torch.isnan(a) & torch.isnan(b))
            assert same.all()


def test_matmul_scale_range(dev):
    """Row scales over the whole e8m0 range that keeps the result finite, and
    weight scales that are not powers of two: one nonzero product per output."""
    torch, moe = dev
    k, n = 256, 32
    e = np.full((12, 4), 127, np.uint8)
    e[:, 0] = [1, 2, 20, 60, 100, 126, 127, 128, 150, 200, 230, 246]
    e[:, 1] = 127
    xc = np.zeros((12, k), np.uint8)
    xc[:, 3] = 0x38  # 1.0
    wc = np.zeros((n, k), np.uint8)
    wc[:, 3] = 0x3C  # 1.5
    ws = np.array([[0.37, 1.0]], np.float32)
    out = torch.empty((12, n), device="cuda")
    moe.moe_block_matmul(torch.from_numpy(xc).cuda(), torch.from_numpy(e).cuda(), torch.from_numpy(wc).cuda(),
                         torch.from_numpy(ws).cuda(), out)
    torch.cuda.synchronize()
    want = (np.ldexp(1.5, e[:, :1].astype(int) - 127) * np.float64(np.float32(0.37))).astype(np.float32)
    got = out.cpu().numpy()
    normal = want[:, 0] >= 2.0 ** -126
    assert np.array_equal(got[normal], np.repeat(want[normal], n, 1))
    assert (np.abs(got[~normal] - want[~normal]) <= 2.0 ** -126).all()


def test_matmul_poison(dev):
    """A row with a NaN scale (or NaN codes) is NaN, its neighbours are not."""
    torch, moe = dev
    for m, n, k in ((5, 64, 256), (70, 300, 400), (300, 256, 512)):
        say("poison", m, n, k)
        x = torch.randn((m, k), device="cuda").bfloat16()
        x[2, k - 1] = float("inf")
        rng = np.random.default_rng(1)
        _, wc, wsc = weights_of(rng, n, k)
        out = torch.empty((m, n), device="cuda")
        moe.moe_block_matmul(x, None, torch.from_numpy(wc).cuda(), torch.from_numpy(wsc).cuda(), out,
                             moe.block_matmul_workspace(x, n))
        torch.cuda.synchronize()
        nan = torch.isnan(out).cpu().numpy()
        assert nan[2].all() and not np.delete(nan, 2, 0).any()


def test_matmul_long_offsets(dev):
    """Weights of more than 2^31 bytes: the last columns of the last rows count."""
    torch, moe = dev
    n, k, m = 20000, 131072, 2
    w = torch.zeros((n, k), dtype=torch.uint8, device="cuda")
    w[n - 1, k - 1] = 0x40  # 2.0
    w[17, 5] = 0x38
    ws = torch.ones((-(-n // 128), k // 128), device="cuda")
    x = torch.zeros((m, k), device="cuda").bfloat16()
    x[1, k - 1], x[1, 5] = 3.0, 1.0
    out = torch.empty((m, n), device="cuda")
    moe.moe_block_matmul(x, None, w, ws, out, moe.block_matmul_workspace(x, n))
    torch.cuda.synchronize()
    assert out[1, n - 1].item() == 6.0 and out[1, 17].item() == 1.0 and out.abs().sum().item() == 7.0


def test_matmul_other_stream_and_graph(dev):
    """On a side stream, and captured: replays on new inputs equal eager calls."""
    torch, moe = dev
    rng = np.random.default_rng(5)
    _, wc, wsc = weights_of(rng, 520, 1040)
    w, ws = torch.from_numpy(wc).cuda(), torch.from_numpy(wsc).cuda()
    for m in (1, 40, 300):
        x = torch.randn((m, 1040), device="cuda").bfloat16()
        out, wk = torch.empty((m, 520), device="cuda"), moe.block_matmul_workspace(x, 520)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            moe.moe_block_matmul(x, None, w, ws, out, wk)
        s.synchronize()
        want = torch.empty_like(out)
        moe.moe_block_matmul(x, None, w, ws, want, wk)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_block_matmul(x, None, w, ws, out, wk)
        for i in range(3):
            x.copy_(torch.randn((m, 1040), device="cuda").bfloat16())
            out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            moe.moe_block_matmul(x, None, w, ws, want, moe.block_matmul_workspace(x, 520))
            torch.cuda.synchronize()
            assert torch.equal(out, want), (m, i)


# ---------------------------------------------------------------------------
# experts and layer
# ---------------------------------------------------------------------------

def make_f8_layer(T, d, E, k, F, Fs=None, n_shared=1, seed=0):
    rng = np.random.default_rng(seed)
    Fs = F if Fs is None else Fs
    L = dict(wr=(rng.standard_normal((E, d)) / np.sqrt(d)).astype(np.float32),
             bias=(rng.random(E) * 0.02 - 0.01).astype(np.float32))
    import torch
    L["x"] = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).bfloat16()
    shapes = dict(gate=(E, F, d), up=(E, F, d), down=(E, d, F), s_gate=(1, Fs, d), s_up=(1, Fs, d), s_down=(1, d, Fs))
    for key, (n, rows, cols) in shapes.items():
        if key[0] != "s" or n_shared:
            v, c, s = weights_of(rng, rows, cols, n)
            L[key] = (c, s)
    return L


def upload(L):
    import torch
    W = {key: tuple(torch.from_numpy(a).cuda() for a in L[key]) for key in L if isinstance(L[key], tuple)}
    W["w_router"], W["bias"] = torch.from_numpy(L["wr"]).cuda(), torch.from_numpy(L["bias"]).cuda()
    return W


def layer_ref(L, idx, w, n_shared):
    """(y, bound) of the layer for a given routing (its products may come from the 8-bit instruction)."""
    cut = True
    xd = R.dequant_rows(*R.quantize(L["x"].double().numpy()))
    T, k = idx.shape

    def mats(e, keys):
        return [R.dequant_weight(R.e4m3_decode(L[key][0][e]), L[key][1][e].astype(np.float64)) for key in keys]

    y, err, mag = np.zeros((T, L["x"].shape[1])), 0.0, 0.0
    if n_shared:
        y, err = R.expert(xd, *mats(0, ("s_gate", "s_up", "s_down")), cut)
        mag = np.abs(y)
    err, mag = np.zeros_like(y) + err, np.zeros_like(y) + mag
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        r, re = R.expert(xd[t], *mats(e, ("gate", "up", "down")), cut)
        wt = w[t, j][:, None].astype(np.float64)
        y[t] += wt * r
        err[t] += np.abs(wt) * re
        mag[t] += np.abs(wt * r)
    return y, err + (k + 2) * 2.0 ** -23 * (mag + err)


LAYERS = [dict(T=1, d=128, E=4, k=1, F=128), dict(T=1, d=192, E=16, k=8, F=64, Fs=320),
          dict(T=3, d=320, E=12, k=3, F=192, n_shared=0), dict(T=8, d=256, E=8, k=2, F=128),
          dict(T=20, d=128, E=4, k=4, F=192), dict(T=33, d=192, E=64, k=6, F=128, Fs=64),
          dict(T=70, d=448, E=6, k=2, F=256), dict(T=150, d=256, E=3, k=1, F=320), dict(T=300, d=192, E=5, k=3, F=128),
          dict(T=700, d=128, E=2, k=2, F=256, Fs=128)]


@pytest.mark.parametrize("spec", LAYERS, ids=lambda s: "T%d_d%d_E%d_k%d_F%d" % (s["T"], s["d"], s["E"], s["k"], s["F"]))
def test_layer(dev, spec):
    torch, moe = dev
    say("layer", spec)
    n_shared = spec.get("n_shared", 1)
    L = make_f8_layer(seed=spec["T"], **spec)
    W = upload(L)
    T, d, E, k = spec["T"], spec["d"], spec["E"], spec["k"]
    c = moe.make_config(T, d, E, k, spec["F"], n_shared=n_shared, Fs=spec.get("Fs"), score="sigmoid", route_scale=1.5,
                        act="bf16", w="f8b128")
    x = L["x"].cuda()
    Wm = moe.make_weights(W)
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    lg = torch.empty((T, E), device="cuda")
    ys = []
    for dt in (torch.float32, torch.bfloat16):
        y = torch.full((T + 1, d), 77.0, dtype=dt, device="cuda")
        ws = moe.workspace(c)
        ws.fill_(0xA5)
        moe.moe_layer_forward_grouped(c, None, x, Wm, y[:T], ws, debug=dict(topk_idx=idx, topk_w=w, logits=lg))
        torch.cuda.synchronize()
        assert (y[T] == 77.0).all()
        ys.append(y[:T].double().cpu().numpy())
    want = (L["x"].double() @ torch.from_numpy(L["wr"]).double().t()).float().numpy()
    assert H.ulp_diff_f32(lg.cpu().numpy(), want).max() <= 1  # one rounding of an fp64 sum
    ref_idx, _ = R.select(lg.cpu().numpy(), L["bias"], k, "sigmoid", 1.5)
    assert np.array_equal(idx.cpu().numpy(), ref_idx)
    ref, err = layer_ref(L, ref_idx, w.cpu().numpy(), n_shared)
    say("   bound / rms %.2e, error / rms %.2e" % (err.max() / ref.std(), np.abs(ys[0] - ref).max() / ref.std()))
    assert (np.abs(ys[0] - ref) <= err).all()
    assert (np.abs(ys[1] - ref) <= R.bf16_bound(ref, err)).all()
    # the split calls and the layer without a workspace give the same bits
    off, perm, inv = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
    moe.moe_permute(c, idx, off, perm, inv, ws)
    slot, sh = torch.full((T * k, d), 5.0, device="cuda"), torch.empty((T, d), device="cuda") if n_shared else None
    moe.moe_expert_ffn(c, x, Wm, off, perm, w, slot, sh, ws)
    y2, y3 = torch.empty((T, d), device="cuda"), torch.empty((T, d), device="cuda")
    moe.moe_combine(c, slot, sh, y2)
    moe.moe_layer_forward_noalloc(c, x, Wm, y3)
    torch.cuda.synchronize()
    assert np.array_equal(y3.double().cpu().numpy(), ys[0])
    if T > 8:
        assert np.array_equal(y2.double().cpu().numpy(), ys[0])
    else:  # the few-token path may add in another order
        assert (np.abs(y2.double().cpu().numpy() - ref) <= err).all()


def f8_exact(T, d, E, k, F, Fs=None, seed=0, skew=0.0):
    """An exact-arithmetic bf16 layer (synth.configs.exact_layer) with its weights as
    e4m3 codes and block scales of 1, 1/2 or 1/4, and its output: h is an
    integer of at most 220, quantised to four significant bits."""
    L = configs.exact_layer(T, d, E, k, F, Fs, act="bf16", w="bf16", seed=seed, skew=skew)
    rng = np.random.default_rng(seed + 1)
    import torch
    out = dict(cfg=L["cfg"], x=L["x"], wr=L["w_router"])
    for key in ("gate", "up", "down", "s_gate", "s_up", "s_down"):
        v = (L[key].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        n, rows, cols = v.shape
        sh = rng.integers(0, 3, (n, -(-rows // 128), -(-cols // 128)))
        full = np.repeat(np.repeat(2.0 ** sh, 128, 1), 128, 2)[:, :rows, :cols]
        c = torch.from_numpy(v * full).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        out[key] = (c, (2.0 ** -sh).astype(np.float32))
        out[key + "_v"] = v
    return out


@pytest.mark.parametrize("spec", [dict(T=1, d=256, E=32, k=8, F=128), dict(T=8, d=192, E=16, k=4, F=192, Fs=64),
                                  dict(T=40, d=320, E=64, k=4, F=128), dict(T=130, d=256, E=8, k=2, F=256),
                                  dict(T=600, d=192, E=16, k=4, F=128, skew=1.5),
                                  dict(T=1500, d=128, E=4, k=2, F=320, skew=1.0)],
                         ids=lambda s: "T%d_E%d_F%d" % (s["T"], s["E"], s["F"]))
def test_layer_exact(dev, spec):
    """Every product and sum is exact, so y must equal the definition's bits."""
    torch, moe = dev
    say("exact", spec)
    L = f8_exact(**spec)
    cfg = L["cfg"]
    T, d, E, k = cfg["T"], cfg["d"], cfg["E"], cfg["k"]
    xv = (L["x"].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    xd = R.dequant_rows(*R.quantize(xv))
    assert np.array_equal(xd, xv)
    c = moe.make_config(T, d, E, k, cfg["F"], Fs=cfg["Fs"], score="sigmoid", act="bf16", w="f8b128")
    W = {key: tuple(torch.from_numpy(a).cuda() for a in L[key]) for key in ("gate", "up", "down", "s_gate", "s_up", "s_down")}
    W["w_router"] = torch.from_numpy(L["wr"]).cuda()
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    y = torch.empty((T, d), device="cuda")
    moe.moe_layer_forward_grouped(c, None, H.to_dev(L["x"]), moe.make_weights(W), y, moe.workspace(c),
                                  debug=dict(topk_idx=idx, topk_w=w))
    torch.cuda.synchronize()
    assert (w == 1.0 / k).all()

    def expert(rows, p, e):
        h = (rows @ L[p + "gate_v"][e].T) * (rows @ L[p + "up_v"][e].T)  # silu(g) = g for g >= 20
        return R.dequant_rows(*R.quantize(h)) @ L[p + "down_v"][e].T

    ref = expert(xd, "s_", 0)
    ii = idx.cpu().numpy()
    for e in range(E):
        t, _ = np.nonzero(ii == e)
        if len(t):
            ref[t] += expert(xd[t], "", e) / k
    assert np.array_equal(y.double().cpu().numpy(), ref)


def test_expert_ffn_partial_routing(dev):
    """Assignments the permutation leaves out (index -1) are not written; offsets
    that are no split of the rows leave every slot row alone."""
    torch, moe = dev
    T, d, E, k, F = 50, 192, 8, 3, 128
    L = make_f8_layer(T, d, E, k, F, seed=3)
    W = upload(L)
    c = moe.make_config(T, d, E, k, F, act="bf16", w="f8b128")
    rng = np.random.default_rng(3)
    idx = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]).astype(np.int32)
    idx[rng.random((T, k)) < 0.4] = -1
    w = torch.rand((T, k), device="cuda")
    ws, Wm = moe.workspace(c), moe.make_weights(W)
    off, perm, inv = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
    moe.moe_permute(c, torch.from_numpy(idx).cuda(), off, perm, inv, ws)
    slot, sh = torch.full((T * k, d), 5.0, device="cuda"), torch.empty((T, d), device="cuda")
    moe.moe_expert_ffn(c, L["x"].cuda(), Wm, off, perm, w, slot, sh, ws)
    torch.cuda.synchronize()
    left = torch.from_numpy((idx < 0).reshape(-1)).cuda()
    assert (slot[left] == 5.0).all() and not (slot[~left] == 5.0).any()
    want_sh, err = layer_ref(L, np.zeros((T, 0), np.int32), np.zeros((T, 0)), 1)
    assert (np.abs(sh.double().cpu().numpy() - want_sh) <= err).all()
    off[3] = T * k + 5
    slot.fill_(5.0)
    moe.moe_expert_ffn(c, L["x"].cuda(), Wm, off, perm, w, slot, sh, ws)
    torch.cuda.synchronize()
    assert (slot == 5.0).all()


@pytest.mark.parametrize("T", [1, 5, 64, 300])
def test_layer_graph(dev, T):
    """Routing, quantisation, experts and sum captured together; two graphs with
    workspaces of their own, replayed in turn on new inputs."""
    torch, moe = dev
    L = make_f8_layer(T, 256, 16, 4, 192, seed=9)
    W = upload(L)
    c = moe.make_config(T, 256, 16, 4, 192, score="softmax", route_scale=2.0, act="bf16", w="f8b128")
    g = moe.make_groups(4, 2, 2)
    Wm = moe.make_weights(W)
    sets = []
    for i in range(2):
        x, y, ws = L["x"].cuda(), torch.empty((T, 256), dtype=torch.bfloat16, device="cuda"), moe.workspace(c)
        moe.moe_layer_forward_grouped(c, g, x, Wm, y, ws)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            moe.moe_layer_forward_grouped(c, g, x, Wm, y, ws)
        sets.append((x, y, ws, gr))
    want, wk = torch.empty((T, 256), dtype=torch.bfloat16, device="cuda"), moe.workspace(c)
    for i in range(3):
        for x, y, ws, gr in sets:
            x.copy_(torch.randn((T, 256), device="cuda").bfloat16())
            y.fill_(float("nan"))
            gr.replay()
        for x, y, ws, gr in sets:
            moe.moe_layer_forward_grouped(c, g, x, Wm, want, wk)
            torch.cuda.synchronize()
            assert torch.equal(y, want), (T, i)


def test_prefetch_changes_no_result(dev):
    """e4m3 experts fetched ahead, on the layer's stream and beside it: the layer's output is the same."""
    torch, moe = dev
    T, d, E, k, F = 6, 256, 16, 4, 192
    L = make_f8_layer(T, d, E, k, F, seed=3)
    W = upload(L)
    c = moe.make_config(T, d, E, k, F, score="softmax", route_scale=2.0, act="bf16", w="f8b128")
    Wm, x, ws = moe.make_weights(W), L["x"].cuda(), moe.workspace(c)
    want, y = (torch.empty((T, d), device="cuda") for _ in range(2))
    moe.moe_layer_forward_grouped(c, None, x, Wm, want, ws)
    ids = torch.tensor([E - 1, 0, -1, E, 1 << 30, 5], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    for which in range(1, 8):
        say("prefetch", which)
        moe.moe_prefetch_experts(c, Wm, ids, which=which, rows=(0, 3, 1 << 30)[which % 3], workgroups=1 + 7 * which)
        side.wait_stream(torch.cuda.current_stream())
        moe.moe_prefetch_experts(c, Wm, ids, which=which, workgroups=64, stream=side.cuda_stream)
        moe.moe_layer_forward_grouped(c, None, x, Wm, y.fill_(9.0), ws)
        torch.cuda.synchronize()
        assert torch.equal(y, want), which


def test_run_together(dev):
    """A serving step as a program runs it: a projection of the rows, grouped routing of
    its output, the experts over that routing, the sum; against the definitions."""
    torch, moe = dev
    T, d, E, k, F = 45, 256, 16, 4, 128
    L = make_f8_layer(T, d, E, k, F, seed=21)
    W = upload(L)
    rng = np.random.default_rng(4)
    pv, pc, ps = weights_of(rng, d, d)
    x0 = L["x"].cuda()
    q, s = torch.empty((T, d), dtype=torch.uint8, device="cuda"), torch.empty((T, 4), dtype=torch.uint8, device="cuda")
    moe.moe_quantize_rows(x0, q, s)
    x = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    moe.moe_block_matmul(q, s, torch.from_numpy(pc).cuda(), torch.from_numpy(ps).cuda(), x)
    c = moe.make_config(T, d, E, k, F, score="softmax", route_scale=1.5, act="bf16", w="f8b128")
    g = moe.make_groups(4, 2, 2)
    lg, idx, w = torch.empty((T, E), device="cuda"), torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    moe.moe_route_grouped(c, g, x, W["w_router"], W["bias"], lg, idx, w, None)
    ws = moe.workspace(c)
    off, perm, inv = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
    moe.moe_permute(c, idx, off, perm, inv, ws)
    slot, sh, y = torch.empty((T * k, d), device="cuda"), torch.empty((T, d), device="cuda"), torch.empty((T, d), device="cuda")
    moe.moe_expert_ffn(c, x, moe.make_weights(W), off, perm, w, slot, sh, ws)
    moe.moe_combine(c, slot, sh, y)
    torch.cuda.synchronize()
    ref, err = R.matmul(R.dequant_rows(*R.quantize(L["x"].double().numpy())), R.dequant_weight(pv, ps.astype(np.float64)), cut=True)
    assert (np.abs(x.double().cpu().numpy() - ref) <= R.bf16_bound(ref, err)).all()
    ri, rw = R.select(lg.cpu().numpy(), L["bias"], k, "softmax", 1.5, 4, 2, 2, True)
    assert np.array_equal(idx.cpu().numpy(), ri)
    L["x"] = x.cpu()
    ref, err = layer_ref(L, ri, w.cpu().numpy(), 1)
    assert (np.abs(y.double().cpu().numpy() - ref) <= err).all()
