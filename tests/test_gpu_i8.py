"""The int8 operators on the GPU against their float64 definitions (i8_ref, which derives the bounds): scales, codes
and products bit for bit, layers within the bound of fp32 roundings carried through the quantised intermediate."""
import sys

import numpy as np
import pytest

import f8_ref
import gpu_harness as H
import i8_ref as R

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


def weights_of(rng, rows, cols, n=None, full=False):
    """int8 codes and row scales; full: every code, -128 among them."""
    shape = (rows, cols) if n is None else (n, rows, cols)
    if full:
        q = rng.integers(-128, 128, shape).astype(np.int8)
    else:
        q = np.clip(np.rint(rng.standard_normal(shape) * 32), -127, 127).astype(np.int8)
    return q, ((rng.random(shape[:-1]) + 0.5) * (0.03 / 32)).astype(np.float32)


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

def quant_rows(rng, rows, cols):
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal((rows, 1)) * 4)
    x[:, ::17] *= 30
    for i, v in enumerate([0.0, 127.0, 128.0, 3e38, 1e-38, 2.0 ** -130, -0.0, 2.0 ** -114]):
        if i < rows:
            x[i] = 0.0
            x[i, i % cols] = v
    if rows > 10:
        x[9] = rng.integers(-254, 255, cols)  # scale 2: every odd value is a tie
        x[9, 0] = 254
        x[10] = rng.integers(-127, 128, cols) / 2.0  # multiples of amax / 127 and halves of them, scaled by fp32(1/127)
        x[10, 0] = 63.5
    if rows > 12:
        x[11] = 1.0
        x[12] = rng.integers(-255, 256, cols) * 2.0 ** -7  # over amax = 1, bf16 values next to borders
        x[12, 0] = 1.0
    return x


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,ld", [(1, 16, 16), (1, 4096, 4096), (3, 112, 128), (33, 128, 128), (17, 144, 160),
                                          (10, 1040, 1040), (129, 512, 640), (13, 2064, 2064), (20, 8176, 8192),
                                          (5, 8208, 8208), (3, 40000, 40000), (1000, 6144, 6144)])
def test_quantize(dev, rows, cols, ld, dt):
    torch, moe = dev
    say("quantize tokens", rows, cols, ld, dt)
    rng = np.random.default_rng(rows + cols)
    buf = torch.full((rows, ld), 7e30, dtype=torch.float32)
    buf[:, :cols] = torch.from_numpy(quant_rows(rng, rows, cols).astype(np.float32))
    buf = buf.bfloat16() if dt == "bf16" else buf
    x = buf.cuda()[:, :cols]
    q = torch.full((rows + 2, cols), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 2,), 7.0, device="cuda")
    moe.moe_quantize_tokens(x, q[1:-1], s[1:-1])
    torch.cuda.synchronize()
    want_q, want_s = R.quantize(buf[:, :cols].double().numpy())
    assert np.array_equal(s[1:-1].cpu().numpy(), want_s)
    assert np.array_equal(q[1:-1].cpu().numpy(), want_q)
    assert (q[[0, -1]] == 77).all() and (s[[0, -1]] == 7.0).all()  # the rows around them are left alone


def test_quantize_every_border(dev):
    """For scales with many different roundings, the values on, just below and just above every border."""
    torch, moe = dev
    rng = np.random.default_rng(7)
    amax = np.concatenate([np.exp(rng.standard_normal(300) * 20), [127.0, 1.0, 0.1, 3.4e38, 2.0 ** -113 * 127, 1e-30]])
    amax = amax.astype(np.float32)
    s = np.maximum((amax.astype(np.float64) / 127).astype(np.float32), np.float32(R.MIN_SCALE))
    mid = (np.arange(-127, 127) + 0.5)[None] * s.astype(np.float64)[:, None]
    v = mid.astype(np.float32)
    x = np.concatenate([amax[:, None], v, np.nextafter(v, np.float32(np.inf)), np.nextafter(v, np.float32(-np.inf))], 1)
    x = np.clip(x, -amax[:, None], amax[:, None])
    x = np.pad(x, ((0, 0), (0, -x.shape[1] % 16)))
    q, sc = torch.empty(x.shape, dtype=torch.int8, device="cuda"), torch.empty(len(x), device="cuda")
    moe.moe_quantize_tokens(torch.from_numpy(x).cuda(), q, sc)
    torch.cuda.synchronize()
    want_q, want_s = R.quantize(x.astype(np.float64))
    assert np.array_equal(sc.cpu().numpy(), want_s) and np.array_equal(want_s, s)
    assert np.array_equal(q.cpu().numpy(), want_q)


def test_quantize_poisoned_rows(dev):
    torch, moe = dev
    x = torch.ones((6, 272), device="cuda")
    x[0, 5], x[1, 130], x[2, 271], x[3, 0], x[3, 1] = float("nan"), float("inf"), float("-inf"), float("inf"), float("nan")
    for t in (x, x.bfloat16()):
        q, s = torch.empty((6, 272), dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
        moe.moe_quantize_tokens(t, q, s)
        torch.cuda.synchronize()
        assert torch.isnan(s).tolist() == [True] * 4 + [False] * 2
        assert (q[:4] == 0).all() and (q[4:] == 127).all()


def test_quantize_many_rows(dev):
    """More rows than one launch has workgroups for."""
    torch, moe = dev
    rows = 140000
    x = torch.randn((rows, 16), device="cuda")
    x[70000] = 0
    q, s = torch.empty((rows, 16), dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    moe.moe_quantize_tokens(x, q, s)
    torch.cuda.synchronize()
    want_q, want_s = R.quantize(x.double().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.cpu().numpy(), want_q)


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

def check_product(torch, got, q, s, w, ws):
    """Bit for bit, in fp32 or rounded once more to bf16."""
    want = R.product_f32(q, s, w, ws)
    if got.dtype == torch.bfloat16:
        want = R.to_bf16(want)
    got = got.float().cpu().numpy()
    bad = np.argwhere(got != want)
    assert not len(bad), (len(bad), bad[:4], got[tuple(bad[0])], want[tuple(bad[0])])


SIZES = [(1, 16, 16), (1, 4096, 6144), (1, 1, 128), (2, 130, 144), (5, 67, 1040), (15, 256, 128), (16, 96, 272),
         (17, 200, 512), (32, 129, 2048), (33, 48, 640), (48, 1000, 4112), (64, 1000, 1152), (65, 256, 256),
         (77, 640, 2048), (128, 384, 896), (200, 130, 304), (257, 512, 512), (300, 1037, 1296), (513, 256, 2048),
         (1030, 770, 400)]


@pytest.mark.parametrize("xdt", ["i8", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_matmul(dev, m, n, k, xdt):
    torch, moe = dev
    rng = np.random.default_rng(m * 7 + n * 3 + k)
    wq, wsc = weights_of(rng, n, k, full=True)
    w, wscale = torch.from_numpy(wq).cuda(), torch.from_numpy(wsc).cuda()
    if xdt == "i8":
        q = rng.integers(-128, 128, (m, k)).astype(np.int8)
        s = np.exp(rng.standard_normal(m) * 3).astype(np.float32)
        x, xs = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
    else:
        x = torch.from_numpy((rng.standard_normal((m, k)) * 3).astype(np.float32))
        x = x.bfloat16() if xdt == "bf16" else x
        q, s = R.quantize(x.double().numpy())
        x, xs = x.cuda(), None
    for odt in (torch.float32, torch.bfloat16):
        say("channel matmul m=%d n=%d k=%d %s -> %s" % (m, n, k, xdt, odt))
        out = torch.full((m + 1, n), 123.0, dtype=odt, device="cuda")
        wk = moe.channel_matmul_workspace(x)
        if wk is not None:
            wk.fill_(0xFF)  # the workspace needs no initialisation
        moe.moe_channel_matmul(x, xs, w, wscale, out[:m], wk)
        torch.cuda.synchronize()
        check_product(torch, out[:m], q, s, wq, wsc)
        assert (out[m] == 123.0).all()  # the row behind the last is left alone


# sizes of every larger tile, with ends in rows, columns and K; K below one step; long K
LARGE = [(1600, 2000, 272), (3500, 3600, 400), (70, 200, 16), (300, 70, 112), (1600, 2000, 48), (3500, 3600, 80),
         (90, 150, 8464), (600, 1000, 8464), (1600, 2000, 8320), (250, 1000, 2064), (8000, 20, 1040), (70, 132, 144),
         (70, 133, 144), (70, 134, 144), (70, 136, 144), (3500, 3601, 144), (3500, 3602, 144), (1700, 2001, 144),
         (2000, 3899, 272), (2000, 3900, 48), (2200, 4100, 400), (2200, 4099, 144), (40, 24000, 400)]


@pytest.mark.parametrize("odt", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k", LARGE)
def test_matmul_large(dev, m, n, k, odt):
    """On a spread of rows and columns, the first and last among them: the definition needs not every one."""
    torch, moe = dev
    rng = np.random.default_rng(m + n + k)
    wq, wsc = weights_of(rng, n, k, full=True)
    q = rng.integers(-128, 128, (m, k)).astype(np.int8)
    s = np.exp(rng.standard_normal(m)).astype(np.float32)
    out = torch.full((m + 1, n), 123.0, dtype=torch.bfloat16 if odt == "bf16" else torch.float32, device="cuda")
    say("channel matmul", m, n, k, odt)
    moe.moe_channel_matmul(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda(), torch.from_numpy(wq).cuda(),
                           torch.from_numpy(wsc).cuda(), out[:m])
    torch.cuda.synchronize()
    assert (out[m] == 123.0).all() and torch.isfinite(out).all()
    rows = np.unique(np.concatenate([np.arange(0, m, 29), np.arange(max(0, m - 40), m)]))
    cols = np.unique(np.concatenate([np.arange(0, n, 13), np.arange(max(0, n - 40), n)]))
    check_product(torch, out[:m].cpu()[np.ix_(rows, cols)], q[rows], s[rows], wq[cols], wsc[cols])


# one size for each kernel of the dense product; every number of whole steps of K from none on, with and without an end
@pytest.mark.parametrize("m,n", [(3, 40), (20, 2100), (70, 2100), (300, 2100), (1500, 1700), (2000, 3900), (2200, 4100), (3500, 3600)])
def test_matmul_every_k(dev, m, n):
    torch, moe = dev
    rng = np.random.default_rng(m + n)
    for k in [16, 112, 128, 144, 256, 272, 384, 400, 512, 528, 640, 656, 768, 784, 896, 1024, 1152, 1168]:
        wq, wsc = weights_of(rng, n, k, full=True)
        q = rng.integers(-128, 128, (m, k)).astype(np.int8)
        s = np.exp(rng.standard_normal(m)).astype(np.float32)
        say("channel matmul", m, n, k)
        out = torch.full((m, n), 123.0, device="cuda")
        moe.moe_channel_matmul(*(torch.from_numpy(a).cuda() for a in (q, s, wq, wsc)), out)
        torch.cuda.synchronize()
        rows, cols = (np.unique(np.concatenate([np.arange(0, e, 37), np.arange(max(0, e - 5), e)])) for e in (m, n))
        check_product(torch, out.cpu()[np.ix_(rows, cols)], q[rows], s[rows], wq[cols], wsc[cols])


def test_matmul_largest_sums(dev):
    """The longest K with every code at its largest magnitude: sums next to 2^31, exact, and all of one sign."""
    torch, moe = dev
    k = 131056
    for m in (1, 20, 130):
        say("largest sums, m =", m)
        q = np.full((m, k), -128, np.int8)
        q[::2] = 127
        wq = np.full((40, k), -128, np.int8)
        wq[::3] = 127
        s, ws = np.ones(m, np.float32), np.ones(40, np.float32)
        out = torch.empty((m, 40), device="cuda")
        moe.moe_channel_matmul(*(torch.from_numpy(a).cuda() for a in (q, s, wq, ws)), out)
        torch.cuda.synchronize()
        check_product(torch, out, q, s, wq, ws)


def test_matmul_long_offsets(dev):
    """Weights, rows and results of more than 2^31 bytes: the last of each count."""
    torch, moe = dev
    k = 131056
    for m, n in ((2, 20000), (17000, 70)):
        say("long offsets", m, n)
        w, x = (torch.zeros((r, k), dtype=torch.int8, device="cuda") for r in (n, m))
        w[n - 1, k - 1], w[17, 5] = 2, 1
        x[m - 1, k - 1], x[m - 1, 5] = 3, 1
        out = torch.empty((m, n), device="cuda")
        moe.moe_channel_matmul(x, torch.ones(m, device="cuda"), w, torch.ones(n, device="cuda"), out)
        torch.cuda.synchronize()
        assert out[m - 1, n - 1].item() == 6.0 and out[m - 1, 17].item() == 1.0 and out.abs().sum().item() == 7.0
    m, n = 40000, 30000
    out = torch.empty((m, n), device="cuda")
    x, w = torch.ones((m, 16), dtype=torch.int8, device="cuda"), torch.ones((n, 16), dtype=torch.int8, device="cuda")
    xs = torch.arange(m, device="cuda").float()
    say("long results", m, n)
    moe.moe_channel_matmul(x, xs, w, torch.ones(n, device="cuda"), out)
    torch.cuda.synchronize()
    for i in range(0, m, 8000):
        assert (out[i:i + 8000] == 16.0 * xs[i:i + 8000, None]).all()


def test_matmul_scale_range(dev):
    """Scales of any sign and size whose products stay in range; zero, infinite and NaN ones as arithmetic has it."""
    torch, moe = dev
    k, n = 144, 40
    rng = np.random.default_rng(3)
    s = np.array([1e-38, 2.0 ** -126, 1e-20, -1.0, 0.0, 3e30, 1e38, 2.0 ** -149], np.float32)
    q = np.zeros((8, k), np.int8)
    q[:, 3], q[5:7, 3] = 100, 1
    wq = np.zeros((n, k), np.int8)
    wq[:, 3] = rng.integers(1, 3, n)
    ws = ((rng.random(n) + 0.5) * np.where(rng.random(n) < 0.5, -1, 1)).astype(np.float32)
    out = torch.empty((8, n), device="cuda")
    moe.moe_channel_matmul(*(torch.from_numpy(a).cuda() for a in (q, s, wq, ws)), out)
    torch.cuda.synchronize()
    check_product(torch, out, q, s, wq, ws)
    s[:3] = np.nan, np.inf, -np.inf
    moe.moe_channel_matmul(*(torch.from_numpy(a).cuda() for a in (q, s, wq, ws)), out)
    torch.cuda.synchronize()
    want = R.product_f32(q, s, wq, ws)
    assert np.array_equal(out.cpu().numpy(), want, equal_nan=True) and np.isnan(want[0]).all() and np.isinf(want[1:3]).all()


@pytest.mark.parametrize("m,n,k", [(1, 640, 2048), (4, 33, 1040), (5, 64, 256), (5, 640, 272), (16, 200, 6144),
                                   (16, 9000, 144), (17, 64, 256), (70, 300, 400), (300, 256, 512), (3, 50, 20000)])
def test_matmul_rows_quantised_first(dev, m, n, k):
    """Rows handed in as bf16 or fp32 give what their quantised codes give, bit for bit, those of zeros, tiny, huge
    and non-finite values too: a row that is not finite is NaN, its neighbours are not."""
    torch, moe = dev
    rng = np.random.default_rng(m * n + k)
    wq, wsc = weights_of(rng, n, k)
    w, ws = torch.from_numpy(wq).cuda(), torch.from_numpy(wsc).cuda()
    x = torch.randn((m, k), device="cuda") * torch.exp(torch.randn((m, 1), device="cuda") * 4)
    vals = (0.0, 2.0 ** -140, 1e30, float("inf"), float("nan"))
    for i, v in enumerate(vals):
        if m > i:
            x[i, k - 3 if i == 3 else 1] = v
            if i < 2:
                x[i] = v
    for dt in (torch.bfloat16, torch.float32):
        xr = x.to(dt)
        q, s = torch.empty((m, k), dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
        moe.moe_quantize_tokens(xr, q, s)
        for odt in (torch.bfloat16, torch.float32):
            say("rows", m, n, k, dt, odt)
            a, b = (torch.full((m, n), 7.0, dtype=odt, device="cuda") for _ in range(2))
            moe.moe_channel_matmul(xr, None, w, ws, a, moe.channel_matmul_workspace(xr))
            moe.moe_channel_matmul(q, s, w, ws, b)
            torch.cuda.synchronize()
            ints = torch.int16 if odt == torch.bfloat16 else torch.int32
            nan = torch.isnan(a)
            assert ((a.view(ints) == b.view(ints)) | (nan & torch.isnan(b))).all()
            assert nan.all(1).tolist() == [i in (3, 4) for i in range(m)] and not nan[[i for i in range(m) if i not in (3, 4)]].any()


def test_matmul_other_stream_and_graph(dev):
    """On a side stream, and captured: replays on new inputs equal eager calls."""
    torch, moe = dev
    rng = np.random.default_rng(5)
    wq, wsc = weights_of(rng, 520, 1040)
    w, ws = torch.from_numpy(wq).cuda(), torch.from_numpy(wsc).cuda()
    for m in (1, 40, 300):
        x = torch.randn((m, 1040), device="cuda").bfloat16()
        out, wk = torch.empty((m, 520), device="cuda"), moe.channel_matmul_workspace(x)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            moe.moe_channel_matmul(x, None, w, ws, out, wk)
        s.synchronize()
        want = torch.empty_like(out)
        moe.moe_channel_matmul(x, None, w, ws, want, wk)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moe.moe_channel_matmul(x, None, w, ws, out, wk)
        for i in range(3):
            x.copy_(torch.randn((m, 1040), device="cuda").bfloat16())
            out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            moe.moe_channel_matmul(x, None, w, ws, want, moe.channel_matmul_workspace(x))
            torch.cuda.synchronize()
            assert torch.equal(out, want), (m, i)


# ---------------------------------------------------------------------------
# experts and layer
# ---------------------------------------------------------------------------

def make_layer(T, d, E, k, F, Fs=None, n_shared=1, seed=0):
    import torch
    rng = np.random.default_rng(seed)
    Fs = F if Fs is None else Fs
    L = dict(wr=(rng.standard_normal((E, d)) / np.sqrt(d)).astype(np.float32),
             bias=(rng.random(E) * 0.02 - 0.01).astype(np.float32),
             x=torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).bfloat16())
    shapes = dict(gate=(E, F, d), up=(E, F, d), down=(E, d, F), s_gate=(1, Fs, d), s_up=(1, Fs, d), s_down=(1, d, Fs))
    for key, (n, rows, cols) in shapes.items():
        if key[0] != "s" or n_shared:
            L[key] = weights_of(rng, rows, cols, n)
    return L


def upload(L):
    import torch
    W = {key: tuple(torch.from_numpy(a).cuda() for a in L[key]) for key in L if isinstance(L[key], tuple)}
    W["w_router"], W["bias"] = torch.from_numpy(L["wr"]).cuda(), torch.from_numpy(L["bias"]).cuda()
    return W


def layer_ref(L, idx, w, n_shared):
    """(y, bound) of the layer for a given routing."""
    xd = R.dequant(*R.quantize(L["x"].double().numpy()))
    T, k = idx.shape

    def mats(e, keys):
        return [R.dequant(L[key][0][e], L[key][1][e]) for key in keys]

    y, err = np.zeros((T, L["x"].shape[1])), np.zeros((T, L["x"].shape[1]))
    if n_shared:
        y, err = R.expert(xd, *mats(0, ("s_gate", "s_up", "s_down")))
    mag = np.abs(y)
    for e in np.unique(idx):
        t, j = np.nonzero(idx == e)
        r, re = R.expert(xd[t], *mats(e, ("gate", "up", "down")))
        wt = w[t, j][:, None].astype(np.float64)
        y[t] += wt * r
        err[t] += np.abs(wt) * re
        mag[t] += np.abs(wt * r)
    return y, err + (k + 2) * R.U * (mag + err)


LAYERS = [dict(T=1, d=128, E=4, k=1, F=128), dict(T=1, d=192, E=16, k=8, F=64, Fs=320),
          dict(T=1, d=4160, E=6, k=2, F=2112, Fs=64), dict(T=2, d=64, E=300, k=32, F=64),
          dict(T=3, d=320, E=12, k=3, F=192, n_shared=0), dict(T=8, d=256, E=8, k=2, F=128),
          dict(T=1, d=192, E=8, k=4, F=576, n_shared=0), dict(T=2, d=320, E=16, k=8, F=1088, Fs=2112),
          dict(T=4, d=128, E=6, k=3, F=8192, Fs=64), dict(T=5, d=64, E=4, k=2, F=8256, Fs=128),
          dict(T=9, d=1088, E=20, k=6, F=576, Fs=1600), dict(T=16, d=128, E=600, k=32, F=320),
          dict(T=16, d=192, E=3, k=3, F=64, Fs=640), dict(T=12, d=64, E=40, k=32, F=64, n_shared=0),
          dict(T=16, d=320, E=40, k=5, F=192), dict(T=17, d=320, E=40, k=5, F=192, n_shared=0),
          dict(T=20, d=128, E=4, k=4, F=192), dict(T=33, d=192, E=64, k=6, F=128, Fs=64),
          dict(T=70, d=448, E=6, k=2, F=256), dict(T=150, d=256, E=3, k=1, F=320), dict(T=300, d=192, E=5, k=3, F=128),
          dict(T=700, d=128, E=2, k=2, F=256, Fs=128), dict(T=170, d=640, E=4, k=2, F=384), dict(T=500, d=768, E=4, k=3, F=192), dict(T=900, d=320, E=2, k=1, F=8256, Fs=64)]


@pytest.mark.parametrize("spec", LAYERS, ids=lambda s: "T%d_d%d_E%d_k%d_F%d" % (s["T"], s["d"], s["E"], s["k"], s["F"]))
def test_layer(dev, spec):
    torch, moe = dev
    say("layer", spec)
    n_shared = spec.get("n_shared", 1)
    L = make_layer(seed=spec["T"], **spec)
    W = upload(L)
    T, d, E, k = spec["T"], spec["d"], spec["E"], spec["k"]
    c = moe.make_config(T, d, E, k, spec["F"], n_shared=n_shared, Fs=spec.get("Fs"), score="sigmoid", route_scale=1.5,
                        act="bf16", w="i8ch")
    x, Wm = L["x"].cuda(), moe.make_weights(W)
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
        ys.append(y[:T].float().cpu().numpy())
    want = (L["x"].double() @ torch.from_numpy(L["wr"]).double().t()).float().numpy()
    assert H.ulp_diff_f32(lg.cpu().numpy(), want).max() <= 1  # one rounding of an fp64 sum
    ref_idx, _ = f8_ref.select(lg.cpu().numpy(), L["bias"], k, "sigmoid", 1.5)
    assert np.array_equal(idx.cpu().numpy(), ref_idx)
    ref, err = layer_ref(L, ref_idx, w.cpu().numpy(), n_shared)
    say("   bound / rms %.2e, error / rms %.2e" % (err.max() / ref.std(), np.abs(ys[0] - ref).max() / ref.std()))
    assert (np.abs(ys[0] - ref) <= err).all()
    assert np.array_equal(ys[1], R.to_bf16(ys[0]))
    # the split calls and the layer without a workspace give the same bits
    off, perm, inv = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
    moe.moe_permute(c, idx, off, perm, inv, ws)
    slot, sh = torch.full((T * k, d), 5.0, device="cuda"), torch.empty((T, d), device="cuda") if n_shared else None
    moe.moe_expert_ffn(c, x, Wm, off, perm, w, slot, sh, ws)
    y2, y3, y4 = (torch.empty((T, d), device="cuda") for _ in range(3))
    moe.moe_combine(c, slot, sh, y2)
    if ws.numel() <= moe.binding.STATIC_SCRATCH_BYTES:
        moe.moe_layer_forward_noalloc(c, x, Wm, y3)
    else:
        with pytest.raises(moe.MoeError):
            moe.moe_layer_forward_noalloc(c, x, Wm, y3)
        y3 = y2
    moe.moe_layer_forward(c, x, Wm, y4, ws)
    torch.cuda.synchronize()
    for other in (y2, y3, y4):
        assert np.array_equal(other.cpu().numpy(), ys[0])


def test_layer_poisoned_token(dev):
    """A token with an infinity or a NaN is NaN in y; the others are what they are without it."""
    torch, moe = dev
    for T in (3, 12, 40, 300):
        L = make_layer(T, 256, 8, 2, 128, seed=T)
        W = upload(L)
        c = moe.make_config(T, 256, 8, 2, 128, score="sigmoid", act="bf16", w="i8ch")
        x, Wm, ws = L["x"].cuda(), moe.make_weights(W), moe.workspace(c)
        want, y = (torch.empty((T, 256), device="cuda") for _ in range(2))
        moe.moe_layer_forward_grouped(c, None, x, Wm, want, ws)
        x[1, 255], x[T - 1, 0] = float("inf"), float("nan")
        say("poisoned tokens of", T)
        moe.moe_layer_forward_grouped(c, None, x, Wm, y, ws)
        torch.cuda.synchronize()
        nan = torch.isnan(y).cpu().numpy()
        bad = [t in (1, T - 1) for t in range(T)]
        assert nan[bad].all() and not nan[np.logical_not(bad)].any()
        keep = torch.tensor([not b for b in bad], device="cuda")
        assert torch.equal(y[keep], want[keep])


def test_expert_ffn_partial_routing(dev):
    """Assignments the permutation leaves out (index -1) are not written; offsets
    that are no split of the rows leave every slot row alone."""
    torch, moe = dev
    T, d, E, k, F = 50, 192, 8, 3, 128
    L = make_layer(T, d, E, k, F, seed=3)
    W = upload(L)
    c = moe.make_config(T, d, E, k, F, act="bf16", w="i8ch")
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


@pytest.mark.parametrize("T", [1, 5, 16, 17, 64, 300])
def test_layer_graph(dev, T):
    """Routing, quantisation, experts and sum captured together; two graphs with
    workspaces of their own, replayed in turn on new inputs."""
    torch, moe = dev
    L = make_layer(T, 256, 16, 4, 192, seed=9)
    W = upload(L)
    c = moe.make_config(T, 256, 16, 4, 192, score="softmax", route_scale=2.0, act="bf16", w="i8ch")
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
    """int8 experts fetched ahead, on the layer's stream and beside it: the layer's output is the same."""
    torch, moe = dev
    T, d, E, k, F = 6, 256, 16, 4, 192
    L = make_layer(T, d, E, k, F, seed=3)
    W = upload(L)
    c = moe.make_config(T, d, E, k, F, score="softmax", route_scale=2.0, act="bf16", w="i8ch")
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
