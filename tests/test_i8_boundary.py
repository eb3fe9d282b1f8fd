"""Refusals of the int8 operators, on the CPU (every call fails its checks before the device is touched), and the
float64 definitions the GPU tests compare with, against cases worked out by hand."""
import ctypes
import os

import numpy as np
import pytest

import i8_ref as R

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)
BYTE = ctypes.c_void_p((1 << 20) + 2)
F32, BF16, Q8, F8, I8 = range(5)
MAX_K = 131056


@pytest.fixture(scope="module")
def moe():
    import sparse_moe_layer_02_amd as m
    if not os.path.exists(m.binding.LIB_PATH):
        from sparse_moe_layer_02_amd import build
        build.build()
    m.load()
    return m


def cfg(moe, **kw):
    base = dict(T=4, d=512, E=32, k=4, F=256, score="sigmoid", act="bf16", w="i8ch")
    base.update(kw)
    return moe.make_config(**base)


def weights(moe, **kw):
    m = moe.binding.moe_mat(FAKE.value, FAKE.value + 4)  # scales may start at any 4-byte address
    mats = dict(gate=m, up=m, down=m, s_gate=m, s_up=m, s_down=m)
    mats.update(kw)
    return moe.binding.moe_weights(FAKE.value, None, *mats.values())


def test_layer_refusals(moe):
    lib = moe.load()

    def call(c, y_dtype=F32, y=FAKE, ws_bytes=1000, W=None, f=None):
        W = weights(moe) if W is None else W
        if f == "noalloc":
            return lib.moe_layer_forward_noalloc(ctypes.byref(c), FAKE, ctypes.byref(W), y, None, None)
        return lib.moe_layer_forward_grouped(ctypes.byref(c), None, FAKE, ctypes.byref(W), y, y_dtype, None, FAKE,
                                             ws_bytes, None)

    assert call(cfg(moe)) == 3 and call(cfg(moe), y_dtype=BF16) == 3  # only the workspace is too small
    assert call(cfg(moe), y_dtype=I8) == 1
    assert call(cfg(moe), y=ODD) == 1
    assert call(cfg(moe, act="f32")) == 2
    assert call(cfg(moe, d=480)) == 2
    assert call(cfg(moe, T=9, path="decode")) == 2
    # int32 sums: at most MOE_I8_MAX_K columns
    limit = MAX_K // 64 * 64
    for key in ("d", "F", "Fs"):
        assert call(cfg(moe, **{key: limit})) == 3, key
        assert call(cfg(moe, **{key: limit + 64})) == 2, key
    assert call(cfg(moe, F=128, Fs=limit + 64, n_shared=0)) == 3  # no shared expert: its size is not looked at
    # the quantised rows are addressed with 32 bits
    assert call(cfg(moe, T=1 << 16, d=1 << 16)) == 2 and call(cfg(moe, T=(1 << 16) - 1, d=1 << 16)) == 3
    for key in ("gate", "up", "down", "s_gate", "s_up", "s_down"):
        for m in (moe.binding.moe_mat(FAKE.value, None), moe.binding.moe_mat(FAKE.value, BYTE.value),
                  moe.binding.moe_mat(None, FAKE.value), moe.binding.moe_mat(ODD.value, FAKE.value)):
            assert call(cfg(moe), W=weights(moe, **{key: m})) == 1, key
    assert call(cfg(moe, T=4096, d=6144, F=2048, E=256), f="noalloc") == 3
    assert lib.moe_workspace_bytes(ctypes.byref(moe.moe_config(4, 512, 32, 4, 256, 1, 256, 0, 1.0, 1, 5, 0))) == 0


def test_prefetch_arguments(moe):
    """Of int8 experts only the codes are fetched: a scale array may start at any 4-byte address."""
    lib = moe.load()
    call = lambda w, ids, n: lib.moe_prefetch_experts(ctypes.byref(cfg(moe)), ctypes.byref(w), ids, n, 7, 0, 4, None, None)
    assert call(weights(moe), None, 0) == 0 and call(weights(moe), None, 4) == 1
    assert call(weights(moe, down=moe.binding.moe_mat(FAKE.value, None)), None, 0) == 1


def test_workspace_monotone(moe):
    lib = moe.load()
    base = dict(T=64, d=512, E=32, k=4, F=256, Fs=256)
    for key, sizes in (("T", (1, 8, 9, 16, 17, 31, 64, 65, 160, 1000, 4096)), ("d", (512, 576, 640)),
                       ("E", (32, 33, 64, 300)), ("k", (4, 5, 8)), ("F", (256, 320, 384)), ("Fs", (256, 320, 512))):
        got = [lib.moe_workspace_bytes(ctypes.byref(cfg(moe, **dict(base, **{key: v})))) for v in sizes]
        assert got == sorted(got) and got[0] > 0, (key, got)


@pytest.mark.parametrize("dt,rows,cols,ld", [(Q8, 4, 128, 128), (I8, 4, 128, 128), (-1, 4, 128, 128),
                                             (F32, -1, 128, 128), (F32, 4, 0, 128), (F32, 4, 120, 128),
                                             (BF16, 4, 129, 136), (F32, 4, (1 << 20) + 16, 1 << 21), (F32, 4, 128, 112),
                                             (F32, 4, 128, 130), (BF16, 4, 128, 132), (F32, 4, 128, 1 << 62)])
def test_quantize_refusals(moe, dt, rows, cols, ld):
    assert moe.load().moe_quantize_tokens(FAKE, dt, rows, cols, ld, FAKE, FAKE, None) == 1


def test_quantize_pointers(moe):
    q = moe.load().moe_quantize_tokens
    assert q(None, F32, 4, 128, 128, FAKE, FAKE, None) == 1
    assert q(ODD, F32, 4, 128, 128, FAKE, FAKE, None) == 1
    assert q(FAKE, F32, 4, 128, 128, ODD, FAKE, None) == 1
    assert q(FAKE, F32, 4, 128, 128, FAKE, BYTE, None) == 1
    assert q(FAKE, F32, 4, 128, 128, FAKE, None, None) == 1
    assert q(None, F32, 0, 128, 128, None, None, None) == 0  # no rows: nothing to do


@pytest.mark.parametrize("xdt,m,n,k,odt", [(Q8, 4, 64, 128, F32), (F8, 4, 64, 128, F32), (F32, 4, 64, 128, I8),
                                           (F32, -1, 64, 128, F32), (F32, (1 << 20) + 1, 64, 128, F32),
                                           (F32, 4, 0, 128, F32), (F32, 4, (1 << 20) + 1, 128, F32), (F32, 4, 64, 8, F32),
                                           (F32, 4, 64, 136, F32), (F32, 4, 64, MAX_K + 16, F32)])
def test_matmul_refusals(moe, xdt, m, n, k, odt):
    lib = moe.load()
    assert lib.moe_channel_matmul(FAKE, xdt, None, FAKE, FAKE, m, n, k, FAKE, odt, FAKE, 1 << 40, None) == 1


def test_matmul_pointers(moe):
    lib = moe.load()

    def call(x=FAKE, xdt=I8, xs=FAKE, w=FAKE, ws=FAKE, m=4, out=FAKE, wk=None, n_wk=0, k=256):
        return lib.moe_channel_matmul(x, xdt, xs, w, ws, m, 64, k, out, F32, wk, n_wk, None)

    assert call(x=None) == 1 and call(x=ODD) == 1 and call(xs=None) == 1 and call(xs=BYTE) == 1
    assert call(w=None) == 1 and call(w=ODD) == 1 and call(ws=None) == 1 and call(ws=BYTE) == 1
    assert call(out=None) == 1 and call(out=ODD) == 1
    assert call(xdt=BF16) == 1                      # x_scale with rows that are not codes
    assert call(xdt=BF16, xs=None) == 1             # no workspace
    need = lib.moe_channel_matmul_workspace_bytes(BF16, 4, 256)
    assert need >= 4 * 256 + 4 * 4
    assert call(xdt=BF16, xs=None, wk=FAKE, n_wk=need - 1) == 3
    assert call(xdt=BF16, xs=None, wk=ODD, n_wk=need) == 1
    assert lib.moe_channel_matmul_workspace_bytes(I8, 4, 256) == 0
    assert lib.moe_channel_matmul_workspace_bytes(BF16, 4, MAX_K) > 0
    assert lib.moe_channel_matmul_workspace_bytes(BF16, 4, MAX_K + 16) == 0
    assert call(xdt=BF16, xs=None, wk=FAKE, n_wk=100, k=MAX_K) == 3
    assert call(x=None, xs=None, w=None, ws=None, m=0, out=None) == 0


def test_binding_checks_tensors(moe):
    """Mismatched tensors are refused before the library is called (CPU tensors never reach it)."""
    import torch
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 256), dtype=torch.int8), torch.zeros(4)
    w, ws, out = torch.zeros((64, 256), dtype=torch.int8), torch.zeros(64), torch.zeros((4, 64))
    bad = [lambda: moe.moe_quantize_tokens(x, q[:3], s), lambda: moe.moe_quantize_tokens(x, q, s[:2]),
           lambda: moe.moe_quantize_tokens(x.t(), q.t(), s), lambda: moe.moe_quantize_tokens(x.double(), q, s),
           lambda: moe.moe_quantize_tokens(x, q.view(torch.uint8), s), lambda: moe.moe_quantize_tokens(x, q, s.double()),
           lambda: moe.moe_quantize_tokens(x, q, s),  # not on the GPU
           lambda: moe.moe_channel_matmul(q, None, w, ws, out), lambda: moe.moe_channel_matmul(x, s, w, ws, out),
           lambda: moe.moe_channel_matmul(q, s, w[:, :128], ws, out), lambda: moe.moe_channel_matmul(q, s, w, ws[:4], out),
           lambda: moe.moe_channel_matmul(q, s, w.view(torch.uint8), ws, out),
           lambda: moe.moe_channel_matmul(q, s, w, ws, out[:, :32]), lambda: moe.moe_channel_matmul(q, s, w, ws, out.half()),
           lambda: moe.moe_channel_matmul(q, s.view(4, 1), w, ws, out), lambda: moe.moe_channel_matmul(q[0], s, w, ws, out)]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoeError) as e:
            f()
        assert e.value.status == 1, i


def test_reference_quantize_by_hand():
    x = np.zeros((4, 16))
    x[0, :4] = 254.0, 3.0, 5.0, -1.0  # scale 2: 1.5 and 2.5 go to 2, -0.5 to 0
    x[1, :2] = 1.0, 0.5               # 0.5 / fp32(1/127) lies below 63.5 or above it, as fp32(1/127) is rounded
    x[2, 0] = 2.0 ** -130
    q, s = R.quantize(x)
    assert s.tolist() == [2.0, float(np.float32(1.0) / np.float32(127.0)), 2.0 ** -120, 1.0]
    assert q[0, :4].tolist() == [127, 2, 2, 0] and q[2].tolist() == [0] * 16 and q[3].tolist() == [0] * 16
    assert q[1, 0] == 127 and q[1, 1] == (63 if float(s[1]) * 63.5 > 0.5 else 64)


def test_reference_interval_covers_perturbed_rows():
    """Quantised perturbations of rows stay within the bound; with a mistake planted in them (codes cut towards
    zero) they do not."""
    rng = np.random.default_rng(0)
    h = rng.standard_normal((40, 200)) * np.exp(rng.standard_normal((40, 1)))
    eh = np.abs(h) * 1e-4
    mid, far = R.quantize_interval(h, eh)
    for _ in range(20):
        v = (h + eh * rng.uniform(-1, 1, h.shape)).astype(np.float32).astype(np.float64)
        q, s = R.quantize(v)
        assert (np.abs(R.dequant(q, s) - mid) <= far + 1e-12).all()
        cut = np.trunc(v / s.astype(np.float64)[:, None])
        assert not (np.abs(R.dequant(cut, s) - mid) <= far + 1e-12).all()
