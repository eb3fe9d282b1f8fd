"""Refusals of the grouped selection and of the 8-bit operators, on the CPU
(every call fails its checks before the device is touched), and the float64
definitions the GPU tests compare with, against cases worked out by hand."""
import ctypes
import os

import numpy as np
import pytest

import f8_ref as R

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)
BYTE = ctypes.c_void_p((1 << 20) + 2)
F32, BF16, Q8, F8 = range(4)


@pytest.fixture(scope="module")
def moe():
    import sparse_moe_layer_02_amd as m
    if not os.path.exists(m.binding.LIB_PATH):
        from sparse_moe_layer_02_amd import build
        build.build()
    m.load()
    return m


def cfg(moe, **kw):
    base = dict(T=4, d=512, E=32, k=4, F=256, score="sigmoid", act="bf16", w="f8b128")
    base.update(kw)
    return moe.make_config(**base)


@pytest.mark.parametrize("groups", [(0, 1, 1, 1), (3, 1, 1, 1), (65, 1, 1, 1), (8, 0, 1, 1), (8, 9, 1, 1), (8, 4, 0, 1),
                                    (8, 4, 3, 1), (8, 4, 1, 2), (8, 4, 1, -1), (-8, 1, 1, 1), (16, 1, 1, 1)])
def test_groups_refused(moe, groups):
    """(the last: two experts stay for top-4)"""
    lib = moe.load()
    c, g = ctypes.byref(cfg(moe)), ctypes.byref(moe.moe_groups(*groups))
    assert lib.moe_select_grouped(c, g, FAKE, None, FAKE, FAKE, None) == 1
    assert lib.moe_route_grouped(c, g, FAKE, FAKE, None, FAKE, FAKE, FAKE, None, 0, None) == 1
    m = moe.binding.moe_mat(FAKE.value, FAKE.value)
    w = moe.binding.moe_weights(FAKE.value, None, m, m, m, m, m, m)
    assert lib.moe_layer_forward_grouped(c, g, FAKE, ctypes.byref(w), FAKE, F32, None, FAKE, 1 << 40, None) == 1


def test_grouped_layer_refusals(moe):
    lib = moe.load()
    m = moe.binding.moe_mat(FAKE.value, FAKE.value)
    w = moe.binding.moe_weights(FAKE.value, None, m, m, m, m, m, m)
    W = ctypes.byref(w)

    def call(c, y_dtype=F32, y=FAKE, ws_bytes=1 << 40, W=W):
        return lib.moe_layer_forward_grouped(ctypes.byref(c), None, FAKE, W, y, y_dtype, None, FAKE, ws_bytes, None)

    assert call(cfg(moe), y_dtype=F8) == 1
    assert call(cfg(moe), y_dtype=9) == 1
    assert call(cfg(moe), y=ODD) == 1
    assert call(cfg(moe, w="bf16"), y_dtype=BF16) == 2  # bf16 y goes with e4m3 weights
    assert call(cfg(moe), ws_bytes=1000) == 3
    assert call(cfg(moe, act="f32")) == 2
    assert call(cfg(moe, d=480)) == 2
    noscale = moe.binding.moe_mat(FAKE.value, None)
    bad = moe.binding.moe_weights(FAKE.value, None, noscale, m, m, m, m, m)
    assert call(cfg(moe), W=ctypes.byref(bad)) == 1
    askew = moe.binding.moe_mat(FAKE.value, BYTE.value)
    bad = moe.binding.moe_weights(FAKE.value, None, m, askew, m, m, m, m)
    assert call(cfg(moe), W=ctypes.byref(bad)) == 1


def test_f8_layer_row_limit(moe):
    """e4m3 layers address the quantised rows with 32 bits: n_tokens * d_model < 2^32."""
    lib = moe.load()
    m = moe.binding.moe_mat(FAKE.value, FAKE.value)
    w = moe.binding.moe_weights(FAKE.value, None, m, m, m, m, m, m)

    def call(**kw):
        return lib.moe_layer_forward_grouped(ctypes.byref(cfg(moe, **kw)), None, FAKE, ctypes.byref(w), FAKE, F32, None,
                                             FAKE, 1000, None)

    assert call(T=4096, d=1 << 20) == 2
    assert call(T=4095, d=1 << 20) == 3  # (the limit is passed: only the workspace is too small)
    assert call(T=4096, d=1 << 20, w="bf16") == 3


def test_f8_prefetch_arguments(moe):
    """Of e4m3 experts only the codes are fetched: a scale array may start at any 4-byte address."""
    lib = moe.load()
    m = moe.binding.moe_mat(FAKE.value, FAKE.value + 4)
    w = moe.binding.moe_weights(FAKE.value, None, m, m, m, m, m, m)
    call = lambda c, w, ids, n: lib.moe_prefetch_experts(ctypes.byref(c), ctypes.byref(w), ids, n, 7, 0, 4, None, None)
    assert call(cfg(moe), w, None, 0) == 0
    assert call(cfg(moe), w, None, 4) == 1
    noscale = moe.binding.moe_mat(FAKE.value, None)
    assert call(cfg(moe), moe.binding.moe_weights(FAKE.value, None, m, m, noscale, m, m, m), None, 0) == 1


def test_f8_workspace_monotone(moe):
    lib = moe.load()
    base = dict(T=64, d=512, E=32, k=4, F=256, Fs=256)
    for key, sizes in (("T", (1, 8, 9, 31, 64, 65, 160, 1000)), ("d", (512, 576, 640)), ("E", (32, 33, 64, 300)),
                       ("k", (4, 5, 8)), ("F", (256, 320, 384)), ("Fs", (256, 320, 512))):
        got = [lib.moe_workspace_bytes(ctypes.byref(cfg(moe, **dict(base, **{key: v})))) for v in sizes]
        assert got == sorted(got) and got[0] > 0, (key, got)


@pytest.mark.parametrize("dt,rows,cols,ld", [(Q8, 4, 128, 128), (F8, 4, 128, 128), (-1, 4, 128, 128), (F32, -1, 128, 128),
                                             (F32, 4, 0, 128), (F32, 4, 120, 128), (BF16, 4, 129, 136),
                                             (F32, 4, (1 << 20) + 16, 1 << 21), (F32, 4, 128, 112), (F32, 4, 128, 130),
                                             (BF16, 4, 128, 132), (F32, 4, 128, 1 << 62)])
def test_quantize_refusals(moe, dt, rows, cols, ld):
    assert moe.load().moe_quantize_rows(FAKE, dt, rows, cols, ld, FAKE, FAKE, None) == 1


def test_quantize_pointers(moe):
    q = moe.load().moe_quantize_rows
    assert q(None, F32, 4, 128, 128, FAKE, FAKE, None) == 1
    assert q(ODD, F32, 4, 128, 128, FAKE, FAKE, None) == 1
    assert q(FAKE, F32, 4, 128, 128, ODD, FAKE, None) == 1
    assert q(FAKE, F32, 4, 128, 128, FAKE, BYTE, None) == 1
    assert q(FAKE, F32, 4, 128, 128, FAKE, None, None) == 1
    assert q(None, F32, 0, 128, 128, None, None, None) == 0  # no rows: nothing to do


@pytest.mark.parametrize("xdt,m,n,k,odt", [(Q8, 4, 64, 128, F32), (F32, 4, 64, 128, F8), (F32, -1, 64, 128, F32),
                                           (F32, (1 << 20) + 1, 64, 128, F32), (F32, 4, 0, 128, F32),
                                           (F32, 4, (1 << 20) + 1, 128, F32), (F32, 4, 64, 8, F32),
                                           (F32, 4, 64, 136, F32), (F32, 4, 64, (1 << 20) + 16, F32)])
def test_matmul_refusals(moe, xdt, m, n, k, odt):
    lib = moe.load()
    assert lib.moe_block_matmul(FAKE, xdt, None, FAKE, FAKE, m, n, k, FAKE, odt, FAKE, 1 << 40, None) == 1


def test_matmul_pointers(moe):
    lib = moe.load()

    def call(x=FAKE, xdt=F8, xs=FAKE, w=FAKE, ws=FAKE, m=4, out=FAKE, wk=None, n_wk=0):
        return lib.moe_block_matmul(x, xdt, xs, w, ws, m, 64, 256, out, F32, wk, n_wk, None)

    assert call(x=None) == 1 and call(x=ODD) == 1 and call(xs=None) == 1 and call(xs=BYTE) == 1
    assert call(w=None) == 1 and call(w=ODD) == 1 and call(ws=None) == 1 and call(ws=BYTE) == 1
    assert call(out=None) == 1 and call(out=ODD) == 1
    assert call(xdt=BF16) == 1                      # x_scale with rows that are not codes
    assert call(xdt=BF16, xs=None) == 1             # no workspace
    need = lib.moe_block_matmul_workspace_bytes(BF16, 4, 256)
    assert need >= 4 * 256 + 4 * 4
    assert call(xdt=BF16, xs=None, wk=FAKE, n_wk=need - 1) == 3
    assert call(xdt=BF16, xs=None, wk=ODD, n_wk=need) == 1
    assert lib.moe_block_matmul_workspace_bytes(F8, 4, 256) == 0
    assert call(x=None, xs=None, w=None, ws=None, m=0, out=None) == 0


def test_binding_checks_tensors(moe):
    """Mismatched tensors are refused before the library is called (CPU tensors never reach it)."""
    import torch
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((4, 4), dtype=torch.uint8)
    w, ws, out = torch.zeros((64, 256), dtype=torch.uint8), torch.zeros((1, 2)), torch.zeros((4, 64))
    bad = [lambda: moe.moe_quantize_rows(x, q[:3], s), lambda: moe.moe_quantize_rows(x, q, s[:, :2]),
           lambda: moe.moe_quantize_rows(x.t(), q.t(), s), lambda: moe.moe_quantize_rows(x.double(), q, s),
           lambda: moe.moe_quantize_rows(x, q, s),  # not on the GPU
           lambda: moe.moe_block_matmul(q, None, w, ws, out), lambda: moe.moe_block_matmul(x, s, w, ws, out),
           lambda: moe.moe_block_matmul(q, s, w[:, :128], ws, out), lambda: moe.moe_block_matmul(q, s, w, ws[:, :1], out),
           lambda: moe.moe_block_matmul(q, s, w, ws, out[:, :32]), lambda: moe.moe_block_matmul(q, s, w, ws.double(), out),
           lambda: moe.moe_block_matmul(q, s, w, ws, out.half())]
    c = cfg(moe)
    idx, wt, lg = torch.zeros((4, 4), dtype=torch.int32), torch.zeros((4, 4)), torch.zeros((4, 32))
    bad += [lambda: moe.moe_select_grouped(c, None, lg[:, :16], None, idx, wt),
            lambda: moe.moe_select_grouped(c, None, lg, torch.zeros(31), idx, wt),
            lambda: moe.moe_select_grouped(c, None, lg, None, idx[:2], wt),
            lambda: moe.moe_select_grouped(c, None, lg, None, idx.long(), wt),
            lambda: moe.moe_route_grouped(c, None, x, torch.zeros((32, 512)), None, lg, idx, wt, None),
            lambda: moe.moe_layer_forward_grouped(c, None, x, moe.binding.moe_weights(), x, None)]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoeError) as e:
            f()
        assert e.value.status == 1, i


def test_reference_quantize_by_hand():
    x = np.zeros((1, 256))
    x[0, 0], x[0, 1], x[0, 2] = 448.0, 17.0, 19.0  # ties to even on the grid of step 2: 16, 20
    x[0, 128], x[0, 129] = 449.0, 1.0
    q, s = R.quantize(x)
    assert s.tolist() == [[1.0, 2.0]]
    assert q[0, :3].tolist() == [448.0, 16.0, 20.0]
    assert q[0, 128] == 224.0 and q[0, 129] == 0.5
    assert R.e4m3_decode(np.array([0x7E, 0x01, 0x80, 0x38], np.uint8)).tolist() == [448.0, 2.0 ** -9, 0.0, 1.0]
    assert np.isnan(R.e4m3_decode(np.array([0x7F, 0xFF], np.uint8))).all()


def test_reference_select_by_hand():
    l = np.array([[0.0, 3.0, 2.0, 2.0, 2.5, -1.0, 1.0, 1.0]], np.float32)
    idx, w = R.select(l, None, 2, "sigmoid", 1.0, n_group=4, topk_group=1, group_top=2)
    assert idx.tolist() == [[2, 3]] and w.tolist() == [[0.5, 0.5]]  # group 1 has the best pair, not the best key
    idx, _ = R.select(l, None, 2, "sigmoid", 1.0, n_group=4, topk_group=2, group_top=1)
    assert idx.tolist() == [[1, 4]]
    _, w = R.select(l, None, 2, "softmax", 2.0, normalise=False)
    e = np.exp(l[0].astype(np.float64) - 3.0)
    assert np.allclose(w, 2.0 * np.array([[e[1], e[4]]]) / e.sum(), rtol=1e-6)
