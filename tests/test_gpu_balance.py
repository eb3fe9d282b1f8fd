"""moe_balance and moe_route_backward on the GPU against their float64 definitions (balance_ref derives the bounds),
and the routing's forward and backward passes with an int8 layer together."""
import sys

import numpy as np
import pytest

import balance_ref as R

pytestmark = pytest.mark.gpu
KINDS = ("softmax", "sigmoid", "sqrt_softplus")


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


def batch(T, E, k, n_seq, seed, sigma=2.0, seqs=True):
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((T, E)) * sigma + rng.standard_normal(E)).astype(np.float32)
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    idx[rng.random((T, k)) < 0.02] = -1
    idx[rng.random((T, k)) < 0.01] = E
    off = mask = None
    if seqs:
        a, b = (0, T) if n_seq % 2 else (min(3, T), max(min(3, T), T - 4))
        off = np.sort(np.concatenate([[a, b], rng.integers(a, b + 1, n_seq - 1)])).astype(np.int32)
        mask = (rng.random(T) > 0.2).astype(np.uint8)
        if T > 40:
            mask[10:30] = 0
        dead = R.seq_index(T, off, mask) < 0
        l[dead] = np.where(rng.random((T, E)) < 0.5, np.nan, np.inf)[dead]  # padding holds anything
        idx[dead] = rng.integers(-2 ** 31, 2 ** 31, (T, k))[dead]
    return l, idx, off, mask, rng


def run_balance(dev, l, idx, kind, off, mask, n_seq):
    torch, moe = dev
    T, E = l.shape
    c = moe.make_config(T, 64, E, idx.shape[1], 64, n_shared=0, score=kind)
    up = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()
    counts = torch.full((n_seq + 1, E), -7, dtype=torch.int32, device="cuda")
    tokens = torch.full((n_seq + 1,), -7, dtype=torch.int32, device="cuda")
    prob, loss = torch.full((n_seq + 1, E), -7.0, device="cuda"), torch.full((n_seq + 1,), -7.0, device="cuda")
    ws = moe.balance_workspace(c, n_seq)
    ws.fill_(0xFF)  # the workspace needs no initialisation
    moe.moe_balance(c, up(l), up(idx), counts[:-1], tokens[:-1], prob[:-1], loss[:-1], ws, mask=up(mask), seq_offsets=up(off))
    torch.cuda.synchronize()
    for t in (counts, tokens, prob, loss):
        assert (t[-1] == -7).all()
    return [t[:-1].cpu().numpy() for t in (counts, tokens, prob, loss)]


def run_backward(dev, l, idx, kind, off, mask, scale=1.0, normalise=True, d_w=None, counts=None, tokens=None, d_loss=None):
    torch, moe = dev
    T, E = l.shape
    c = moe.make_config(T, 64, E, idx.shape[1], 64, n_shared=0, score=kind, route_scale=scale)
    up = lambda a, dt=None: None if a is None else torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()
    d = torch.full((T + 1, E), 9.0, device="cuda")
    moe.moe_route_backward(c, moe.make_groups(normalise=normalise), up(l), up(idx), d[:T], d_topk_w=up(d_w, np.float32),
                           counts=up(counts, np.int32), tokens=up(tokens, np.int32), d_loss=up(d_loss, np.float32),
                           mask=up(mask), seq_offsets=up(off))
    torch.cuda.synchronize()
    assert (d[T] == 9.0).all()
    return d[:T].double().cpu().numpy()


# tokens, experts, k, sequences: one of each, no multiples of 64 or 4, E at, below and above every layout's edge,
# more sequences than tokens, long batches
SIZES = [(1, 1, 1, 1), (1, 8, 2, 3), (3, 61, 5, 2), (16, 64, 8, 1), (17, 65, 32, 4), (37, 192, 8, 5), (70, 256, 8, 200),
         (129, 257, 6, 3), (300, 320, 8, 7), (1000, 40, 4, 6), (300, 1023, 8, 3), (500, 1024, 32, 2), (4100, 128, 6, 10),
         (9000, 60, 4, 12), (20000, 16, 2, 3)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,k,n_seq", SIZES)
def test_balance(dev, T, E, k, n_seq, kind):
    for seqs in (True, False):
        n = n_seq if seqs else 1
        l, idx, off, mask, _ = batch(T, E, k, n, T + E, seqs=seqs)
        say("balance", T, E, k, n, kind, seqs)
        counts, tokens, prob, loss = run_balance(dev, l, idx, kind, off, mask, n)
        rc, rt, rp, rl, rel = R.balance(l, idx, kind, off, mask, n)
        assert np.array_equal(counts, rc) and np.array_equal(tokens, rt)
        assert (np.abs(prob - rp) <= rel * rp).all()
        assert (np.abs(loss - rl) <= rel * rl).all()


# the last tokens of one workgroup and the first of two, one sequence's ranges joined by one workgroup and by several
EDGES = [(16, 300, 4), (17, 300, 4), (64, 100, 8), (65, 100, 8), (128, 200, 8), (5000, 200, 8), (8191, 130, 6), (8193, 130, 6),
         (20001, 260, 4)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,k", EDGES)
def test_balance_of_one_sequence(dev, T, E, k, kind):
    l, idx, off, mask, rng = batch(T, E, k, 1, T + E)
    say("one sequence", T, E, k, kind)
    for o, m in ((None, mask), (np.array([T // 3, T - T // 5], np.int32), mask), (np.array([T, T], np.int32), None)):
        counts, tokens, prob, loss = run_balance(dev, l, idx, kind, o, m, 1)
        rc, rt, rp, rl, rel = R.balance(l, idx, kind, o, m, 1)
        assert np.array_equal(counts, rc) and np.array_equal(tokens, rt)
        assert (np.abs(prob - rp) <= rel * rp).all()
        assert (np.abs(loss - rl) <= rel * rl).all()


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_rows_at_any_address(dev, shift):
    """Rows that begin 4, 8 and 12 bytes off a multiple of 16: the same bits."""
    torch, moe = dev
    T, E, k = 300, 128, 4
    l, idx, _, _, rng = batch(T, E, k, 1, 3, seqs=False)
    c = moe.make_config(T, 64, E, k, 64, n_shared=0, score="sigmoid")
    idx, d_w, d_loss = (torch.from_numpy(a).cuda() for a in (idx, rng.standard_normal((T, k)).astype(np.float32), np.ones(1, np.float32)))
    out = []
    for s in (0, shift):
        lg = torch.empty(T * E + s, device="cuda")[s:].view(T, E)
        lg.copy_(torch.from_numpy(l))
        counts = torch.empty(E + s, dtype=torch.int32, device="cuda")[s:].view(1, E)
        tokens, prob, loss = torch.empty(1, dtype=torch.int32, device="cuda"), torch.empty((1, E), device="cuda"), torch.empty(1, device="cuda")
        d = torch.empty(T * E + s, device="cuda")[s:].view(T, E)
        say("address", s)
        moe.moe_balance(c, lg, idx, counts, tokens, prob, loss, moe.balance_workspace(c, 1))
        moe.moe_route_backward(c, None, lg, idx, d, d_topk_w=d_w, counts=counts, tokens=tokens, d_loss=d_loss)
        torch.cuda.synchronize()
        out.append((counts, prob, loss, d))
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,E,k,n_seq", SIZES)
def test_backward(dev, T, E, k, n_seq, kind, normalise):
    for seqs in (True, False):
        n = n_seq if seqs else 1
        l, idx, off, mask, rng = batch(T, E, k, n, T + E + 1, seqs=seqs)
        if T > 5:
            idx[T // 2] = idx[T // 2][0]  # the same expert k times
        rc, rt, _, _, _ = R.balance(l, idx, kind, off, mask, n)
        d_w = rng.standard_normal((T, k)).astype(np.float32)
        d_w[R.seq_index(T, off, mask) < 0] = np.nan
        d_loss = rng.standard_normal(n).astype(np.float32)
        for use_w, use_loss in ((True, True), (True, False), (False, True)):
            say("backward", T, E, k, n, kind, normalise, use_w, use_loss)
            kw = dict(scale=1.5, normalise=normalise, d_w=d_w if use_w else None)
            if use_loss:
                kw.update(counts=rc, tokens=rt, d_loss=d_loss)
            got = run_backward(dev, l, idx, kind, off, mask, **kw)
            want, err = R.backward(l, idx, kind, off=off, mask=mask, **kw)
            assert (np.abs(got - want) <= err).all(), np.abs(got - want).max()


@pytest.mark.parametrize("kind", KINDS)
def test_extreme_logits(dev, kind):
    """Logits whose scores vanish, saturate or differ by the whole range; rows of -inf count with probability 0."""
    E, k = 12, 3
    l = np.zeros((8, E), np.float32)
    l[0], l[1], l[2] = -80.0, 80.0, -60.0
    l[2, 3] = 60.0
    l[3, :6], l[3, 6:] = 1e4, -1e4
    l[4] = np.linspace(-30, 30, E)
    l[5] = -np.inf
    l[6, 1:] = -np.inf
    l[7] = 1e-30
    idx = np.tile(np.array([[3, 0, 7]], np.int32), (8, 1))
    say("extreme", kind)
    # (the definition has no value for a row of -inf: it is left out there)
    rows = [i for i in range(8) if i != 5]
    with np.errstate(all="ignore"):
        rc, rt, rp, rl, _ = R.balance(l[rows], idx[rows], kind)
    counts, tokens, prob, loss = run_balance(dev, l, idx, kind, None, None, 1)
    assert tokens[0] == 8 and counts[0, 3] == 8
    # arguments of up to 120 in an exponential, 64 roundings: (2 * 120 + 64 + 20) U
    rel = (2 * 120 + 64 + 20) * R.U
    assert (np.abs(prob * 8 - rp * 7) <= rel * rp * 7 + 1e-37).all()
    d_w = np.ones((8, k), np.float32) * np.array([1.0, -2.0, 0.5], np.float32)
    for normalise in (True, False):
        got = run_backward(dev, l, idx, kind, None, None, 1.0, normalise, d_w, counts, tokens, np.ones(1, np.float32))
        assert np.isfinite(got).all() and (got[5] == 0).all()
        with np.errstate(all="ignore"):
            want, err = R.backward(l, idx, kind, 1.0, normalise, d_w, counts.astype(np.float64), tokens, np.ones(1),
                                   eps=(2 * 120 + 64) * R.U)
        for t in (1, 2, 3, 4, 7):
            assert (np.abs(got[t] - want[t]) <= err[t] + 1e-37).all(), (t, normalise)


def test_nan_reaches_its_sequence_only(dev):
    for E in (40, 256, 300):
        l, idx, _, _, rng = batch(50, E, 4, 1, 5, seqs=False)
        l[20, 3] = np.nan
        off = np.array([0, 10, 30, 50], np.int32)
        for kind in KINDS:
            say("nan", E, kind)
            counts, tokens, prob, loss = run_balance(dev, l, idx, kind, off, None, 3)
            assert np.isnan(loss).tolist() == [False, True, False]
            assert np.isnan(prob[1]).any() and np.isfinite(prob[[0, 2]]).all()
            d = run_backward(dev, l, idx, kind, off, None, counts=counts, tokens=tokens, d_loss=np.ones(3, np.float32))
            assert np.isnan(d[20]).any() and np.isfinite(np.delete(d, 20, 0)).all()


def test_no_sequences_with_tokens(dev):
    """Every token masked, or every sequence empty: counts, losses and gradients are zeros."""
    l, idx, _, _, rng = batch(40, 96, 4, 1, 5, seqs=False)
    for off, mask, n in ((None, np.zeros(40, np.uint8), 1), (np.array([7, 7, 7], np.int32), None, 2), (np.array([40, 40], np.int32), None, 1)):
        counts, tokens, prob, loss = run_balance(dev, l, idx, "softmax", off, mask, n)
        assert not counts.any() and not tokens.any() and not prob.any() and not loss.any()
        d = run_backward(dev, l, idx, "softmax", off, mask, d_w=np.full((40, 4), np.inf), counts=counts, tokens=tokens, d_loss=np.ones(n))
        assert not d.any()


@pytest.mark.parametrize("kind", KINDS)
def test_even_load_has_little_gradient(dev, kind):
    """With an even load the loss is 1 and its gradient 0, up to roundings, whatever the probabilities."""
    T, E = 64, 32
    rng = np.random.default_rng(0)
    l = rng.standard_normal((T, E)).astype(np.float32)
    idx = (np.arange(T)[:, None] * 2 + np.arange(2)).astype(np.int32) % E
    counts, tokens, prob, loss = run_balance(dev, l, idx, kind, None, None, 1)
    assert (counts == T * 2 // E).all() and abs(loss[0] - 1.0) <= (2 * 8 + 64 + 20) * R.U
    d = run_backward(dev, l, idx, kind, None, None, counts=counts, tokens=tokens, d_loss=np.ones(1))
    assert (d == 0).all()  # f - 1 is exactly 0


def test_long_offsets(dev):
    """More than 2^31 bytes of logits: the last tokens count, and their gradients are written."""
    torch, moe = dev
    T, E = 1 << 20, 1024
    l = torch.zeros((T, E), device="cuda")
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    l[T - 1, E - 1], idx[T - 1] = 50.0, E - 1
    off = torch.tensor([0, T - 1, T], dtype=torch.int32, device="cuda")
    c = moe.make_config(T, 64, E, 1, 64, n_shared=0, score="softmax")
    counts, tokens = torch.empty((2, E), dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    prob, loss = torch.empty((2, E), device="cuda"), torch.empty(2, device="cuda")
    say("long balance")
    moe.moe_balance(c, l, idx, counts, tokens, prob, loss, moe.balance_workspace(c, 2), seq_offsets=off)
    torch.cuda.synchronize()
    assert tokens.tolist() == [T - 1, 1] and counts[0, 0].item() == T - 1 and counts[1, E - 1].item() == 1
    assert torch.allclose(prob[0], torch.full((E,), 1.0 / E, device="cuda"), rtol=1e-4) and abs(loss[1].item() - E) < 1e-3
    d = torch.full((T, E), 9.0, device="cuda")
    say("long backward")
    moe.moe_route_backward(c, moe.make_groups(normalise=False), l, idx, d, d_topk_w=torch.ones((T, 1), device="cuda"), seq_offsets=off)
    torch.cuda.synchronize()
    p = 1.0 / E
    assert abs(d[T - 2, 0].item() - p * (1 - p)) < 1e-9 and abs(d[T - 2, 5].item() + p * p) < 1e-9
    assert abs(d[T - 1, E - 1].item()) < 1e-15 and d.abs().max().item() < 1e-3


def test_same_bits_streams_and_graph(dev):
    """The same call gives the same bits; on a side stream and from replayed graphs (two, with workspaces of their
    own) too, with other work and other inputs between the replays."""
    torch, moe = dev
    T, E, k, n = 3000, 256, 8, 5
    l0, idx, off, mask, rng = batch(T, E, k, n, 8)
    c = moe.make_config(T, 64, E, k, 64, n_shared=0, score="sigmoid", route_scale=2.5)
    up = lambda a: torch.from_numpy(a).cuda()
    idx, off, mask, dw, dl = up(idx), up(off), up(mask), up(rng.standard_normal((T, k)).astype(np.float32)), up(rng.standard_normal(n).astype(np.float32))

    def state():
        return dict(l=up(l0), counts=torch.empty((n, E), dtype=torch.int32, device="cuda"),
                    tokens=torch.empty(n, dtype=torch.int32, device="cuda"), prob=torch.empty((n, E), device="cuda"),
                    loss=torch.empty(n, device="cuda"), d=torch.empty((T, E), device="cuda"), ws=moe.balance_workspace(c, n))

    def both(s):
        moe.moe_balance(c, s["l"], idx, s["counts"], s["tokens"], s["prob"], s["loss"], s["ws"], mask=mask, seq_offsets=off)
        moe.moe_route_backward(c, None, s["l"], idx, s["d"], d_topk_w=dw, counts=s["counts"], tokens=s["tokens"], d_loss=dl,
                               mask=mask, seq_offsets=off)

    def same(a, b):
        torch.cuda.synchronize()
        return all(torch.equal(a[key], b[key]) for key in ("counts", "tokens", "prob", "loss", "d"))

    want, got = state(), state()
    both(want)
    for _ in range(5):
        both(got)
        assert same(got, want)
    side = torch.cuda.Stream()
    got = state()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(got)
    side.synchronize()
    assert same(got, want)
    sets = []
    for _ in range(2):
        s = state()
        both(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            both(s)
        sets.append((s, g))
    live = up(R.seq_index(T, off.cpu().numpy(), mask.cpu().numpy()) >= 0)
    for i in range(3):
        for s, g in sets:
            s["l"][live] = torch.randn((int(live.sum()), E), device="cuda")
            for key in ("counts", "tokens", "prob", "loss", "d"):
                s[key].zero_()
            g.replay()
        for s, g in sets:
            want["l"].copy_(s["l"])
            both(want)
            assert same(s, want), i


def test_long_sequence_again_streams_and_graph(dev):
    """A sequence whose ranges several workgroups join: the same bits from calls in a row over one workspace, from two
    streams at once with workspaces of their own, and from a graph replayed on new inputs."""
    torch, moe = dev
    T, E, k = 20000, 130, 6
    l0, idx, _, mask, rng = batch(T, E, k, 1, 9, seqs=False)
    c = moe.make_config(T, 64, E, k, 64, n_shared=0, score="softmax")
    idx = torch.from_numpy(idx).cuda()

    def state():
        return dict(l=torch.from_numpy(l0).cuda(), counts=torch.empty((1, E), dtype=torch.int32, device="cuda"),
                    tokens=torch.empty(1, dtype=torch.int32, device="cuda"), prob=torch.empty((1, E), device="cuda"),
                    loss=torch.empty(1, device="cuda"), ws=moe.balance_workspace(c, 1))

    def call(s):
        moe.moe_balance(c, s["l"], idx, s["counts"], s["tokens"], s["prob"], s["loss"], s["ws"])

    def same(a, b):
        torch.cuda.synchronize()
        return all(torch.equal(a[key], b[key]) for key in ("counts", "tokens", "prob", "loss"))

    want, got, other = state(), state(), state()
    call(want)
    say("in a row")
    for _ in range(5):
        got["loss"].fill_(-1.0)
        call(got)
        assert same(got, want)
    say("two streams")
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, s in zip(streams, (got, other)):
        s["loss"].fill_(-1.0)
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(3):
                call(s)
    torch.cuda.synchronize()
    assert same(got, want) and same(other, want)
    say("graph")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(got)
    for _ in range(3):
        got["l"].copy_(torch.randn((T, E), device="cuda"))
        want["l"].copy_(got["l"])
        got["loss"].fill_(-1.0)
        g.replay()
        call(want)
        assert same(got, want)


def test_run_together(dev):
    """A step of tuning a router over int8 experts: routing, load and balance loss, the layer over that selection, the
    gradient of the selected weights from the experts' outputs, of the logits, of the router's weights; against
    automatic differentiation of the same in float64, and the loss against differences along the gradient."""
    torch, moe = dev
    import test_gpu_i8 as I
    T, d, E, k, F = 60, 128, 16, 4, 64
    L = I.make_layer(T, d, E, k, F, seed=5)
    W = I.upload(L)
    x, Wm = L["x"].cuda(), moe.make_weights(W)
    c = moe.make_config(T, d, E, k, F, score="sigmoid", route_scale=1.5, act="bf16", w="i8ch")
    grp = moe.make_groups(4, 2, 2)
    lg, idx, w = torch.empty((T, E), device="cuda"), torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    moe.moe_route_grouped(c, grp, x, W["w_router"], W["bias"], lg, idx, w, None)
    off = torch.tensor([0, 25, 60], dtype=torch.int32, device="cuda")
    counts, tokens = torch.empty((2, E), dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    prob, loss = torch.empty((2, E), device="cuda"), torch.empty(2, device="cuda")
    moe.moe_balance(c, lg, idx, counts, tokens, prob, loss, moe.balance_workspace(c, 2), seq_offsets=off)
    ws = moe.workspace(c)
    o, perm, inv = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
    moe.moe_permute(c, idx, o, perm, inv, ws)
    assert torch.equal(counts.sum(0), o[1:] - o[:-1])
    slot, sh, y = torch.empty((T * k, d), device="cuda"), torch.empty((T, d), device="cuda"), torch.empty((T, d), device="cuda")
    ones = torch.ones((T, k), device="cuda")
    moe.moe_expert_ffn(c, x, Wm, o, perm, ones, slot, sh, ws)  # the experts' outputs themselves: weights of 1
    dy = torch.randn((T, d), device="cuda")
    d_w = (slot.view(T, k, d) * dy[:, None]).sum(2).contiguous()
    d_loss = torch.tensor([0.3, 0.7], device="cuda")
    d_lg = torch.empty((T, E), device="cuda")
    moe.moe_route_backward(c, grp, lg, idx, d_lg, d_topk_w=d_w, counts=counts, tokens=tokens, d_loss=d_loss, seq_offsets=off)
    d_router = d_lg.double().t() @ x.double()

    wr = W["w_router"].double().requires_grad_(True)

    def objective(wr):
        s = torch.sigmoid(x.double() @ wr.t())
        sel = torch.gather(s, 1, idx.long())
        wt = 1.5 * sel / sel.sum(1, keepdim=True)
        out = (wt[:, :, None] * slot.view(T, k, d).double()).sum(1)
        p = s / s.sum(1, keepdim=True)
        total = (out * dy.double()).sum()
        for q, (a, b) in enumerate(((0, 25), (25, 60))):
            f = counts[q].double() * E / (k * (b - a))
            total = total + d_loss[q].double() * (f * p[a:b].mean(0)).sum()
        return total

    torch.cuda.synchronize()
    want, = torch.autograd.grad(objective(wr), wr)
    # the logits are fp32 there, float64 here, and d_w is a sum of d fp32 products: 2^-18 covers both
    assert (d_router - want).abs().max().item() <= 2.0 ** -18 * want.abs().max().item()
    step = 1e-3 * want / want.norm()
    with torch.no_grad():
        diff = (objective(wr + step) - objective(wr - step)) / 2
    # (second-order differences: an error of the third derivative, about step^2 of the gradient)
    assert abs(diff.item() - (d_router * step).sum().item()) <= 1e-4 * abs(diff.item())
