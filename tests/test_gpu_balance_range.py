"""moe_balance and moe_route_backward where scores leave fp32's range or come near its end, against the float64
definitions.  balance_ref derives the bounds: its eps_p has nothing that grows with a sigmoid or sqrt(softplus) logit, so
they hold wherever a token's scores sum to 2^-126 and more.  A value below fp32's normal range is a multiple of 2^-149:
DENORMAL allows for the roundings to such multiples on the way of a gradient (the selected weights' part, its product with
the derivative, the sum with the balance part, the result: half of one each, and one for a rounded border)."""
import numpy as np
import pytest

import balance_ref as R
from test_gpu_balance import KINDS, dev, run_backward, run_balance, say  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu
DENORMAL = 3 * 2.0 ** -149


def rows_around(centres, E, k, width, seed):
    """One token around each centre, its k best experts in a shuffled order, a sequence of its own for each."""
    rng = np.random.default_rng(seed)
    T = len(centres)
    l = (np.asarray(centres)[:, None] + rng.uniform(-width, width, (T, E))).astype(np.float32)
    idx = rng.permuted(np.argsort(-l, axis=1)[:, :k], axis=1).astype(np.int32)
    return l, idx, np.arange(T + 1, dtype=np.int32), rng


@pytest.mark.parametrize("E,k", [(61, 5), (100, 32), (256, 8), (300, 4), (1024, 32)])
@pytest.mark.parametrize("kind", ["sigmoid", "sqrt_softplus"])
def test_low_scores(dev, kind, E, k):
    """Logits down to where a token's scores sum to 2^-126: probabilities, losses and gradients keep their digits."""
    lowest = (0.5 - 126 * np.log(2.0) - np.log(E)) * (1 if kind == "sigmoid" else 2)
    centres = np.concatenate([np.arange(lowest, -50.0, 3.0), np.linspace(-24.0, -16.0, 9), [0.0, 50.0, 86.0, 95.0, 104.0]])
    l, idx, off, rng = rows_around(centres, E, k, 2.0, E)
    T = len(centres)
    s, _ = R.score(l, kind)
    assert (s.sum(1) >= 2.0 ** -126).all()
    say("low scores", kind, E)
    counts, tokens, prob, loss = run_balance(dev, l, idx, kind, off, None, T)
    rc, rt, rp, rl, rel = R.balance(l, idx, kind, off, None, T)
    assert np.array_equal(counts, rc) and np.array_equal(tokens, rt)
    worst = (np.abs(prob - rp) / rp).max(1)
    assert (worst <= rel).all(), [(c, w / R.U) for c, w in zip(centres, worst) if w > rel]
    assert (np.abs(loss - rl) <= rel * rl).all()
    d_loss = rng.uniform(0.5, 2.0, T).astype(np.float32)
    d_w = (rng.standard_normal((T, k)) * 1e3).astype(np.float32)
    for use_w, use_loss in ((False, True), (True, False), (True, True)):
        kw = dict(scale=2.5, normalise=False, d_w=d_w if use_w else None)
        if use_loss:
            kw.update(counts=rc, tokens=rt, d_loss=d_loss)
        say("low scores, gradient", kind, E, use_w, use_loss)
        got = run_backward(dev, l, idx, kind, off, None, **kw)
        want, err = R.backward(l, idx, kind, off=off, **kw)
        bad = (np.abs(got - want) > err + DENORMAL).any(1)
        assert not bad.any(), centres[bad]


@pytest.mark.parametrize("kind", KINDS)
def test_gradients_of_saturated_rows(dev, kind):
    """Rows of -80 throughout, and of one finite logit beside -inf: the gradients of the definition."""
    E, k = 12, 3
    l = np.full((3, E), -80.0, np.float32)
    l[1, 1:], l[1, 0] = -np.inf, 0.0
    l[2, 1:], l[2, 0] = -1e4, 2.0
    idx = np.tile(np.array([[3, 0, 7]], np.int32), (3, 1))
    off = np.arange(4, dtype=np.int32)
    d_w = np.array([[1.0, -2.0, 0.5], [3.0, -1.0, 2.0], [0.5, 0.25, -4.0]], np.float32)
    counts, tokens = np.zeros((3, E), np.int64), np.ones(3, np.int64)
    counts[:, [3, 0, 7]] = 1
    for normalise in (True, False):
        kw = dict(scale=1.5, normalise=normalise, d_w=d_w, counts=counts, tokens=tokens, d_loss=np.ones(3))
        say("saturated", kind, normalise)
        got = run_backward(dev, l, idx, kind, off, None, **kw)
        with np.errstate(all="ignore"):
            want, err = R.backward(l, idx, kind, off=off, eps=64 * R.U, **kw)  # (no finite softmax exponent but 0)
        assert (np.abs(got - want) <= err + DENORMAL).all(), np.abs(got - want).max()


# A renormalised weight's gradient, (dw_j - sum dw w) w_j (log s)'(l_j), has no factor that leaves fp32's range: its bound
# is balance_ref's, whose terms are these (for softmax with the range of its logits, which an exponential's argument can
# reach).  The selection's own weights tell where it is no more: scores below 2^-150 are 0 in fp32, and weights and gradient
# with them.
@pytest.mark.parametrize("E,k", [(12, 2), (61, 5), (100, 32), (256, 8), (1024, 32)])
@pytest.mark.parametrize("kind,lowest", [("sigmoid", -99.0), ("sqrt_softplus", -203.0), ("softmax", -88.0)])
def test_renormalised_weights_of_small_scores(dev, kind, lowest, E, k):
    """Selected scores from ordinary ones down to fp32's smallest, large gradients of the weights."""
    centres = np.arange(lowest, 10.0, 2.5 if kind != "sqrt_softplus" else 5.0)
    T = len(centres)
    l, idx, off, rng = rows_around(centres, E, k, 3.0, E + 1)
    if kind == "softmax":
        top = np.setdiff1d(np.arange(E), idx[0])[0]  # not selected: the others' scores are small beside it
        l[:, top] = 0.0
        for t in range(T):
            sel = np.argsort(-np.where(np.arange(E) == top, -np.inf, l[t]))[:k]
            idx[t] = rng.permutation(sel)
    d_w = (rng.choice([-1.0, 1.0], (T, k)) * rng.uniform(10.0, 1e4, (T, k))).astype(np.float32)
    kw = dict(scale=2.5, normalise=True, d_w=d_w)
    say("renormalised", kind, E)
    got = run_backward(dev, l, idx, kind, off, None, **kw)
    want, err = R.backward(l, idx, kind, off=off, **kw)
    bad = ~(np.abs(got - want) <= err + DENORMAL).all(1)
    assert not bad.any(), (centres[bad], np.abs(got - want)[bad].max(1), np.abs(want)[bad].max(1))


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_ends_where_the_weights_do(dev, kind):
    """Tokens whose selected scores are all 0 in fp32 have weights of 0 (moe_select_grouped) and no gradient; just above,
    both are there."""
    torch, moe = dev
    E, k, T = 64, 4, 4
    half = 2.0 if kind == "sqrt_softplus" else 1.0
    l = np.full((T, E), -1e4, np.float32)
    l[:, :k] = half * np.array([[-103.0], [-103.5], [-104.5], [-120.0]]) + 0.25 * np.arange(k) * np.array([1, 1, -1, -1])[:, None]
    bias = np.zeros(E, np.float32)
    bias[:k] = 2.0  # selected whatever their scores
    if kind == "softmax":
        l[:, k] = 0.0
    c = moe.make_config(T, 64, E, k, 64, n_shared=0, score=kind)
    up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    idx, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    say("weights' end", kind)
    moe.moe_select_grouped(c, None, up(l), up(bias), idx, w)
    torch.cuda.synchronize()
    idx, w = idx.cpu().numpy(), w.cpu().numpy()
    assert sorted(idx[0].tolist()) == list(range(k))
    d_w = np.tile(np.array([[1.0, -2.0, 3.0, 50.0]], np.float32), (T, 1))
    got = run_backward(dev, l, idx, kind, None, None, d_w=d_w)
    assert np.isfinite(got).all()
    assert (w > 0).any(1).tolist() == [True, True, False, False] == (got != 0).any(1).tolist()
    # (a selection's fp32 scores there are one or two multiples of 2^-149; the gradient is the definition's)
    want, err = R.backward(l, idx, kind, d_w=d_w)
    assert (np.abs(got - want) <= err + DENORMAL)[:2].all()


def test_renormalised_weights_with_nan(dev):
    """A NaN among a token's selected logits reaches its gradient, for softmax one anywhere in the row; no other token's."""
    E, k = 61, 5
    for kind in KINDS:
        l, idx, off, rng = rows_around(np.array([0.0, -90.0, -90.0]), E, k, 2.0, 7)
        l[1, idx[1, 2] if kind != "softmax" else np.setdiff1d(np.arange(E), idx[1])[3]] = np.nan
        say("nan", kind)
        got = run_backward(dev, l, idx, kind, off, None, d_w=rng.standard_normal((3, k)))
        assert np.isnan(got[1]).any() and np.isfinite(got[[0, 2]]).all()


@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("kind,centre", [("sigmoid", -95.0), ("sqrt_softplus", -190.0), ("softmax", -20.0)])
def test_small_scores_listed_again(dev, kind, centre, normalise):
    """Experts listed several times, and entries that are none, among small scores."""
    for E, k in ((61, 7), (100, 32), (300, 9)):
        l, idx, off, rng = rows_around(np.full(6, centre), E, k, 3.0, E)
        if kind == "softmax":
            l[:, -1] = 60.0
        idx[0] = idx[0, 0]
        idx[1, 1:3] = idx[1, 0]
        idx[2, 2] = idx[2, k - 1]
        idx[3, :3] = -1, E, 2 ** 31 - 1
        idx[4] = -1
        kw = dict(scale=1.5, normalise=normalise, d_w=(rng.standard_normal((6, k)) * 100).astype(np.float32))
        say("listed again", kind, E, normalise)
        got = run_backward(dev, l, idx, kind, off, None, **kw)
        want, err = R.backward(l, idx, kind, off=off, **kw)
        # (a sum of up to k parts, each rounded to a multiple of 2^-149 where it is that small)
        assert (np.abs(got - want) <= err + DENORMAL + k * 2.0 ** -150).all(), np.abs(got - want).max()
