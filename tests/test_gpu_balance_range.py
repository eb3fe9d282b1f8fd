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


@pytest.mark.parametrize("E,k", [(61, 5), (256, 8), (300, 4), (1024, 32)])
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
