"""Pins of the oracle's linear attention, gradients and beam selection (CPU)."""
import itertools

import numpy as np
import pytest

import oracle
from oracle import attention


def problem(T=11, H=4, G=2, N=3, P=5, nseq=1, seed=0):
    r = np.random.default_rng(seed)
    cuts = np.sort(r.integers(0, T + 1, nseq - 1)) if nseq > 1 else np.zeros(0, int)
    offs = np.concatenate([[0], cuts, [T]]).astype(int)
    return dict(q=r.standard_normal((T, G, N)), k=r.standard_normal((T, G, N)), v=r.standard_normal((T, H, P)),
                log_decay=-r.uniform(0, 1.5, (T, H)), scale=0.7, init=r.standard_normal((nseq, H, P, N)), offsets=offs)


def test_equals_the_ssd_recurrence():
    """With dt = 1 the SSD's decay is exp(A): constant decays, C = scale q, B = k, x = v."""
    p = problem(T=23, H=4, G=2)
    A = -np.array([0.1, 0.7, 1.3, 0.0001])
    y, fin = attention.forward(p["q"], p["k"], p["v"], A, p["scale"], p["init"])
    y2, fin2 = oracle.ssd_forward(p["v"], np.ones(p["v"].shape[:2]), A, p["k"], p["scale"] * p["q"], None, p["init"])
    np.testing.assert_allclose(y, y2, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(fin, fin2, rtol=1e-12, atol=1e-12)


def test_equals_the_dense_masked_product():
    p = problem(T=9, H=2, G=1)
    y, _ = attention.forward(p["q"], p["k"], p["v"], p["log_decay"], p["scale"])
    for h in range(2):
        M = np.zeros((9, 9))
        for i in range(9):
            for j in range(i + 1):
                M[i, j] = np.prod(np.exp(p["log_decay"][j + 1:i + 1, h])) * p["q"][i, 0] @ p["k"][j, 0] * p["scale"]
        np.testing.assert_allclose(y[:, h], M @ p["v"][:, h], rtol=1e-12, atol=1e-12)


def test_zero_decay_forgets():
    p = problem(T=6)
    p["log_decay"][3] = -np.inf
    y, fin = attention.forward(**p)
    q = {n: (v[3:] if n in ("q", "k", "v", "log_decay") else v) for n, v in p.items()}
    y2, fin2 = attention.forward(**{**q, "init": None, "offsets": [0, 3]})
    np.testing.assert_allclose(y[3:], y2, atol=1e-14)
    np.testing.assert_allclose(fin, fin2, atol=1e-14)


@pytest.mark.parametrize("constant", [False, True])
def test_gradients_against_differences(constant):
    p = problem(T=7, H=2, G=1, N=2, P=3, nseq=3, seed=4)
    if constant:
        p["log_decay"] = -np.array([0.3, 1.1])
    r = np.random.default_rng(5)
    dy, dfin = r.standard_normal(p["v"].shape), r.standard_normal(p["init"].shape)

    def loss(x):
        y, fin = attention.forward(**x)
        return float((y * dy).sum() + (fin * dfin).sum())

    got = dict(zip(("q", "k", "v", "log_decay", "init"),
                   attention.backward(dy, p["q"], p["k"], p["v"], p["log_decay"], p["scale"], p["init"], dfin, p["offsets"])))
    for name, g in got.items():
        for at in itertools.product(*map(range, p[name].shape)):
            hi, lo = ({**p, name: p[name].copy()} for _ in range(2))
            hi[name][at] += 1e-5
            lo[name][at] -= 1e-5
            # central differences: the third derivatives (of order 1 to 100 here) times 1e-10 / 6,
            # and rounding 1e-15 * |loss| / 1e-5
            assert abs((loss(hi) - loss(lo)) / 2e-5 - g[at]) < 1e-7, (name, at)


def test_dlog_decay_as_a_difference_of_sums():
    """What the library computes: sum over s >= t of q.dq - k.dk, and <dfinal, final>."""
    p = problem(T=12, H=3, G=3, seed=7)
    r = np.random.default_rng(8)
    dy, dfin = r.standard_normal(p["v"].shape), r.standard_normal(p["init"].shape)
    dq, dk, _, dl, _ = attention.backward(dy, p["q"], p["k"], p["v"], p["log_decay"], p["scale"], p["init"], dfin)
    _, fin = attention.forward(**p)
    d = (p["q"] * dq).sum(-1) - (p["k"] * dk).sum(-1)
    np.testing.assert_allclose(np.cumsum(d[::-1], axis=0)[::-1] + (dfin * fin).sum((-1, -2)), dl, rtol=1e-10, atol=1e-10)


def test_beam_select_hand_worked():
    # beam 0: uniform over 4; beam 1: token 2 certain
    logits = np.array([[0.0, 0.0, 0.0, 0.0], [-np.inf, -np.inf, 5.0, -np.inf]])
    s, w, p = attention.beam_select(logits, [-1.0, -1.0 - np.log(4.0)], count=6)
    np.testing.assert_allclose(s[:5], -1.0 - np.log(4.0), rtol=1e-15)
    assert w.tolist() == [0, 1, 2, 3, 2, 0] and p.tolist() == [0, 0, 0, 0, 1, 1]
    assert s[5] == -np.inf
    s, w, p = attention.beam_select(logits, [-1.0, -0.5], finished=[False, True], eos=1, count=2)
    assert w.tolist() == [1, 0] and p.tolist() == [1, 0] and s[0] == -0.5
    s, w, p = attention.beam_select(np.full((2, 3), np.nan), [0.0, 0.0], eos=2)
    assert (s == -np.inf).all() and w.tolist() == [2, 2] and p.tolist() == [0, 1]
