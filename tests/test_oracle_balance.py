"""Pins of the router-forward and balance-loss oracle: brute force, finite
differences and cases with known answers."""
import numpy as np
import pytest

from oracle import router as R


def test_topk_order_ties_closed_experts_and_masks():
    z = np.array([[1.0, 3.0, 3.0, -0.0, 0.0], [-np.inf, 2.0, -np.inf, np.nan, -np.inf],
                  [-np.inf] * 5, [5.0, 4.0, 3.0, 2.0, 1.0]])
    idx, is_open = R.topk(z, 4, mask=[1, 1, 1, 0])
    assert idx.tolist() == [[1, 2, 0, 3], [1, -1, -1, -1], [-1] * 4, [-1] * 4]
    assert is_open.sum(axis=1).tolist() == [4, 1, 0, 0]


@pytest.mark.parametrize("mode,renorm", [(0, False), (1, False), (1, True), (2, False)])
def test_forward_topk_scores(mode, renorm):
    rng = np.random.default_rng(1)
    z = rng.normal(size=(20, 9))
    z[3, :7] = -np.inf
    idx, scores, aff = R.forward_topk(mode, z, 4, renorm)
    p = np.exp(z) / np.exp(z).sum(axis=1, keepdims=True)
    for t in range(20):
        sel = idx[t][idx[t] >= 0]
        assert len(sel) == (2 if t == 3 else 4)
        ref = {0: np.exp(z[t, sel]) / np.exp(z[t, sel]).sum(), 1: p[t, sel], 2: z[t, sel]}[mode]
        if renorm:
            ref = p[t, sel] / p[t, sel].sum()
        assert np.allclose(scores[t, :len(sel)], ref, rtol=1e-12)
        assert np.allclose(aff[t, sel], ref, rtol=1e-12) and np.count_nonzero(aff[t]) <= len(sel)
    assert not scores[3, 2:].any()


def _problem(seed, T=23, E=6, K=3):
    rng = np.random.default_rng(seed)
    z = rng.normal(0, 1.5, (T, E))
    z[rng.random((T, E)) < 0.1] = -np.inf
    z[5] = -np.inf
    mask = rng.random(T) < 0.8
    idx, _ = R.topk(z, K, mask)
    idx[rng.random(idx.shape) < 0.1] = -1
    return z, idx, mask, [2, 9, 9, 16, T - 2]


def test_balance_gradient_matches_finite_differences():
    z, idx, mask, seq = _problem(3)
    dl = (0.7, -1.3)
    _, _, num, d = R.balance(z, idx, 0.5, 0.25, mask, seq, dl)
    assert num[4] == 3 and num[1] == 0 and num[5] == num[:4].sum()
    h = 1e-5
    for t in range(z.shape[0]):
        for e in range(z.shape[1]):
            if z[t, e] == -np.inf:
                assert d[t, e] == 0
                continue
            hi, lo = z.copy(), z.copy()
            hi[t, e] += h
            lo[t, e] -= h
            f = lambda x: np.dot(dl, R.balance(x, idx, 0.5, 0.25, mask, seq)[0])
            # central difference: h^2 times the third derivative (order 1), and 1e-16 / h of rounding
            assert abs((f(hi) - f(lo)) / (2 * h) - d[t, e]) < 1e-9


def test_balance_known_answers():
    # even routing, even probabilities: the coefficient itself
    z = np.zeros((8, 4))
    idx = np.array([[t % 4] for t in range(8)])
    loss, counts, num, d = R.balance(z, idx, 0.01, 0.001)
    assert np.isclose(loss[0], 0.01) and np.isclose(loss[1], 0.001 * np.log(4) ** 2)
    assert counts.tolist() == [[2, 2, 2, 2]] and num.tolist() == [8, 1, 8]
    # all tokens to one certain expert: E times it
    z[:, 0] = 1e3
    loss, _, _, _ = R.balance(z, np.zeros((8, 1), dtype=int), 0.01, 0.0)
    assert np.isclose(loss[0], 0.04)
    # nothing takes part
    loss, counts, num, d = R.balance(z, idx, 0.01, 0.1, mask=np.zeros(8))
    assert not loss.any() and not counts.any() and not num.any() and not d.any()
