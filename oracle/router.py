"""Router backward oracle -- TEST INFRASTRUCTURE ONLY.

Plain numpy in fp64.  Only the test suite, ``__graft_entry__.smoke()`` and the
``cpu_baseline`` leg of ``bench.py`` may import it; the GPU library never does.

What it follows: page 3 (sonic-moe, functional/backward.py), the router
backward that consumes the affinity gradient d(a): its softmax-over-top-k,
top-k-over-softmax (with or without renormalisation of the selected
probabilities) and plain top-k scatter kernels.  The pages give those kernels'
closed forms; here each mode is written as the forward map from the router
logits to the K scores of a token and the vector-Jacobian product of that map,
built from the softmax Jacobian diag(p) - p p^T, so that the tests can pin it by
finite differences of the forward.

Shapes (one row per token): logits [T, E], idx [T, K] int (distinct expert ids
in [0, E)), scores [T, K], g = d(score) [T, K]; the result d(logits) is [T, E].
Positions a mode gives no gradient are 0.
"""
from __future__ import annotations

import numpy as np

SOFTMAX_OVER_TOPK = 0   # scores = softmax over the K selected logits
TOPK_OVER_SOFTMAX = 1   # scores = the K selected entries of softmax over all E logits
TOPK = 2                # scores = the K selected logits themselves


def _softmax(z: np.ndarray) -> np.ndarray:
    z = np.asarray(z, dtype=np.float64)
    e = np.exp(z - z.max(axis=-1, keepdims=True))
    return e / e.sum(axis=-1, keepdims=True)


def forward(mode: int, logits: np.ndarray, idx: np.ndarray, renorm: bool = False) -> np.ndarray:
    """Scores [T, K] of each token for router mode `mode` (fp64)."""
    z = np.asarray(logits, dtype=np.float64)
    idx = np.asarray(idx, dtype=np.int64)
    sel = np.take_along_axis(z, idx, axis=1)
    if mode == SOFTMAX_OVER_TOPK:
        return _softmax(sel)
    if mode == TOPK_OVER_SOFTMAX:
        ps = np.take_along_axis(_softmax(z), idx, axis=1)
        return ps / ps.sum(axis=1, keepdims=True) if renorm else ps
    if mode == TOPK:
        return sel
    raise ValueError(f"unknown router mode {mode}")


def backward(mode: int, logits: np.ndarray, idx: np.ndarray, g: np.ndarray, renorm: bool = False,
             scores: np.ndarray | None = None) -> np.ndarray:
    """d(logits) [T, E] for upstream score gradients g [T, K] (fp64).

    SOFTMAX_OVER_TOPK: with y = softmax(logits[idx]) (or the given forward
      scores), the selected positions get J_y g = y * (g - <g, y>) (J_y is the
      symmetric softmax Jacobian); all other positions get 0.
    TOPK_OVER_SOFTMAX: p = softmax(logits) over all E.  Without renorm the
      scores are p[idx], so d(p) is g scattered to idx; with renorm they are
      p[idx] / S, S = sum p[idx], so d(p)[idx] = (g - <g, scores>) / S.  Then
      d(logits) = J_p d(p) = p * (d(p) - <d(p), p>) over every position.
    TOPK: g scattered to the selected positions.
    """
    z = np.asarray(logits, dtype=np.float64)
    idx = np.asarray(idx, dtype=np.int64)
    g = np.asarray(g, dtype=np.float64)
    T, E = z.shape
    out = np.zeros((T, E), dtype=np.float64)
    rows = np.arange(T)[:, None]
    if mode == SOFTMAX_OVER_TOPK:
        y = forward(mode, z, idx) if scores is None else np.asarray(scores, dtype=np.float64)
        out[rows, idx] = y * (g - (g * y).sum(axis=1, keepdims=True))
        return out
    if mode == TOPK_OVER_SOFTMAX:
        p = _softmax(z)
        dp = np.zeros((T, E), dtype=np.float64)
        if renorm:
            s = forward(mode, z, idx, True) if scores is None else np.asarray(scores, dtype=np.float64)
            S = np.take_along_axis(p, idx, axis=1).sum(axis=1, keepdims=True)
            dp[rows, idx] = (g - (g * s).sum(axis=1, keepdims=True)) / S
        else:
            dp[rows, idx] = g
        return p * (dp - (dp * p).sum(axis=1, keepdims=True))
    if mode == TOPK:
        out[rows, idx] = g
        return out
    raise ValueError(f"unknown router mode {mode}")


def backward_jacobian(mode: int, logits: np.ndarray, idx: np.ndarray, g: np.ndarray,
                      renorm: bool = False) -> np.ndarray:
    """The same product formed from explicit per-token Jacobians (small E):
    d(logits)_t = J_t^T g_t with J_t[k, j] = d score_k / d logit_j, built entry
    by entry from d p_i / d z_j = p_i (delta_ij - p_j)."""
    z = np.asarray(logits, dtype=np.float64)
    idx = np.asarray(idx, dtype=np.int64)
    g = np.asarray(g, dtype=np.float64)
    T, E = z.shape
    K = idx.shape[1]
    out = np.zeros((T, E), dtype=np.float64)
    for t in range(T):
        J = np.zeros((K, E))
        if mode == SOFTMAX_OVER_TOPK:
            y = _softmax(z[t, idx[t]])
            for k in range(K):
                for m in range(K):
                    J[k, idx[t, m]] = y[k] * ((1.0 if k == m else 0.0) - y[m])
        elif mode == TOPK_OVER_SOFTMAX:
            p = _softmax(z[t])
            dp = np.array([[p[i] * ((1.0 if i == j else 0.0) - p[j]) for j in range(E)] for i in range(E)])
            if renorm:
                S = p[idx[t]].sum()
                for k in range(K):
                    for i in idx[t]:
                        # d (p_ik / S) / d p_i
                        dsi = ((1.0 if i == idx[t, k] else 0.0) / S) - p[idx[t, k]] / S ** 2
                        J[k] += dsi * dp[i]
            else:
                for k in range(K):
                    J[k] = dp[idx[t, k]]
        elif mode == TOPK:
            for k in range(K):
                J[k, idx[t, k]] = 1.0
        else:
            raise ValueError(f"unknown router mode {mode}")
        out[t] = J.T @ g[t]
    return out


def gather_scores(daff: np.ndarray, idx: np.ndarray) -> np.ndarray:
    """g [T, K] from an affinity gradient laid out [T, E] (the masked layout of
    the affinities, index t*E + e): g[t, k] = daff[t, idx[t, k]]."""
    return np.take_along_axis(np.asarray(daff, dtype=np.float64), np.asarray(idx, dtype=np.int64), axis=1)


def topk(logits: np.ndarray, K: int, mask: np.ndarray | None = None):
    """Top-k selection of each token: (idx [T, K], open [T, K] bool).

    Descending logit, equal logits by ascending expert; an expert at -inf or
    NaN is closed.  Selections that find no open expert (all of them for a
    token whose mask is 0) hold id -1 and open False."""
    z = np.array(logits, dtype=np.float64)
    z[np.isnan(z)] = -np.inf
    if mask is not None:
        z[~np.asarray(mask, dtype=bool)] = -np.inf
    idx = np.argsort(-z, axis=1, kind="stable")[:, :K]
    is_open = np.take_along_axis(z, idx, axis=1) > -np.inf
    return np.where(is_open, idx, -1).astype(np.int32), is_open


def forward_topk(mode: int, logits: np.ndarray, K: int, renorm: bool = False, mask: np.ndarray | None = None):
    """(idx [T, K], scores [T, K], affinities [T, E]) of the whole router
    forward, token by token; closed selections score 0."""
    z = np.asarray(logits, dtype=np.float64)
    T, E = z.shape
    idx, is_open = topk(z, K, mask)
    scores, aff = np.zeros((T, K)), np.zeros((T, E))
    for t in range(T):
        n = int(is_open[t].sum())
        if n:
            scores[t, :n] = forward(mode, z[t:t + 1], idx[t:t + 1, :n], renorm)[0]
            aff[t, idx[t, :n]] = scores[t, :n]
    return idx, scores, aff


def balance(logits, idx, balance_coef, z_coef, mask=None, seq_starts=None, dloss=(1.0, 1.0)):
    """The load-balance and z losses: (loss [2], counts [S, E], num [S+2], d(logits) [T, E]).

    Sequence by sequence: f_e = c_e / (K n) the share of the selections, P_e the
    mean softmax probability, balance = coef E <f, P> averaged over the
    sequences with tokens; z = coef mean(lse^2) over all tokens that take part
    (in a sequence, mask not 0, some logit above -inf).  The gradient is the
    softmax Jacobian's product with the constant f, and of lse^2."""
    z = np.asarray(logits, dtype=np.float64)
    T, E = z.shape
    K = np.asarray(idx).shape[1]
    bounds = [0, T] if seq_starts is None else list(seq_starts)
    S = len(bounds) - 1
    counts, num = np.zeros((S, E), dtype=np.int64), np.zeros(S + 2, dtype=np.int64)
    rows = []
    for s in range(S):
        rows.append([t for t in range(bounds[s], bounds[s + 1])
                     if (mask is None or mask[t]) and np.any(z[t] > -np.inf)])
        num[s] = len(rows[s])
        for t in rows[s]:
            for e in np.asarray(idx)[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
    num[S], num[S + 1] = np.count_nonzero(num[:S]), num[:S].sum()
    loss, d = np.zeros(2), np.zeros((T, E))
    for s in range(S):
        if not rows[s]:
            continue
        x = z[rows[s]]
        m = x.max(axis=1, keepdims=True)
        p = np.exp(x - m)
        lse = m[:, 0] + np.log(p.sum(axis=1))
        p /= p.sum(axis=1, keepdims=True)
        f = counts[s] / (K * num[s])
        loss[0] += balance_coef * E * (f * p.mean(axis=0)).sum() / num[S]
        loss[1] += z_coef * (lse ** 2).sum() / num[S + 1]
        g = dloss[0] * balance_coef * E * f / (num[S] * num[s])
        d[rows[s]] = p * (g - (p * g).sum(axis=1, keepdims=True)) + \
            dloss[1] * z_coef * 2 / num[S + 1] * lse[:, None] * p
    return loss, counts, num, d
