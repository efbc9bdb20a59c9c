"""moe_balance_loss and moe_balance_loss_bwd on the GPU against the fp64 oracle.

Counts are exact.  A probability is within REL = 2e-5 of its value (fp32; the
bound of the router forward's tests: the exponent's argument rounds by 2^-24
|z - m|, the sum adds at most 70 * 2^-24).  The balance loss is a sum of
probabilities with positive weights, so it keeps that relative bound.  lse =
m + log(sum) is off by at most dl = 2^-23 (|m| + 16) + REL.  A gradient entry
p (w - <w, p> + c lse) has errors of at most p (3 REL (W + |c lse|) + c dl)
with W the largest w: w itself rounds a few times in fp32, <w, p> <= W is a
mean of w with weights off by REL."""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_amd as mx
from oracle import router as R

pytestmark = pytest.mark.gpu
REL = 2e-5


def _problem(T, E, K, S, dtype, seed, masked=0.2, closed=0.1, dropped=0.1):
    rng = np.random.default_rng(seed)
    z = rng.normal(0, 2, (T, E)).astype(np.float32)
    if closed:
        z[rng.random((T, E)) < closed] = -np.inf
    z = torch.from_numpy(z).to(dtype)
    if closed and T > 4:
        z[T // 2] = -torch.inf
    mask = torch.from_numpy(rng.random(T) >= masked) if masked else None
    idx, _ = R.topk(z.double().numpy(), K, None if mask is None else mask.numpy())
    if dropped:
        idx[rng.random(idx.shape) < dropped] = -1
        idx[rng.random(idx.shape) < 0.02] = E   # out of range: counts nowhere
    if mask is not None:
        idx[~mask.numpy()] = 0                  # a masked token's ids are not counted
        z[~mask] = torch.nan
    seq = None
    if S > 1:
        seq = np.sort(rng.integers(0, T + 1, S + 1)).astype(np.int32)
    return z, idx, mask, seq


def _dev(x):
    return None if x is None else torch.as_tensor(x).cuda()


def _check(z, idx, mask, seq, coefs, dloss, got, d):
    bal, zc = coefs
    T, E = z.shape
    x = z.double().numpy().copy()
    if mask is not None:
        x[~mask.numpy()] = 0
    ref, counts, num, rd = R.balance(x, idx, bal, zc, None if mask is None else mask.numpy(), seq,
                                     (1.0, 1.0) if dloss is None else tuple(dloss.tolist()))
    loss, c, n = (v.cpu().numpy() for v in got)
    assert np.array_equal(c, counts) and np.array_equal(n, num)
    assert abs(loss[0] - ref[0]) <= REL * abs(ref[0])
    fin = np.where(np.isfinite(x), x, 0)
    m = np.abs(fin).max(initial=0)
    dl = 2.0 ** -23 * (m + 16) + REL
    big = m + np.log(E)   # the largest |lse|
    assert abs(loss[1] - ref[1]) <= abs(zc) * (2 * big * dl + dl * dl) + REL * abs(ref[1])
    if d is None:
        return rd
    with np.errstate(invalid="ignore"):
        some = np.isfinite(x).any(1, keepdims=True)
        e = np.where(some, np.exp(x - np.where(some, x.max(1, keepdims=True), 0)), 0)
    p = e / np.maximum(e.sum(1, keepdims=True), 1)
    S = counts.shape[0]
    bounds = [0, T] if seq is None else seq
    W = np.zeros((T, 1))
    for s in range(S):
        if num[s]:
            W[bounds[s]:bounds[s + 1]] = abs(bal) * E * counts[s].max() / (num[S] * idx.shape[1] * num[s] ** 2)
    g = np.abs(np.ones(2) if dloss is None else dloss.double().numpy())
    cz = 2 * abs(zc) / max(num[S + 1], 1)
    tol = p * (3 * REL * (g[0] * W + g[1] * cz * big) + g[1] * cz * dl) + 1e-37
    assert np.all(np.abs(d.cpu().numpy() - rd) <= tol)
    return rd


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K,S", [(1, 1, 1, 1), (1, 8, 2, 1), (5, 3, 2, 3), (1000, 8, 2, 1), (257, 16, 4, 9),
                                     (777, 60, 6, 5), (333, 64, 6, 40), (2000, 128, 8, 17), (600, 200, 8, 4),
                                     (130, 300, 32, 1), (90, 513, 8, 6), (40, 1025, 5, 3), (17, 2049, 3, 2),
                                     (33, 4096, 8, 4), (5000, 4, 1, 2), (3000, 24, 3, 300)])
def test_matches_oracle(dtype, T, E, K, S):
    z, idx, mask, seq = _problem(T, E, K, S, dtype, T + E + S)
    print(f"{dtype} T {T} E {E} K {K} S {S}", flush=True)
    coefs, dloss = (0.02, 0.003), torch.tensor([0.7, -1.6])
    args = _dev(z), _dev(idx)
    kw = dict(token_mask=_dev(mask), seq_starts=_dev(seq))
    got = mx.moe_balance_loss(*args, *coefs, **kw)
    d = mx.moe_balance_loss_bwd(args[0], got[1], got[2], K, *coefs, dloss=_dev(dloss), **kw)
    _check(z, idx, mask, seq, coefs, dloss, got, d)
    # the same bits on a second run
    again = mx.moe_balance_loss(*args, *coefs, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    # accumulation: the prior plus the gradient, rows that take no part as they were
    prior = torch.randn(T, E, device="cuda")
    out = prior.clone()
    r = mx.moe_balance_loss_bwd(args[0], got[1], got[2], K, *coefs, dloss=_dev(dloss), out=out, accumulate=True, **kw)
    assert r is out and torch.equal(out, prior + d)


@pytest.mark.parametrize("T,E,K", [(32768, 128, 8), (16384, 8, 2)])
def test_workload_sizes(T, E, K):
    z, idx, mask, seq = _problem(T, E, K, 1, torch.float32, 3, masked=0, closed=0, dropped=0)
    got = mx.moe_balance_loss(_dev(z), _dev(idx), 0.01, 0.001)
    d = mx.moe_balance_loss_bwd(_dev(z), got[1], got[2], K, 0.01, 0.001)
    _check(z, idx, mask, seq, (0.01, 0.001), None, got, d)


def test_nothing_takes_part():
    z = torch.full((50, 8), torch.nan, device="cuda")
    idx = torch.zeros(50, 2, dtype=torch.int32, device="cuda")
    closed = torch.full_like(z, -torch.inf)
    none = torch.zeros(50, dtype=torch.bool, device="cuda")
    empty = torch.full((4,), 7, dtype=torch.int32, device="cuda")
    for x, kw in ((z, dict(token_mask=none)), (closed, {}), (z, dict(seq_starts=empty))):
        loss, counts, num = mx.moe_balance_loss(x, idx, 1.0, 1.0, **kw)
        assert not loss.any() and not counts.any() and not num.any()
        d = mx.moe_balance_loss_bwd(x, counts, num, 2, 1.0, 1.0, **kw)
        assert not d.any()
        prior = torch.randn(50, 8, device="cuda")
        out = prior.clone()
        mx.moe_balance_loss_bwd(x, counts, num, 2, 1.0, 1.0, out=out, accumulate=True, **kw)
        assert torch.equal(out, prior)
    loss, counts, num = mx.moe_balance_loss(z[:0], idx[:0], 1.0, 1.0)
    assert not loss.any() and not counts.any() and not num.any()
    assert mx.moe_balance_loss_bwd(z[:0], counts, num, 2, 1.0, 1.0).shape == (0, 8)


def test_tokens_outside_the_sequences_and_entries_out_of_range():
    """seq_starts beyond the tokens is kept in range; NaN rows outside the
    sequences reach nothing."""
    T, E, K = 100, 8, 2
    z, idx, _, _ = _problem(T, E, K, 1, torch.float32, 1, masked=0)
    z[:10] = torch.nan
    z[90:] = torch.nan
    seq = np.array([10, 40, 40, 90], dtype=np.int32)
    got = mx.moe_balance_loss(_dev(z), _dev(idx), 0.1, 0.1, seq_starts=_dev(seq))
    d = mx.moe_balance_loss_bwd(_dev(z), got[1], got[2], K, 0.1, 0.1, seq_starts=_dev(seq))
    _check(z.nan_to_num(0.0, neginf=-torch.inf), idx, None, seq, (0.1, 0.1), None, got, d)
    assert not d[:10].any() and not d[90:].any()
    z, idx, _, _ = _problem(T, E, K, 1, torch.float32, 2, masked=0)
    over = mx.moe_balance_loss(_dev(z), _dev(idx), 0.1, 0.1, seq_starts=_dev(np.array([-5, 60, 2 ** 31 - 1], dtype=np.int32)))
    same = mx.moe_balance_loss(_dev(z), _dev(idx), 0.1, 0.1, seq_starts=_dev(np.array([0, 60, T], dtype=np.int32)))
    assert all(torch.equal(a, b) for a, b in zip(over, same))


def test_in_a_graph_with_a_shared_workspace():
    T, E, K, S = 700, 20, 3, 5
    z, idx, mask, seq = _problem(T, E, K, S, torch.float32, 11)
    zc, ic, mc, sc = _dev(z), _dev(idx), _dev(mask), _dev(seq)
    ws = torch.empty(mx.lib().moe_balance_loss_workspace_size(T, E, S), dtype=torch.uint8, device="cuda")
    out = (torch.empty(2, device="cuda"), torch.empty(S, E, dtype=torch.int32, device="cuda"),
           torch.empty(S + 2, dtype=torch.int32, device="cuda"))
    d = torch.empty(T, E, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        mx.moe_balance_loss(zc, ic, 0.1, 0.1, token_mask=mc, seq_starts=sc, workspace=ws, out=out)
        mx.moe_balance_loss_bwd(zc, out[1], out[2], K, 0.1, 0.1, token_mask=mc, seq_starts=sc, out=d)

    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.stream(s):
        step()
        for g in graphs:
            with torch.cuda.graph(g, stream=s):
                step()
    torch.cuda.synchronize()
    for seed in range(3):
        z, idx, mask, seq = _problem(T, E, K, S, torch.float32, 20 + seed)
        for dst, src in ((zc, z), (ic, idx), (mc, mask), (sc, seq)):
            dst.copy_(torch.as_tensor(src))
        for g in graphs:
            for v in out:
                v.fill_(-1)
            g.replay()
            torch.cuda.synchronize()
            _check(z, idx, mask, seq, (0.1, 0.1), None, out, d)


@pytest.mark.parametrize("E", [8, 60, 128, 700])
def test_both_sides_of_the_one_workgroup_rule(E):
    """Up to two rounds of a workgroup's rows in up to four sequences
    take one launch: sizes just inside and past the limits, against the oracle."""
    threads, lanes = (256, 64) if E > 512 else (512, max(1, 2 ** int(np.ceil(np.log2(E / 8)))))
    edge = threads // lanes
    for T in (edge - 1, edge, edge + 1, 2 * edge - 1, 2 * edge, 2 * edge + 1):
        for S in (1, 4, 5, 64, 65):
            z, idx, mask, seq = _problem(T, E, 3, S, torch.float32, T + S)
            kw = dict(token_mask=_dev(mask), seq_starts=_dev(seq))
            got = mx.moe_balance_loss(_dev(z), _dev(idx), 0.02, 0.003, **kw)
            _check(z, idx, mask, seq, (0.02, 0.003), None, got, None)
    z, idx, mask, seq = _problem(1, E, 3, 9, torch.float32, 0, masked=0, closed=0, dropped=0)
    none = torch.zeros(10, dtype=torch.int32, device="cuda")
    loss, counts, num = mx.moe_balance_loss(_dev(z)[:0], _dev(idx)[:0], 1.0, 1.0, seq_starts=none)
    assert counts.shape == (9, E) and not loss.any() and not counts.any() and not num.any()


@pytest.mark.parametrize("T,E,S", [(2000, 24, 5000), (300, 8, 5000), (1500, 130, 700), (40, 16, 300)])
def test_many_sequences_most_of_them_empty(T, E, S):
    """More sequences than one look-up step holds, hundreds that start at one token."""
    rng = np.random.default_rng(S)
    z, idx, mask, _ = _problem(T, E, 3, 1, torch.float32, S)
    seq = np.sort(np.concatenate([rng.integers(0, T + 1, S + 1 - 2 * 150), np.full(150, T // 3), np.full(150, T // 2)]))
    seq = seq.astype(np.int32)
    kw = dict(token_mask=_dev(mask), seq_starts=_dev(seq))
    dloss = torch.tensor([1.3, 0.4])
    got = mx.moe_balance_loss(_dev(z), _dev(idx), 0.02, 0.003, **kw)
    d = mx.moe_balance_loss_bwd(_dev(z), got[1], got[2], 3, 0.02, 0.003, dloss=_dev(dloss), **kw)
    _check(z, idx, mask, seq, (0.02, 0.003), dloss, got, d)


def test_starts_that_decrease_stay_in_range():
    """Unspecified results, but no access out of range: guard words around every output."""
    T, E, K, S = 500, 12, 2, 40
    z, idx, _, _ = _problem(T, E, K, 1, torch.float32, 5, masked=0)
    rng = np.random.default_rng(1)
    for seq in (rng.integers(-10 ** 6, 10 ** 6, S + 1), np.arange(S, -1, -1) * 12, rng.integers(0, T, S + 1)):
        q = _dev(seq.astype(np.int32))
        bufs = [torch.full((n + 128,), 7, dtype=dt, device="cuda")
                for n, dt in ((2, torch.float32), (S * E, torch.int32), (S + 2, torch.int32), (T * E, torch.float32))]
        out = (bufs[0][:2], bufs[1][:S * E].view(S, E), bufs[2][:S + 2])
        mx.moe_balance_loss(_dev(z), _dev(idx), 0.1, 0.1, seq_starts=q, out=out)
        mx.moe_balance_loss_bwd(_dev(z), out[1], out[2], K, 0.1, 0.1, seq_starts=q, out=bufs[3][:T * E].view(T, E))
        torch.cuda.synchronize()
        for b, n in zip(bufs, (2, S * E, S + 2, T * E)):
            assert b[n:].eq(7).all()


def test_repeated_ids_count_as_often_as_they_stand():
    z = torch.randn(64, 8, device="cuda")
    idx = torch.full((64, 3), 5, dtype=torch.int32, device="cuda")
    _, counts, _ = mx.moe_balance_loss(z, idx, 1.0)
    assert counts.tolist() == [[0, 0, 0, 0, 0, 192, 0, 0]]


def test_two_streams_at_once():
    T, E, K = 9000, 40, 4
    probs = [_problem(T, E, K, 6, torch.float32, s) for s in (1, 2)]
    args = [[_dev(x) for x in p] for p in probs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            z, idx, mask, seq = args[i]
            with torch.cuda.stream(s):
                outs[i].append(mx.moe_balance_loss(z, idx, 0.1, 0.1, token_mask=mask, seq_starts=seq))
    torch.cuda.synchronize()
    for i in range(2):
        _check(*probs[i], (0.1, 0.1), None, outs[i][0], None)
        for o in outs[i][1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, outs[i][0]))


@pytest.mark.parametrize("T,E,S", [(100, 8, 1), (3000, 60, 7), (5000, 128, 1), (40, 700, 3)])
def test_rows_at_the_lowest_value(T, E, S):
    """Tokens whose logits are all the type's lowest value (a mask put in by hand): their
    lse^2, 1.2e77, passes fp32.  Without a z loss its value is 0, with a coefficient that
    brings the mean back into range the mean itself; probabilities stay uniform."""
    z, idx, mask, seq = _problem(T, E, 3, S, torch.float32, 3 * T, closed=0)
    for value, zc in ((torch.finfo(torch.float32).min, 0.0), (-1e20, 0.002), (-1e25, 2.0 ** -50)):
        z[::7] = value
        kw = dict(token_mask=_dev(mask), seq_starts=_dev(seq))
        got = mx.moe_balance_loss(_dev(z), _dev(idx), 0.02, zc, **kw)
        d = mx.moe_balance_loss_bwd(_dev(z), got[1], got[2], 3, 0.02, zc, **kw)
        _check(z, idx, mask, seq, (0.02, zc), None, got, d)
        assert torch.isfinite(got[0]).all() and torch.isfinite(d).all()
    assert 1e30 < got[0][1]
    low = z.to(torch.bfloat16)
    low[::7] = torch.finfo(torch.bfloat16).min
    loss = mx.moe_balance_loss(_dev(low), _dev(idx), 0.02, **kw)[0].tolist()
    assert loss[1] == 0 and 0 < loss[0] < 1
