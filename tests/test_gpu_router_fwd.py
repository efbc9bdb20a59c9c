"""moe_router_fwd on the GPU against the fp64 oracle: ids exactly, scores by a
relative bound.

The kernel's y = exp(z - m) / sum is fp32: z - m rounds by 2^-24 |z - m|, which
the exponential turns into that much relative error (|z - m| < 64 here), the
exponential and the division add a few 2^-24, and the sum of up to 4096
positive terms, 64 in a row and then a tree of 6, at most 70 * 2^-24: within
(64 + 70 + 16) * 2^-24 = 9e-6 of y, taken as 2e-5 with the same for the
denominator's own terms.  Scores under 2^-126 may be flushed."""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_amd as mx
from oracle import router as R

pytestmark = pytest.mark.gpu
REL, TINY = 2e-5, 2.0 ** -126
MODES = [(R.SOFTMAX_OVER_TOPK, False), (R.TOPK_OVER_SOFTMAX, False), (R.TOPK_OVER_SOFTMAX, True), (R.TOPK, False)]


def _logits(T, E, dtype, seed, closed=0.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * 2
    if closed:
        z[torch.rand(T, E, generator=g) < closed] = -torch.inf
    return z.to(dtype).cuda()


def _check(mode, renorm, z, K, got, mask=None):
    idx, scores, aff = (x.cpu().numpy() for x in got)
    ri, rs, ra = R.forward_topk(mode, z.double().cpu().numpy(), K, renorm,
                                None if mask is None else mask.cpu().numpy())
    assert np.array_equal(idx, ri)
    assert np.all(np.abs(scores - rs) <= REL * np.abs(rs) + TINY)
    aff = aff.reshape(ra.shape)
    assert np.all(np.abs(aff - ra) <= REL * np.abs(ra) + TINY)
    assert not aff[ra == 0].any()
    # the affinity at a selected expert is that selection's score, bit for bit
    rows, ks = np.nonzero(idx >= 0)
    assert np.array_equal(aff[rows, idx[rows, ks]], scores[rows, ks])


@pytest.mark.parametrize("mode,renorm", MODES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 128, 8), (7, 3, 3), (1000, 8, 2), (257, 16, 4), (100, 17, 5),
                                   (333, 64, 6), (129, 33, 32), (301, 100, 7), (50, 300, 32), (67, 256, 8),
                                   (64, 513, 8), (20, 1025, 16), (13, 2049, 3), (9, 4096, 32)])
def test_router_fwd_matches_oracle(mode, renorm, dtype, T, E, K):
    z = _logits(T, E, dtype, T + E + K)
    print(f"mode {mode} renorm {renorm} {dtype} T {T} E {E} K {K}", flush=True)
    _check(mode, renorm, z, K, mx.moe_router_fwd(mode, z, K, renorm=renorm))


@pytest.mark.parametrize("mode,renorm", MODES)
@pytest.mark.parametrize("T,E,K", [(200, 12, 5), (99, 70, 8), (40, 600, 12)])
def test_ties_closed_experts_and_masked_tokens(mode, renorm, T, E, K):
    """Few distinct logits (both zeros among them), experts at -inf up to
    whole rows, and masked tokens that hold NaN and infinities."""
    g = torch.Generator().manual_seed(E)
    z = torch.randint(-2, 3, (T, E), generator=g).float()
    z = torch.where((z == 0) & (torch.rand(T, E, generator=g) < 0.5), -z, z)
    z[torch.rand(T, E, generator=g) < 0.3] = -torch.inf
    z[::7] = -torch.inf
    z[3::11, : E - 2] = -torch.inf
    mask = torch.rand(T, generator=g) < 0.7
    bad = torch.tensor([torch.nan, torch.inf, -torch.inf, torch.finfo(torch.float32).min])
    z[~mask] = bad[torch.randint(0, 4, (int((~mask).sum()), E), generator=g)]
    zc = z.cuda()
    for m in (mask.cuda(), mask.cuda().to(torch.uint8) * 7):
        got = mx.moe_router_fwd(mode, zc, K, renorm=renorm, token_mask=m)
        _check(mode, renorm, torch.where(mask[:, None], z, 0.0), K, got, mask)
        assert all(torch.isfinite(x.float()).all() for x in got)


def test_masks_of_the_lowest_finite_value_and_extreme_logits():
    """The type's lowest finite value is a logit like any other: selected last,
    with score 0 (or itself in the plain mode)."""
    for dtype in (torch.float32, torch.bfloat16):
        low = torch.finfo(dtype).min
        z = torch.full((3, 6), low, dtype=dtype)
        z[0, 4] = 1.0
        z[1, 2], z[1, 3] = torch.finfo(dtype).max, 0.0
        z = z.cuda()
        for mode, renorm in MODES:
            idx, scores, _ = mx.moe_router_fwd(mode, z, 3, renorm=renorm)
            assert idx.tolist() == [[4, 0, 1], [2, 3, 0], [0, 1, 2]]
            if mode == R.TOPK:
                assert torch.equal(scores, torch.gather(z.float(), 1, idx.long()))
            else:
                assert scores[0].tolist() == [1, 0, 0] and scores[1].tolist() == [1, 0, 0]
                even = 1 / 6 if mode == R.TOPK_OVER_SOFTMAX and not renorm else 1 / 3
                assert torch.allclose(scores[2], torch.full((3,), even, device="cuda"), rtol=1e-6)


def test_nan_and_infinite_logits_of_live_tokens():
    z = torch.tensor([[0.0, torch.nan, 1.0, 2.0], [0.0, torch.inf, 1.0, 2.0]], device="cuda")
    idx, scores, _ = mx.moe_router_fwd(R.TOPK_OVER_SOFTMAX, z, 3)
    assert idx.tolist() == [[3, 2, 0], [1, 3, 2]]
    assert torch.isnan(scores[0]).all() and torch.isnan(scores[1, 0])
    idx, scores, _ = mx.moe_router_fwd(R.SOFTMAX_OVER_TOPK, z[:1], 3)
    assert idx.tolist() == [[3, 2, 0]] and torch.isfinite(scores).all()


def test_outputs_stay_inside_their_buffers_and_affinities_are_optional():
    T, E, K = 37, 20, 3
    z = _logits(T, E, torch.float32, 5)
    bufs = [torch.full((T * K + 64,), -77, dtype=torch.int32, device="cuda"),
            torch.full((T * K + 64,), -77.0, device="cuda"), torch.full((T * E + 64,), -77.0, device="cuda")]
    out = (bufs[0][:T * K].view(T, K), bufs[1][:T * K].view(T, K), bufs[2][:T * E])
    got = mx.moe_router_fwd(1, z, K, out=out)
    _check(1, False, z, K, got)
    assert bufs[0][T * K:].eq(-77).all() and bufs[1][T * K:].eq(-77).all() and bufs[2][T * E:].eq(-77).all()
    idx, scores = torch.empty_like(out[0]), torch.empty_like(out[1])
    assert mx.lib().moe_router_fwd(1, T, E, K, z.data_ptr(), 0, None, 0, idx.data_ptr(), scores.data_ptr(), None,
                                   torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(idx, got[0]) and torch.equal(scores, got[1])
    assert [tuple(x.shape) for x in mx.moe_router_fwd(1, z[:0], K)] == [(0, K), (0, K), (0,)]


def test_on_a_side_stream_and_in_a_graph():
    T, E, K = 500, 40, 4
    z = _logits(T, E, torch.float32, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = mx.moe_router_fwd(0, z, K)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            mx.moe_router_fwd(0, z, K, out=out)
    torch.cuda.synchronize()
    for seed in (1, 2, 3):
        z.copy_(_logits(T, E, torch.float32, seed))
        graph.replay()
        torch.cuda.synchronize()
        _check(0, False, z, K, out)
        assert all(torch.equal(a, b) for a, b in zip(out, mx.moe_router_fwd(0, z, K)))


@pytest.mark.parametrize("mode,renorm", MODES)
def test_router_backward_of_a_token_without_a_selection(mode, renorm):
    """The selections' backward gives such tokens zeros, whatever they hold."""
    T, E, K = 60, 10, 3
    z = _logits(T, E, torch.float32, 4)
    mask = torch.arange(T, device="cuda") % 5 != 0
    z[::10] = torch.nan
    z[5::10] = -torch.inf
    z[1] = -torch.inf
    idx, scores, _ = mx.moe_router_fwd(mode, z, K, renorm=renorm, token_mask=mask)
    g = torch.randn(T, K, device="cuda")
    d = mx.moe_router_bwd(mode, idx, dscores=g, topk_scores=scores, logits=z, renorm=renorm)
    dead = (idx < 0).all(1)
    assert int(dead.sum()) == 13
    assert not d[dead].any() and torch.isfinite(d).all() and d[~dead].any(1).all()


@pytest.mark.parametrize("E,K", [(7, 3), (64, 8), (128, 8), (128, 5), (256, 1), (512, 8), (512, 2), (700, 8)])
def test_logits_an_ulp_apart(E, K):
    """fp32 logits that differ in their last bits, inside the selection and across its
    end, of both signs: the order is by value, not by expert."""
    g = torch.Generator().manual_seed(E + K)
    T = 400
    z = torch.randn(T, E, generator=g)
    base = torch.randn(T, 1, generator=g) + torch.where(torch.arange(T) % 2 == 0, 4.0, -4.0)[:, None]
    steps = torch.randint(-40, 40, (T, E), generator=g, dtype=torch.int32)
    close = (base.view(torch.int32) + steps).view(torch.float32)
    some = torch.rand(T, E, generator=g) < 0.5
    z = torch.where(some, close, z - 8).cuda()
    z[::5] = close[::5].cuda()
    for mode, renorm in MODES:
        _check(mode, renorm, z, K, mx.moe_router_fwd(mode, z, K, renorm=renorm))


@pytest.mark.parametrize("E", [5, 8, 40, 128, 300, 600])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_fewer_open_experts_than_selections(E, dtype):
    """0 .. K open experts beside each other in a wave, NaN among the closed ones."""
    K, T = min(E, 8), 200
    g = torch.Generator().manual_seed(E)
    z = torch.full((T, E), -torch.inf)
    for t in range(T):
        n = t % (K + 1)
        at = torch.randperm(E, generator=g)[:n]
        z[t, at] = torch.randn(n, generator=g)
    z = z.to(dtype)
    for mode, renorm in MODES:
        _check(mode, renorm, z.cuda(), K, mx.moe_router_fwd(mode, z.cuda(), K, renorm=renorm))
    nan = torch.where((z == -torch.inf) & (torch.rand(T, E, generator=g) < 0.3), torch.nan, z.float()).to(dtype)
    for mode in (R.SOFTMAX_OVER_TOPK, R.TOPK):   # over the selection alone, NaN is closed like -inf
        _check(mode, False, z.cuda(), K, mx.moe_router_fwd(mode, nan.cuda(), K))


def test_two_streams_at_once():
    """Calls on two streams with inputs of their own, interleaved."""
    T, E, K = 4000, 96, 6
    zs = [_logits(T, E, torch.float32, s) for s in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(mx.moe_router_fwd(0, zs[i], K))
    torch.cuda.synchronize()
    for i in range(2):
        _check(0, False, zs[i], K, outs[i][0])
        for o in outs[i][1:]:
            assert all(torch.equal(a, b) for a, b in zip(o, outs[i][0]))
