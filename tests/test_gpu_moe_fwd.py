"""moe_fwd_mxfp8 on the GPU against the layer in 64 bits (oracle/ffn.py, whose bounds the tolerances are)."""
import numpy as np
import pytest
import torch

import oracle
from ffn_common import HALF, Problem, bf16_values, check_rows
from oracle import ffn

pytestmark = pytest.mark.gpu

CASES = {
    # the gate/up product's tiles: 256 x 256 on either ring, 128 x 128 (short H, I < 128, blocks of 128 slots)
    "tiles_256": dict(T=700, H=1024, I=384, E=3, K=2, B=512, residual=True),
    "tiles_256_ragged": dict(T=300, H=1056, I=192, E=2, K=1, B=256, bias=True),
    "tiles_128": dict(T=300, H=128, I=256, E=4, K=2, B=128, bias=True),
    "tiles_128_short_I": dict(T=300, H=384, I=96, E=4, K=1, B=256, on_i=True),
    # the down projection's: 256 x 256, 128 x 256 (256 of them or more), aligned and not; 128 x 128 above
    "down_256": dict(T=300, H=288, I=1024, E=2, K=1, B=256, residual=True),
    "down_256_ragged": dict(T=300, H=288, I=1056, E=2, K=1, B=256),
    "down_128x256": dict(T=120, H=2304, I=128, E=30, K=2, bias=True),
    "down_128x256_ragged": dict(T=120, H=2336, I=160, E=30, K=2),
    "down_long_ragged": dict(T=100, H=96, I=4128, E=1, K=1),
    # H, I or both not a multiple of 128
    "ragged_H": dict(T=260, H=160, I=128, E=2, K=2, B=256, geglu=True, bias=True),
    "ragged_I": dict(T=200, H=128, I=160, E=3, K=2, B=128, geglu=True, on_i=True, residual=True),
    "ragged_both": dict(T=330, H=608, I=352, E=3, K=3, B=256, bias=True, p=0.2, residual=True, dropped=0.2),
    "smallest": dict(T=1, H=32, I=32, E=1, K=1, B=128, bias=True, residual=True),
    "one_token_many_experts": dict(T=1, H=128, I=128, E=70, K=8, B=128, p=0.5),
    # a contraction long enough for cut tiles, and a wide row
    "long_I": dict(T=150, H=256, I=4224, E=2, K=1, B=256, on_i=True),
    "wide_H": dict(T=140, H=2304, I=128, E=2, K=2, B=128, bias=True, p=0.1, dropped=0.5),
    # large values: the activation's flat parts
    "large_values": dict(T=200, H=128, I=128, E=2, K=1, B=128, sigma=40.0),
    "large_values_geglu": dict(T=200, H=128, I=128, E=2, K=1, B=128, sigma=40.0, geglu=True),
}


def _run(p, checkpoint=None, **more):
    import mxfp8_grouped_gemm_amd as mx
    pos, kw = p.on()
    r = mx.moe_fwd_mxfp8(*pos, **{**kw, **more}, checkpoint=checkpoint)
    torch.cuda.synchronize()
    return r


def _gate_up(p, gus):
    """gu and its bound in the checkpoint's layout [N, 2, I, B], zeros in the slots of no token."""
    ck, d = np.zeros((2, p.N, 2, p.I, p.B))
    seen = {}
    for b, e in enumerate(p.b2e):
        n = int((p.tpid[b * p.B:(b + 1) * p.B] >= 0).sum())
        k = seen.get(e, 0)
        if n:
            for dst, src in ((ck, gus[e][0]), (d, gus[e][1])):
                dst[b, :, :, :n] = src[k:k + n].transpose(1, 2, 0)
        seen[e] = k + n
    return ck, d


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    p = Problem(**CASES[name], seed=sum(map(ord, name)))
    y, dy, gus = p.exact()
    r = _run(p, "bf16")
    check_rows(r["out"], y, dy, name)
    ck, d = _gate_up(p, gus)
    got = bf16_values(r["checkpoint"])
    assert (np.abs(got - ck) <= d + (np.abs(ck) + d) * HALF).all()
    assert not got[(p.tpid < 0).reshape(p.N, 1, 1, p.B).repeat(2, 1).repeat(p.I, 2)].any()
    # without a checkpoint, and again: the same bits
    assert torch.equal(_run(p)["out"], r["out"])
    # the 8-bit checkpoint is the bf16 one, quantised
    for fmt in (oracle.E4M3, oracle.E5M2):
        r8 = _run(p, "mxfp8", fmt_checkpoint=fmt)
        bits = r["checkpoint"].cpu().view(torch.int16).numpy().view(np.uint16)
        codes, scales = oracle.quantize(bits.reshape(-1, p.B), 1, fmt)
        assert np.array_equal(r8["checkpoint"][0].cpu().numpy().reshape(codes.shape), codes)
        assert np.array_equal(r8["checkpoint"][1].cpu().numpy().reshape(scales.shape), scales)
        assert torch.equal(r8["out"], r["out"])


@pytest.mark.parametrize("B", [128, 256, 512, 1024])
def test_block_sizes(B):
    """Partly filled and empty blocks of every size: what the checkpoint holds in tiles without a token."""
    p = Problem(T=37, H=1024, I=160, E=3, K=2, B=B, seed=B)
    y, dy, gus = p.exact()
    r = _run(p, "bf16")
    check_rows(r["out"], y, dy)
    ck, d = _gate_up(p, gus)
    assert (np.abs(bf16_values(r["checkpoint"]) - ck) <= d + (np.abs(ck) + d) * HALF).all()
    codes, scales = _run(p, "mxfp8")["checkpoint"]
    dead = torch.from_numpy((p.tpid < 0).reshape(p.N, 1, 1, B)).cuda()
    assert not (codes.bool() & dead).any()
    assert not (scales.bool() & dead.view(p.N, 1, 1, B // 32, 32).all(-1)).any()


def test_rows_of_far_apart_sizes():
    """A token whose output is 2^40 times another's in the same tile leaves that one as exact."""
    p = Problem(T=128, H=128, I=64, E=1, K=1, B=128, idx=np.zeros((128, 1), np.int32), seed=21)
    p.x[::2] *= 2.0 ** 20        # g and u alike: y by 2^40 (SiLU is the identity or 0 there)
    y, dy, _ = p.exact()
    out = _run(p)["out"]
    check_rows(out, y, dy)
    rel = np.abs(bf16_values(out) - y)[1::2].max() / np.abs(y[1::2]).max()
    assert rel < 2.0 ** -7


def test_many_blocks():
    """More blocks than the set-up's one-workgroup lists take, most of them empty, and more than one round of tiles."""
    p = Problem(T=600, H=128, I=64, E=40, K=4, B=128, seed=5)
    pad = 1100 - p.N
    p.tpid = np.concatenate([p.tpid, np.full(pad * p.B, -1, np.int32)])
    p.b2e = np.concatenate([p.b2e, np.full(pad, 39, np.int32)])
    p.N = 1100
    y, dy, _ = p.exact()
    check_rows(_run(p, "mxfp8")["out"], y, dy)


@pytest.mark.parametrize("I", [64, 160, 256])
def test_short_contractions_over_many_tiles(I):
    """Enough blocks that a workgroup of the short down projection goes through several tiles of H, the last one partial."""
    p = Problem(T=300, H=2080, I=I, E=3, K=2, B=128, bias=I == 64, dropped=0.1, seed=40 + I)
    pad = 512 - p.N
    p.tpid = np.concatenate([p.tpid, np.full(pad * p.B, -1, np.int32)])
    p.b2e = np.concatenate([p.b2e, np.full(pad, 2, np.int32)])
    p.N = 512
    y, dy, _ = p.exact()
    check_rows(_run(p)["out"], y, dy)


# name: the problem and how many blocks its list is padded to, those behind of no token
PADDED = {
    # 256 x 256 tiles, whole and ragged contractions
    "tiles_256": (dict(T=300, H=1024, I=384, E=3, K=2, B=256, dropped=0.1, bias=True), 60),
    "tiles_256_ragged": (dict(T=300, H=1056, I=416, E=3, K=2, B=512, dropped=0.1, geglu=True), 40),
    # X quantised slot by slot; rows of fp32 and of fp16
    "by_slot": (dict(T=330, H=1056, I=4096, E=2, K=1, B=256, dropped=0.1, residual=True), 12),
    "by_slot_f16": (dict(T=330, H=1024, I=4128, E=2, K=1, B=512, dropped=0.1, bias=True), 9),
    # the scaled MFMA at 128 x 128
    "tiles_128": (dict(T=300, H=768, I=160, E=5, K=2, B=128, on_i=True), 200),
}


@pytest.mark.parametrize("name", PADDED)
def test_padded_block_list(name):
    """Lists as long as a fixed capacity needs: more tiles than one round of the CUs, most of no token."""
    args, N = PADDED[name]
    p = Problem(**args, seed=sum(map(ord, name)))
    assert p.N <= N
    p.tpid = np.concatenate([p.tpid, np.full((N - p.N) * p.B, -1, np.int32)])
    p.b2e = np.concatenate([p.b2e, np.full(N - p.N, p.E - 1, np.int32)])
    p.N = N
    y, dy, gus = p.exact()
    r = _run(p, "bf16")
    check_rows(r["out"], y, dy, name)
    ck, d = _gate_up(p, gus)
    gu = bf16_values(r["checkpoint"])
    assert (np.abs(gu - ck) <= d + (np.abs(ck) + d) * HALF).all()
    assert not gu[(p.tpid < 0).reshape(p.N, 1, 1, p.B).repeat(2, 1).repeat(p.I, 2)].any()
    bits = r["checkpoint"].cpu().view(torch.int16).numpy().view(np.uint16)
    codes, scales = oracle.quantize(bits.reshape(-1, p.B), 1, oracle.E4M3)
    r8 = _run(p, "mxfp8")
    assert torch.equal(r8["out"], r["out"])
    assert np.array_equal(r8["checkpoint"][0].cpu().numpy().reshape(codes.shape), codes)
    assert np.array_equal(r8["checkpoint"][1].cpu().numpy().reshape(scales.shape), scales)


def test_valid_tokens_and_foreign_blocks():
    """Tokens from num_valid_tokens on are in no slot; blocks of an expert outside [0, E) are skipped."""
    p = Problem(T=200, H=128, I=128, E=3, K=2, B=128, residual=True, seed=6)
    n = torch.tensor([150], dtype=torch.int32, device="cuda")
    p.b2e[-1] = 7
    p.tpid[-p.B:-p.B + 5] = np.arange(5)
    for e, (t, a) in p.pairs.items():
        p.pairs[e] = (t[t < 150], a[t < 150])
    y, dy, _ = p.exact()
    out = _run(p, num_valid_tokens=n)["out"]
    check_rows(out, y, dy)
    assert torch.equal(out[150:].cpu(), p.residual[150:])


def test_in_place_residual_and_padding_garbage():
    """out may be the residual; rows of hidden_states that no slot reads may hold anything."""
    import mxfp8_grouped_gemm_amd as mx
    p = Problem(T=130, H=256, I=128, E=2, K=1, B=128, residual=True, dropped=0.4, seed=8)
    y, dy, _ = p.exact()
    unused = np.nonzero((p.idx < 0).all(1))[0]
    pos, kw = p.on()
    pos[0][torch.from_numpy(unused).cuda()] = float("nan")
    res = kw["residual"]
    mx.moe_fwd_mxfp8(*pos, **kw, out=res)
    torch.cuda.synchronize()
    check_rows(res, y, dy)


def test_nan_stays_in_its_row():
    """A NaN in one token's row reaches no other token."""
    p = Problem(T=140, H=128, I=128, E=2, K=2, B=128, seed=9)
    clean = _run(p)["out"]
    p.x[77, 5] = float("nan")
    out = _run(p)["out"]
    rows = torch.arange(140) != 77
    assert torch.equal(out[rows.cuda()], clean[rows.cuda()])


def test_dense_block():
    """One expert that every token is routed to: a dense gated FFN."""
    p = Problem(T=300, H=256, I=256, E=1, K=1, B=256, idx=np.zeros((300, 1), np.int32), seed=10)
    p.aff[:] = 1.0
    p.pairs = {0: (np.arange(300), np.ones(300))}
    y, dy, _ = p.exact()
    check_rows(_run(p)["out"], y, dy)


def test_two_streams_and_a_graph():
    """Calls on another stream; a captured call replayed on changed inputs, another dropout offset among them, with eager
    work in between."""
    import mxfp8_grouped_gemm_amd as mx
    p = Problem(T=300, H=256, I=256, E=4, K=2, B=128, residual=True, p=0.3, seed=11)
    pos, kw = p.on()
    eager = mx.MoeFwd(*pos, **kw, checkpoint="mxfp8")
    want = eager.run()["out"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    op = mx.MoeFwd(*pos, **kw, checkpoint="mxfp8")
    with torch.cuda.stream(s):
        got = op.run()["out"].clone()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.run()
    x0 = pos[0].clone()
    for k in range(4):
        pos[0].copy_(x0 * (1 + k))
        kw["dropout_rng"][1] = 1000 + k
        want = {n: v for n, v in eager.run().items()}
        op.out["out"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(op.out["out"], want["out"])
        assert torch.equal(op.out["checkpoint"][0], want["checkpoint"][0])
        assert torch.equal(op.out["checkpoint"][1], want["checkpoint"][1])


@pytest.mark.parametrize("checkpoint", ["bf16", "mxfp8"])
def test_forward_and_backward(checkpoint):
    """A layer's forward and backward as a training step makes them: weights quantised for both, the forward's checkpoint
    into the backward, the gradient through the residual's dropout.  The backward from the forward's checkpoint gives the
    oracle's gradients for the same checkpoint."""
    import mxfp8_grouped_gemm_amd as mx
    from helpers import assert_parity, bf, parity_stats
    from moe_gpu_common import host
    p = Problem(T=256, H=128, I=256, E=4, K=2, B=128, residual=True, p=0.25, seed=12)
    dev = "cuda"
    x, wgu, wd = p.x.to(dev), p.w_gate_up.to(dev), p.w_down.to(dev)
    topk = torch.from_numpy(p.idx).to(dev)
    tpid, b2e = mx.moe_build_blocks(topk, p.E, p.B)
    aff = torch.from_numpy(p.aff.reshape(-1)).to(dev)
    rng = torch.tensor(p.seed_offset, dtype=torch.int64, device=dev)
    gu_c, gu_s = mx.mxfp8_quantize_transposed(wgu.view(p.E, p.H, 2 * p.I))
    d_c, d_s = mx.mxfp8_quantize_transposed(wd)
    assert np.array_equal(gu_c.cpu().numpy().reshape(p.q[0].shape), p.q[0]) and np.array_equal(d_s.cpu().numpy(), p.q[3])
    f = mx.moe_fwd_mxfp8(x, aff, gu_c.view(p.E, 2, p.I, p.H), gu_s.view(p.E, 2, p.I, p.H // 32), d_c, d_s, tpid, b2e, p.B,
                         checkpoint=checkpoint, residual=p.residual.to(dev), dropout_p=p.p, dropout_rng=rng)
    y, dy, _ = p.exact()
    check_rows(f["out"], y, dy)
    dout = torch.randn(p.T, p.H, device=dev, generator=torch.Generator(dev).manual_seed(1)).to(torch.bfloat16)
    dlayer = mx.dropout_add_bwd(dout, p.p, rng)
    bgu_c, bgu_s = mx.mxfp8_quantize(wgu.view(-1, p.I))
    bd_c, bd_s = mx.mxfp8_quantize(wd.view(-1, p.H))
    E, H, I = p.E, p.H, p.I
    ck = f["checkpoint"]
    kw = dict(gate_up_checkpoint=ck) if checkpoint == "mxfp8" else {}
    g = mx.moe_bwd_mxfp8(x, aff, bgu_c.view(E, H, 2, I), bgu_s.view(E, H, 2, I // 32), bd_c.view(E, I, H),
                         bd_s.view(E, I, H // 32), tpid, b2e, dlayer, p.B, ck if checkpoint == "bf16" else None, **kw)
    torch.cuda.synchronize()
    keep = ffn.dropout_keep(p.T * H, p.p, *p.seed_offset).reshape(p.T, H)
    want = np.where(keep, bf16_values(dout) * ffn.dropout_scale(p.p), 0.0)
    assert (np.abs(bf16_values(dlayer) - want) <= np.abs(want) * (HALF + 2.0 ** -23)).all()
    if checkpoint == "mxfp8":
        v = ffn.mx_values(ck[0].cpu().numpy(), ck[1].cpu().numpy())
        ck = torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16)    # exact: 4 significant bits
    N = b2e.numel()
    prob = oracle.MoeProblem(T=p.T, H=H, I=I, E=E, N=N, B=p.B, hidden=host(x), aff=host(aff).reshape(-1),
                             wgu_codes=bgu_c.cpu().numpy().reshape(E, H, 2, I),
                             wgu_scales=bgu_s.cpu().numpy().reshape(E, H, 2, I // 32),
                             wd_codes=bd_c.cpu().numpy().reshape(E, I, H), wd_scales=bd_s.cpu().numpy().reshape(E, I, H // 32),
                             tpid=tpid.cpu().numpy(), b2e=b2e.cpu().numpy(), dy=host(dlayer), ckpt=host(ck), b2=None,
                             affinity_on=0, has_bias=0, nthreads=0)
    ref = oracle.moe_bwd(prob)
    for k, rows, experts in (("dx", p.T, None), ("daff", None, None), ("dwgu", None, E), ("dwd", None, E)):
        assert_parity(k, parity_stats(bf(host(g[k])), bf(ref[k]), rows=rows, experts=experts))


def test_rows_past_32_bits():
    """2^20 slots whose rows take more than 2^32 bytes: 512 tokens 256 times over, all the same, the first against the oracle."""
    import mxfp8_grouped_gemm_amd as mx
    p = Problem(T=512, H=2080, I=32, E=8, K=8, B=1024, seed=21)
    pos, kw = p.on()
    n = 256
    T = n * p.T
    x, aff = pos[0].repeat(n, 1), pos[1].view(p.T, p.E).repeat(n, 1)
    tpid = torch.arange(T, dtype=torch.int32, device="cuda").repeat(p.E)
    b2e = torch.arange(p.E, dtype=torch.int32, device="cuda").repeat_interleave(T // p.B)
    assert tpid.numel() * p.H * 2 > 1 << 32
    y = mx.moe_fwd_mxfp8(x, aff.view(-1), *pos[2:6], tpid, b2e, p.B)["out"].view(n, p.T, p.H)
    assert (y == y[:1]).all()
    want, dy, _ = p.exact()
    check_rows(y[0], want, dy)


def test_weights_past_32_bits():
    """An expert whose weights lie behind the 2^32nd byte gives what it gives alone, with block lists and for few tokens."""
    import mxfp8_grouped_gemm_amd as mx
    E, H, I, B, T = 38, 4096, 14336, 128, 96
    g = torch.Generator("cuda").manual_seed(3)

    def codes(*shape):   # E4M3 of magnitude 0.5 to 0.94
        c = torch.randint(0x30, 0x38, shape, generator=g, device="cuda", dtype=torch.uint8)
        return c | (torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.uint8) << 7)
    wgu, wd = codes(E, 2, I, H), codes(E, H, I)
    assert wgu[:-1].numel() > 1 << 32
    sgu = torch.full((E, 2, I, H // 32), 127 - 5, dtype=torch.uint8, device="cuda")
    sd = torch.full((E, H, I // 32), 127 - 6, dtype=torch.uint8, device="cuda")
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    tpid = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    tpid[:T] = torch.arange(T, device="cuda")
    aff = torch.zeros(T, E, device="cuda")
    aff[:, -1] = 0.75
    many = mx.moe_fwd_mxfp8(x, aff.view(-1), wgu, sgu, wd, sd, tpid, torch.full((1,), E - 1, dtype=torch.int32, device="cuda"), B)
    last = [t[-1:].contiguous() for t in (wgu, sgu, wd, sd)]
    one = mx.moe_fwd_mxfp8(x, aff[:, -1].contiguous(), *last, tpid, torch.zeros(1, dtype=torch.int32, device="cuda"), B)
    assert many["out"].float().norm() > 0 and torch.equal(many["out"], one["out"])
    for n in (1, 3, 9, T):
        ids = torch.full((n, 1), E - 1, dtype=torch.int32, device="cuda")
        a = torch.full((n, 1), 0.75, device="cuda")
        y = mx.moe_tokens_fwd_mxfp8(x[:n], ids, a, wgu, sgu, wd, sd)
        z = mx.moe_tokens_fwd_mxfp8(x[:n], torch.zeros_like(ids), a, *last)
        # E chooses how many columns a workgroup takes, not how a column is summed, up to the split of the contraction
        assert y.float().norm() > 0 and (y.double() - z.double()).norm() <= 2 ** -8 * z.double().norm()
