"""moe_bwd_mxfp8 from an MXFP8 gate/up checkpoint, and a whole layer's training
step around it.

A code times its scale is exact in bf16 (4 significant bits at most), so the
backward from codes and scales must give the bits of the backward from the
dequantised bf16 checkpoint, which the parity tests hold against the oracle.
The bias gradients are atomic fp32 sums, whose order varies from run to run: they
may differ by one bf16 step (2^-7 of the value) where a sum lands on a
rounding border, and by 2^-20 of the largest entry where terms cancel."""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_amd as mx
import oracle
import synthetic as S
from helpers import assert_parity, bf, parity_stats, quantize_weights
from moe_gpu_common import gpu_problem, host, oracle_problem
from oracle import router as R

pytestmark = pytest.mark.gpu

CFGS = {
    "tiny": S.TINY,                                                             # fused epilogue, 128 slots a block
    "medium_s": S.scaled(S.MEDIUM, T=512, H=256, I=352, E=8, K=4, B=128),      # I not a multiple of 64
    "large_s": S.scaled(S.LARGE, T=256, H=256, I=1024, E=4, K=2, B=256),       # stand-alone epilogue, affinity on I
    "fine_s": S.scaled(S.FINE, T=512, H=192, I=128, E=16, K=4, B=128),         # H % 128 != 0, bias
    "fine_h256": S.scaled(S.FINE, T=512, H=256, I=128, E=16, K=4, B=128),      # fused, bias
    "b512": S.scaled(S.MEDIUM, T=640, H=128, I=96, E=4, K=2, B=512),
    "b1024": S.scaled(S.LARGE, T=300, H=128, I=576, E=3, K=2, B=1024),
}


def _bound(gp, ckpt, ck8=None, **kw):
    t, cfg = gp["t"], gp["cfg"]
    gu_c, gu_s, d_c, d_s = gp["wq"]
    E, H, I = cfg.E, cfg.H, cfg.I
    return mx.MoeBwd(t["hidden"], torch.from_numpy(gp["aff"]).cuda(), gu_c.view(E, H, 2, I), gu_s.view(E, H, 2, I // 32),
                     d_c.view(E, I, H), d_s.view(E, I, H // 32), gp["tpid"], gp["b2e"], t["dy"], cfg.B, ckpt,
                     down_proj_bias=t["b2"], affinity_on=cfg.affinity_on, gate_up_checkpoint=ck8, **kw)


def _dequant(codes, scales, fmt):
    n = codes.shape[-1]
    v = oracle.dequantize(host(codes).reshape(-1, n), host(scales).reshape(-1, n // 32), 1, fmt)
    t = torch.from_numpy(np.ascontiguousarray(v)).to(torch.bfloat16)
    assert np.array_equal(t.double().numpy(), np.asarray(v, dtype=np.float64))
    return t.view(codes.shape).cuda()


def _same(cfg, got, ref):
    for k in ("dx", "daff", "dwgu", "dwd"):
        assert torch.equal(got[k].view(torch.int16), ref[k].view(torch.int16)), k
    if cfg.has_bias:
        for k in ("db1", "db2"):
            a, b = got[k].float(), ref[k].float()
            assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -20 * b.abs().max()).all(), k


def _checkpoint(gp, fmt, geglu=0):
    cfg = gp["cfg"]
    _, codes, scales = mx.mxfp8_gated_act_fwd(gp["t"]["ckpt"], geglu, fmt, token_position_to_id=gp["tpid"], T=cfg.T)
    return codes, scales


@pytest.mark.parametrize("geglu", [0, 1])
@pytest.mark.parametrize("fmt", [mx.E4M3, mx.E5M2])
@pytest.mark.parametrize("name", list(CFGS))
def test_same_bits_as_the_dequantised_bf16_checkpoint(name, fmt, geglu):
    cfg = CFGS[name]
    print("checkpoint8", name, fmt, geglu, flush=True)
    gp = gpu_problem(cfg)
    ck = _checkpoint(gp, fmt, geglu)
    ref = _bound(gp, _dequant(*ck, fmt), activation=geglu).run()
    got = _bound(gp, None, ck, fmt_checkpoint=fmt, activation=geglu).run()
    torch.cuda.synchronize()
    _same(cfg, got, ref)
    # what padding holds reaches nothing: NaN codes there, NaN scales where a whole group is padding
    pad = ((gp["tpid"] < 0) | (gp["tpid"] >= cfg.T)).view(-1, 1, 1, cfg.B)
    codes = torch.where(pad, torch.full_like(ck[0], 0x7f), ck[0])
    whole = pad.view(-1, 1, 1, cfg.B // 32, 32).all(-1)
    scales = torch.where(whole, torch.full_like(ck[1], 255), ck[1])
    junk = _bound(gp, None, (codes, scales), fmt_checkpoint=fmt, activation=geglu).run()
    torch.cuda.synchronize()
    _same(cfg, junk, ref)


@pytest.mark.parametrize("name", ["tiny", "large_s", "fine_s"])
def test_against_the_oracle_and_with_the_other_options(name):
    """Against the oracle on the dequantised checkpoint; then with a token
    count and with accumulation, against the bf16 checkpoint's bits."""
    cfg = CFGS[name]
    gp = gpu_problem(cfg)
    ck = _checkpoint(gp, mx.E4M3)
    deq = _dequant(*ck, mx.E4M3)
    op = _bound(gp, None, ck)
    got = op.run()
    torch.cuda.synchronize()
    gp["t"]["ckpt"] = deq
    p, _ = oracle_problem(gp)
    ref = oracle.moe_bwd(p)
    E, H, I, T = cfg.E, cfg.H, cfg.I, cfg.T
    for k, rows, experts in (("dx", T, None), ("daff", T, None), ("dwgu", E * H, E), ("dwd", E * I, E)):
        assert_parity(k, parity_stats(bf(host(got[k])).reshape(-1), bf(ref[k]).reshape(-1), rows=rows, experts=experts))
    n = torch.tensor([T * 2 // 3], dtype=torch.int32, device="cuda")
    for kw in (dict(num_valid_tokens=n), dict(accumulate=True)):
        a, b = _bound(gp, None, ck, **kw), _bound(gp, deq, **kw)
        for _ in range(2 if "accumulate" in kw else 1):
            x, y = a.run(), b.run()
        torch.cuda.synchronize()
        _same(cfg, x, y)
    # stage by stage is one call (a fresh output, the filled workspace)
    before = {k: v.clone() for k, v in got.items() if v is not None}
    for s in range(op.NUM_STAGES):
        op.stage(s)
    torch.cuda.synchronize()
    _same(cfg, op.out, before)


def test_refusals():
    gp = gpu_problem(S.TINY)
    codes, scales = _checkpoint(gp, mx.E4M3)
    bf16 = gp["t"]["ckpt"]
    side = torch.zeros(gp["N"], S.TINY.I, S.TINY.B, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mx.MxError, match="not both"):
        _bound(gp, bf16, (codes, scales)).run()
    with pytest.raises(mx.MxError, match="null"):
        _bound(gp, None).run()
    with pytest.raises(mx.MxError, match="together"):
        _bound(gp, None, (codes, None)).run()
    with pytest.raises(mx.MxError, match="together"):
        _bound(gp, bf16, (None, scales)).run()
    with pytest.raises(mx.MxError, match="fmt_checkpoint"):
        _bound(gp, None, (codes, scales), fmt_checkpoint=3).run()
    with pytest.raises(mx.MxError, match="checkpoints go with"):
        _bound(gp, None, (codes, scales), gate_act_checkpoint_T=side).run()
    with pytest.raises(ValueError, match="shape"):
        _bound(gp, None, (codes, scales[:, :, :, :2]))
    with pytest.raises(TypeError):
        _bound(gp, None, (codes.view(torch.int8), scales))


def _layer_step(z, x, dy, wq, w_up, cfg, mode, renorm, mask, coefs):
    """One training step of a MoE layer, as a user strings the operators together."""
    T, H, I, E, K, B = cfg.T, cfg.H, cfg.I, cfg.E, cfg.K, cfg.B
    idx, scores, aff = mx.moe_router_fwd(mode, z, K, renorm=renorm, token_mask=mask)
    loss, counts, num = mx.moe_balance_loss(z, idx, *coefs, token_mask=mask)
    tpid, b2e = mx.moe_build_blocks(idx, E, B)
    N = b2e.numel()
    # the gate/up product of each block (the caller's forward)
    rows = x.float()[tpid.view(N, B).clamp(min=0).long()].transpose(1, 2).contiguous()   # [N, H, B]
    gate_up = torch.bmm(w_up[b2e.long()], rows).view(N, 2, I, B).to(torch.bfloat16)
    inter, *ck = mx.mxfp8_gated_act_fwd(gate_up, token_position_to_id=tpid, T=T)
    grads = mx.moe_bwd_mxfp8(x, aff, *wq, tpid, b2e, dy, B, None, affinity_on=cfg.affinity_on, gate_up_checkpoint=ck)
    dz = mx.moe_router_bwd(mode, idx, daff=grads["daff"], topk_scores=scores, logits=z, renorm=renorm)
    from_layer = dz.clone()
    mx.moe_balance_loss_bwd(z, counts, num, K, *coefs, token_mask=mask, out=dz, accumulate=True)
    return dict(idx=idx, aff=aff, loss=loss, counts=counts, tpid=tpid, b2e=b2e, gate_up=gate_up, inter=inter, ck=ck,
                grads=grads, from_layer=from_layer, dz=dz)


@pytest.mark.parametrize("mode,renorm", [(R.SOFTMAX_OVER_TOPK, False), (R.TOPK_OVER_SOFTMAX, True)])
@pytest.mark.parametrize("name", ["tiny", "large_s"])
def test_a_layers_training_step(name, mode, renorm):
    """Router, losses, blocks, activation, MoE backward, router backward and the
    losses' gradient in a row, on a padded batch whose padding holds NaN logits;
    each result against the oracle on what the step handed to it."""
    cfg = CFGS[name]
    T, H, I, E, K = cfg.T, cfg.H, cfg.I, cfg.E, cfg.K
    rng = np.random.default_rng(7)
    z = torch.from_numpy(rng.normal(0, 1.5, (T, E)).astype(np.float32))
    mask = torch.from_numpy(rng.random(T) < 0.85)
    z[~mask] = torch.nan
    t = S.moe_tensors(cfg, 1, "cpu")
    gu_c, gu_s, d_c, d_s = quantize_weights(S.bf16_bits(t["w_gate_up"]), S.bf16_bits(t["w_down"]))
    wq = [torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in (gu_c, gu_s, d_c, d_s)]
    w_up = torch.from_numpy(np.asarray(oracle.dequantize(gu_c.reshape(-1, I), gu_s.reshape(-1, I // 32), 1, 0),
                                       dtype=np.float32)).view(E, H, 2 * I).transpose(1, 2).contiguous().cuda()
    r = _layer_step(z.cuda(), t["hidden"].cuda(), t["dy"].cuda(), wq, w_up, cfg, mode, renorm, mask.cuda(), (0.01, 0.001))
    torch.cuda.synchronize()
    zc = torch.where(mask[:, None], z, 0.0).double().numpy()
    idx, sc, aff = R.forward_topk(mode, zc, K, renorm, mask.numpy())
    assert np.array_equal(host(r["idx"]), idx)
    assert np.abs(host(r["aff"]).reshape(T, E) - aff).max() <= 2e-5
    loss, counts, _, dbal = R.balance(zc, idx, 0.01, 0.001, mask.numpy())
    assert np.array_equal(host(r["counts"]), counts) and np.all(np.abs(host(r["loss"]) - loss) <= 5e-5 * loss)
    N = r["b2e"].numel()
    tpid, b2e = oracle.build_blocks(idx, E, cfg.B, N)
    assert np.array_equal(host(r["tpid"]), tpid) and np.array_equal(host(r["b2e"]), b2e)
    deq = _dequant(*r["ck"], 0)
    p = oracle.MoeProblem(T=T, H=H, I=I, E=E, N=N, B=cfg.B, hidden=S.bf16_bits(t["hidden"]), aff=host(r["aff"]),
                          wgu_codes=gu_c, wgu_scales=gu_s, wd_codes=d_c, wd_scales=d_s, tpid=tpid, b2e=b2e,
                          dy=S.bf16_bits(t["dy"]), ckpt=S.bf16_bits(deq), b2=None, affinity_on=cfg.affinity_on,
                          has_bias=0, nthreads=0)
    ref = oracle.moe_bwd(p)
    for k, rows, experts in (("dx", T, None), ("daff", T, None), ("dwgu", E * H, E), ("dwd", E * I, E)):
        assert_parity(k, parity_stats(bf(host(r["grads"][k])).reshape(-1), bf(ref[k]).reshape(-1), rows=rows, experts=experts))
    # the router's backward and the losses' gradient, from the step's own d(affinity)
    live = mask.numpy()
    g = np.take_along_axis(r["grads"]["daff"].double().cpu().numpy().reshape(T, E), np.maximum(idx, 0).astype(np.int64), axis=1)
    rb = R.backward(mode, zc[live], idx[live], g[live], renorm)
    G = np.abs(g[live]).max(axis=1, keepdims=True)
    if renorm:
        G = G / R.forward(R.TOPK_OVER_SOFTMAX, zc[live], idx[live]).sum(axis=1, keepdims=True)
    got = host(r["from_layer"])
    assert np.all(np.abs(got[live] - rb) <= 2e-5 * G + 1e-30) and not got[~live].any()
    dz = host(r["dz"])
    assert np.isfinite(dz).all() and not dz[~live].any()
    # one fp32 addition on top of the gradient's own error
    add = np.abs(dz[live] - got[live] - dbal[live])
    assert np.all(add <= 2.0 ** -23 * np.abs(dz[live]) + 6e-5 * np.abs(dbal).max())


def test_a_captured_backward_replays():
    """The backward with the 8-bit checkpoint made in the same graph, replayed on
    new inputs with eager work between."""
    cfg = CFGS["large_s"]
    gp = gpu_problem(cfg)
    ckpt = gp["t"]["ckpt"]
    inter, codes, scales = mx.mxfp8_gated_act_fwd(ckpt, token_position_to_id=gp["tpid"], T=cfg.T)
    op = _bound(gp, None, (codes, scales))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        op.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            mx.mxfp8_gated_act_fwd(ckpt, token_position_to_id=gp["tpid"], T=cfg.T, out=(inter, codes, scales))
            op.run()
    torch.cuda.synchronize()
    for k in range(3):
        ckpt.copy_(S.normal_bf16(ckpt.shape, 0.3, k + 1, 55, "cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in op.out.items() if v is not None}
        ref = _bound(gp, None, _checkpoint(gp, mx.E4M3)).run()
        torch.cuda.synchronize()
        _same(cfg, got, ref)


@pytest.mark.parametrize("name", ["medium_s", "fine_s"])
def test_beside_the_down_projection_checkpoint(name):
    """The a * dY checkpoint goes with either form of the gate/up checkpoint."""
    cfg = CFGS[name]
    gp = gpu_problem(cfg)
    ck = _checkpoint(gp, mx.E4M3)
    tok = gp["tpid"].long().clamp(0, cfg.T - 1)
    a = torch.from_numpy(gp["aff"]).cuda().view(cfg.T, cfg.E)[tok, gp["b2e"].long().repeat_interleave(cfg.B)]
    ady = (a[:, None] * gp["t"]["dy"].float()[tok]).to(torch.bfloat16).view(gp["N"], cfg.B, cfg.H)
    got = _bound(gp, None, ck, down_proj_act_checkpoint=ady).run()
    ref = _bound(gp, _dequant(*ck, mx.E4M3), down_proj_act_checkpoint=ady).run()
    torch.cuda.synchronize()
    _same(cfg, got, ref)
