"""Phase 1 with its epilogue in one kernel, and what the epilogue's converters rest on.

The fused kernel takes layers of at least 256 Phase-1 tiles; blocks of padding bring
small layers there.  Each case asserts from the workspace's layout which of the two
paths it takes."""
import dataclasses

import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_amd as mx
import oracle
import synthetic as S
from helpers import pairs_to_rows, quantize_weights, stage_major_to_rows
from moe_gpu_common import gpu_problem, host, oracle_problem
from test_gpu_moe import _check_outputs
from test_gpu_moe_checkpoint8 import _dequant

pytestmark = pytest.mark.gpu

# configuration and the blocks that make 256 tiles of it
CFGS = {
    "tiny": (S.TINY, 300),
    "bias": (S.scaled(S.FINE, T=512, H=256, I=128, E=16, K=4, B=128), 300),
    "i512_on_i": (S.scaled(S.LARGE, T=300, H=384, I=512, E=3, K=2, B=256), 40),
    "ragged_i": (S.scaled(S.MEDIUM, T=200, H=128, I=160, E=5, K=2, B=512), 40),
    "b1024": (S.scaled(S.MEDIUM, T=300, H=256, I=96, E=3, K=2, B=1024), 40),
}
E4, E5 = mx.E4M3, mx.E5M2
OPTIONS = {
    "default": {},
    "geglu": dict(activation=mx.ACT_GEGLU),
    "count": dict(num_valid_tokens=2 / 3),
    "accumulate": dict(accumulate=True),
    "grad_e4m3": dict(fmt_grad=E4, fmt_act=E5),
    "weight_e5m2": dict(fmt_weight=E5),
    "all_e5m2_count": dict(fmt_weight=E5, fmt_act=E5, num_valid_tokens=1 / 2),
}


def fused(op):
    """Whether the layout has no room for the product and its tile ranges."""
    L = op.layout
    assert (L["phase1_ds"] == L["phase1_tiles"]) == (L["phase1_tiles"] == L["phase3_tiles"])
    return L["phase1_ds"] == L["phase1_tiles"]


def _weights(gp, fmt):
    """The problem's weight codes in `fmt` (the library's e4m3 ones, or the oracle's)."""
    cfg, (gu_c, gu_s, d_c, d_s) = gp["cfg"], gp["wq"]
    E, H, I = cfg.E, cfg.H, cfg.I
    w = gu_c.view(E, H, 2, I), gu_s.view(E, H, 2, I // 32), d_c.view(E, I, H), d_s.view(E, I, H // 32)
    if fmt == E4:
        return w
    q = quantize_weights(host(gp["t"]["w_gate_up"]), host(gp["t"]["w_down"]), fmt)
    return tuple(torch.from_numpy(np.ascontiguousarray(v)).cuda() for v in q)


def _bound(gp, weights, blocks, ckpt, ck8=None, num_valid_tokens=None, **kw):
    """The layer with its first `blocks` blocks."""
    t, cfg = gp["t"], gp["cfg"]
    if num_valid_tokens is not None:
        kw["num_valid_tokens"] = torch.tensor([int(cfg.T * num_valid_tokens)], dtype=torch.int32, device="cuda")
    cut = lambda x: None if x is None else x[:blocks].contiguous()
    return mx.MoeBwd(t["hidden"], torch.from_numpy(gp["aff"]).cuda(), *weights, gp["tpid"][:blocks * cfg.B].contiguous(),
                     gp["b2e"][:blocks].contiguous(), t["dy"], cfg.B, cut(ckpt), down_proj_bias=t["b2"],
                     affinity_on=cfg.affinity_on, gate_up_checkpoint=None if ck8 is None else tuple(cut(x) for x in ck8), **kw)


def _runs(op, prior):
    """Two runs onto the same prior values (the same bits, but for the atomic bias sums)."""
    for k, v in op.out.items():
        if v is not None:
            v.copy_(prior[k]) if prior else v.fill_(torch.nan)
    op.workspace.fill_(0xC3)
    op.run()
    torch.cuda.synchronize()
    return {k: v.clone() for k, v in op.out.items() if v is not None}


def _same(cfg, got, ref, what):
    """db1 and db2 are atomic fp32 sums, whose order moves a term's rounding (2^-20 of the largest); each
    side may then round to the other bf16 neighbour, 2^-7 of the value."""
    for k in ("dx", "daff", "dwgu", "dwd"):
        assert torch.equal(got[k].view(torch.int16), ref[k].view(torch.int16)), (what, k)
    if cfg.has_bias:
        for k in ("db1", "db2"):
            a, b = got[k].float(), ref[k].float()
            assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -20 * b.abs().max()).all(), (what, k)


@pytest.mark.parametrize("option", list(OPTIONS))
@pytest.mark.parametrize("name", list(CFGS))
def test_fused_is_separate_bit_for_bit(name, option):
    """From bf16 and from e4m3 (whose padding holds NaN codes and scales), against the two
    kernels on the same layer without the blocks of padding; an e5m2 checkpoint takes the
    two kernels at any size."""
    cfg, N = CFGS[name]
    kw = OPTIONS[option]
    print("fused", name, option, flush=True)
    gp = gpu_problem(cfg, N=N)
    few = mx.moe_num_blocks(cfg.T, cfg.K, cfg.E, cfg.B)
    weights = _weights(gp, kw.get("fmt_weight", E4))
    geglu = kw.get("activation", 0)
    g = torch.Generator(device="cuda").manual_seed(1)
    prior = None
    if "accumulate" in kw:
        one = _bound(gp, weights, few, gp["t"]["ckpt"]).out
        prior = {k: torch.randn(v.shape, generator=g, device="cuda").to(v.dtype) for k, v in one.items() if v is not None}
    pad = ((gp["tpid"] < 0) | (gp["tpid"] >= cfg.T)).view(N, 1, 1, cfg.B)
    whole = pad.view(N, 1, 1, cfg.B // 32, 32).all(-1)
    for fmt in (E4, E5):
        _, codes, scales = mx.mxfp8_gated_act_fwd(gp["t"]["ckpt"], geglu, fmt, token_position_to_id=gp["tpid"], T=cfg.T)
        deq = torch.where(pad, torch.nan, _dequant(codes, scales, fmt))
        junk = torch.where(pad, torch.full_like(codes, 0x7f), codes), torch.where(whole, torch.full_like(scales, 255), scales)
        small = _bound(gp, weights, few, deq, **kw)
        assert not fused(small)
        ref = _runs(small, prior)
        assert all(v.isfinite().all() for v in ref.values())
        for what, op, is_fused in (("bf16", _bound(gp, weights, N, deq, **kw), True),
                                   ("8 bits", _bound(gp, weights, N, None, junk, fmt_checkpoint=fmt, **kw), fmt == E4),
                                   ("8 bits, separate", _bound(gp, weights, few, None, junk, fmt_checkpoint=fmt, **kw), False)):
            assert fused(op) == is_fused, what
            _same(cfg, _runs(op, prior), ref, (what, fmt))


@pytest.mark.parametrize("option", ["default", "geglu", "count", "grad_e4m3", "all_e5m2_count"])
@pytest.mark.parametrize("name", ["tiny", "bias", "i512_on_i"])
def test_fused_against_the_oracle(name, option):
    cfg, N = CFGS[name]
    kw = OPTIONS[option]
    print("fused oracle", name, option, flush=True)
    gp = gpu_problem(cfg, N=N)
    weights = _weights(gp, kw.get("fmt_weight", E4))
    op = _bound(gp, weights, N, gp["t"]["ckpt"], **kw)
    assert fused(op)
    out = _runs(op, None)
    p, _ = oracle_problem(gp)
    count = int(cfg.T * kw.get("num_valid_tokens", 1))
    wgu, wgu_s, wd, wd_s = (host(w) for w in weights)
    p = dataclasses.replace(p, tpid=np.where(p.tpid >= count, -1, p.tpid).astype(np.int32), wgu_codes=wgu, wgu_scales=wgu_s,
                            wd_codes=wd, wd_scales=wd_s, fmt_w=kw.get("fmt_weight", E4), fmt_act=kw.get("fmt_act", E4),
                            fmt_grad=kw.get("fmt_grad", E5), activation=kw.get("activation", 0))
    _check_outputs(cfg, out, oracle.moe_bwd(p), unrouted_zero=False)
    assert not out["dx"][count:].any() and not out["daff"].view(cfg.T, cfg.E)[count:].any()


# ----------------------------------------------------------------------------- the converters
# One expert, every slot a token in order, affinity 1, H = 128: dS is a sum of 128 exact
# products that fp32 holds exactly in any order (dY's values have 3 significant bits and
# W_down's codes 4, within few binades).  A gate of 64 has sigmoid 1 in fp32, so that
# inter = 64 u, dUp = bf16(64 dS) and, with u = 1, dGate = bf16(dS), without an error.
B, H, I = 128, 128, 512


def _layer(N, k, ckpt=None, ck8=None, fmt_grad=E5, fmt_act=E4, fmt_checkpoint=E4):
    """The bound layer and dS [slots, I] (float64), with dY times 2^k."""
    T = N * B
    rng = np.random.default_rng(17)
    few = np.array([0.0, 0.25, 0.3125, 0.375, 0.4375, 0.5, 0.625, 0.75, 0.875, 1.0, 1.25, 1.5, 1.75])
    dy = rng.choice(few, (T, H)) * rng.choice([-1, 1], (T, H))
    codes = rng.integers(0x30, 0x40, (1, I, H)).astype(np.uint8) | (rng.integers(0, 2, (1, I, H)).astype(np.uint8) << 7)
    w = oracle.dequantize(codes.reshape(I, H), np.full((I, H // 32), 127, np.uint8), 1, E4)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    u8 = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda")
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8, device="cuda")
    op = mx.MoeBwd(torch.ones(T, H, dtype=torch.bfloat16, device="cuda"), torch.ones(T, device="cuda"), u8(1, H, 2, I),
                   one(1, H, 2, I // 32), dev(codes), one(1, I, H // 32),
                   torch.arange(T, dtype=torch.int32, device="cuda"), torch.zeros(N, dtype=torch.int32, device="cuda"),
                   dev(dy * 2.0 ** k).to(torch.bfloat16), B, ckpt, gate_up_checkpoint=ck8, fmt_grad=fmt_grad,
                   fmt_act=fmt_act, fmt_checkpoint=fmt_checkpoint)
    return op, dy @ w.T * 2.0 ** k


def _operands(op, N):
    """The epilogue's operands as it left them: name -> (codes, scales), rows over the grouped axis."""
    op.workspace.fill_(0xC3)
    op.run()
    torch.cuda.synchronize()
    ws, L, P = op.workspace.cpu().numpy(), op.layout, N * B
    get = lambda n, rows, over: (stage_major_to_rows(ws[L[n + "_codes"]:][:rows * over], rows, over),
                                 pairs_to_rows(ws[L[n + "_scales"]:][:rows * over // 32], rows, over))
    return {"inter_tok": get("inter_tok", I, P), "dgu_tok": get("dgu_tok", 2 * I, P), "dgu_row": get("dgu_row", P, 2 * I)}


def _bf16_bits(x):
    """float64 -> bf16 bits: one rounding, half to even (the values are fp32 numbers)."""
    assert np.array_equal(x, x.astype(np.float32).astype(np.float64))
    return S.bf16_bits(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16))


def _expect(bits, fmt):
    return tuple(oracle.quantize(np.ascontiguousarray(bits), 1, fmt))


def _equal(got, want):
    for g, w in zip(got, want):
        assert np.array_equal(g, w.reshape(g.shape))


BLOCKS = {"separate": 8, "fused": 64}


@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("path", list(BLOCKS))
def test_encoded_gradients_at_scales_across_the_range(path, fmt):
    """dGate and dUp along both axes, bit for bit: groups whose largest value is past the format's
    (significands over 1.75) saturate there, from scales clamped at 2^-127 (e5m2) on."""
    N = BLOCKS[path]
    ck = torch.ones(N, 2, I, B, dtype=torch.bfloat16, device="cuda")
    ck[:, 0] = 64
    for k in (-116, -100, -40, 0, 40, 100):
        op, ds = _layer(N, k, ck, fmt_grad=fmt)
        assert fused(op) == (path == "fused")
        print("encode", path, fmt, k, flush=True)
        got = _operands(op, N)
        dgu = np.concatenate([_bf16_bits(ds), _bf16_bits(64 * ds)], 1)          # [P, 2I]
        row, tok = _expect(dgu, fmt), _expect(dgu.T, fmt)
        _equal(got["dgu_row"], row)
        _equal(got["dgu_tok"], tok)
        top = 0x7E if fmt == E4 else 0x7B
        assert ((row[0] & 0x7F) == top).mean() > 1e-3 and ((tok[0] & 0x7F) == top).mean() > 1e-3
        assert k > -116 or fmt == E4 or (row[1] == 0).any()
        assert np.array_equal(oracle.bf16_to_float(S.bf16_bits(op.out["daff"])), _daff(ds))


def _daff(ds):
    """d(affinity) = sum_i dS * 64, rounded once (the sums are exact)."""
    return oracle.bf16_to_float(_bf16_bits((ds * 64).sum(1)))


@pytest.mark.parametrize("order", ["ascending", "shuffled"])
@pytest.mark.parametrize("fmt", [E4, E5])
@pytest.mark.parametrize("path", list(BLOCKS))
def test_encoded_intermediate_of_every_bf16_pattern(path, fmt, order):
    """Ups of every bf16 magnitude below 2^100, both signs: in groups of neighbours, each is encoded at its own scale."""
    N = BLOCKS[path]
    bits = np.arange((127 + 100) << 7, dtype=np.uint16)
    bits = np.concatenate([bits, bits | 0x8000])
    if order == "shuffled":
        bits = np.random.default_rng(3).permutation(bits)
    u = np.resize(bits, N * I * B).reshape(N, I, B)
    ck = torch.full((N, 2, I, B), 64.0, dtype=torch.bfloat16, device="cuda")
    ck[:, 1] = S.from_bits(u, "cuda")
    op, _ = _layer(N, 0, ck, fmt_act=fmt)
    assert fused(op) == (path == "fused")
    inter = oracle.bf16_to_float(u).astype(np.float64) * 64
    want = _bf16_bits(inter.transpose(1, 0, 2).reshape(I, N * B))
    _equal(_operands(op, N)["inter_tok"], _expect(want, fmt))


@pytest.mark.parametrize("which", ["gate", "up"])
@pytest.mark.parametrize("path,fmt", [("separate", E4), ("fused", E4), ("separate", E5), ("large_e5m2", E5)])
def test_every_code_at_every_scale(path, fmt, which):
    """A checkpoint of every code at every scale byte from 0 to 254, in live slots (code 0 where
    bf16 does not hold the value), against the bf16 checkpoint of the same values, all operands
    bit for bit; and the intermediate of 64 times the ups against the definition."""
    N = BLOCKS.get(path, 64)
    codes = np.arange(256, dtype=np.uint8)
    codes = codes[(codes & 0x7F) != 0x7F] if fmt == E4 else codes[(codes & 0x7C) != 0x7C]
    rng = np.random.default_rng(fmt)
    c = np.resize(rng.permutation(np.repeat(codes, 4)), (N, I, B))
    # one scale for 32 rows and 32 slots (so that the groups along I keep to one size too), every byte in turn
    s = np.resize(np.arange(255, dtype=np.uint8), (N, I // 32, B // 32)).repeat(32, 1)
    v = np.asarray(oracle.dequantize(c.reshape(-1, B), s.reshape(-1, B // 32), 1, fmt), np.float64).reshape(c.shape)
    limit = 2.0 ** 121 if which == "up" else 2.0 ** 127                          # 64 u stays finite
    holds = (v == np.trunc(v / 2.0 ** -133) * 2.0 ** -133) & (np.abs(v) <= 1.75 * limit)
    c, v = np.where(holds, c, 0).astype(np.uint8), np.where(holds, v, 0.0)
    assert set(np.unique(s.repeat(32, 2)[(c & 0x7F) != 0])) >= {0, 1, 127, 240, 254}
    other = 0x38 if fmt == E4 else 0x3C                                          # 1.0
    const, cs = (1.0, 127) if which == "gate" else (64.0, 133)
    ck_c, ck_s = np.full((N, 2, I, B), other, np.uint8), np.full((N, 2, I, B // 32), cs, np.uint8)
    bf = torch.full((N, 2, I, B), const, dtype=torch.bfloat16, device="cuda")
    j = 0 if which == "gate" else 1
    ck_c[:, j], ck_s[:, j] = c, s
    exact = torch.from_numpy(v).to(torch.bfloat16)
    assert np.array_equal(exact.double().numpy(), v)
    bf[:, j] = exact.cuda()
    op8, _ = _layer(N, -8, None, (torch.from_numpy(ck_c).cuda(), torch.from_numpy(ck_s).cuda()), fmt_checkpoint=fmt)
    op16, _ = _layer(N, -8, bf)
    assert fused(op8) == (path == "fused")
    assert fused(op16) == (path != "separate")
    print("decode", path, fmt, which, flush=True)
    got, ref = _operands(op8, N), _operands(op16, N)
    for k in ref:
        _equal(got[k], ref[k])
    if which == "up":
        _equal(got["inter_tok"], _expect(_bf16_bits((v * 64).transpose(1, 0, 2).reshape(I, N * B)), E4))
