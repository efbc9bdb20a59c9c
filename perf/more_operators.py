"""What the MoE layer's forward and its neighbours are measured on: their plain forms, the calls a user makes of them,
and the cases.

  ffn      moe_fwd_mxfp8: the routed gated feed-forward block, both projections, activation and product from MXFP8
           operands, with the gate/up checkpoint that moe_bwd_mxfp8 reads, a residual and dropout
  tokens   moe_tokens_fwd_mxfp8: the same layer for few tokens, straight from the router's selections
  dropout  dropout_add / dropout_add_bwd: dropout from a counter-based generator whose mask is never stored
  weights  mxfp8_quantize_transposed: weights quantised along the axis that the forward contracts

`own` False computes the plain form with elementary torch operations; True calls the library.
"""
import math

import torch

own = False

SWIGLU, GEGLU = 0, 1
ON_H, ON_I = 0, 1
_EMAX, _MAX = 8, 448.0      # E4M3
_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # the smallest layer of the tests, evaluation: latency
        dict(name="ffn_tiny_T256_H128_I256_E4_top2", op="ffn", T=256, H=128, I=256, E=4, K=2, B=128, affinity_on=ON_H,
             activation=SWIGLU, bias=False, ckpt="none", p=0.0, residual=False, dropped=0.0),
        # the medium workload's training forward: 8-bit checkpoint, residual and dropout
        dict(name="ffn_medium_T8192_H2048_I1408_E16_top4_train", op="ffn", T=8192, H=2048, I=1408, E=16, K=4, B=512,
             affinity_on=ON_H, activation=SWIGLU, bias=False, ckpt="mxfp8", p=0.1, residual=True, dropped=0.0),
        # the fine-grained workload's training forward: many small experts, biases, bf16 checkpoint
        dict(name="ffn_fine_T32768_H1536_I256_E128_top8_train", op="ffn", T=32768, H=1536, I=256, E=128, K=8, B=128,
             affinity_on=ON_H, activation=SWIGLU, bias=True, ckpt="bf16", p=0.0, residual=False, dropped=0.0),
        # the large workload's forward, affinity on the intermediate
        dict(name="ffn_large_T16384_H4096_I14336_E8_top2", op="ffn", T=16384, H=4096, I=14336, E=8, K=2, B=1024,
             affinity_on=ON_I, activation=SWIGLU, bias=False, ckpt="none", p=0.0, residual=False, dropped=0.0),
        # odd sizes: contractions that fill no whole tile, tokens without an expert, GeGLU
        dict(name="ffn_ragged_T1500_H608_I352_E6_top3_geglu", op="ffn", T=1500, H=608, I=352, E=6, K=3, B=256,
             affinity_on=ON_H, activation=GEGLU, bias=True, ckpt="bf16", p=0.2, residual=True, dropped=0.1),
        # decoding: one sequence in the fine-grained layer and in the large one
        dict(name="tokens_T1_H1536_I256_E128_top8", op="tokens", T=1, H=1536, I=256, E=128, K=8, affinity_on=ON_H,
             activation=SWIGLU, bias=True, residual=True),
        dict(name="tokens_T1_H4096_I14336_E8_top2", op="tokens", T=1, H=4096, I=14336, E=8, K=2, affinity_on=ON_I,
             activation=SWIGLU, bias=False, residual=True),
        # decoding: a batch of sequences
        dict(name="tokens_T200_H1536_I256_E128_top8", op="tokens", T=200, H=1536, I=256, E=128, K=8,
             affinity_on=ON_H, activation=GEGLU, bias=True, residual=True),
        # the residual branch's dropout: the large workload's rows, and an odd fp32 batch's backward
        dict(name="dropout_forward_16384x4096", op="dropout", rows=16384, cols=4096, dtype="bf16", p=0.1,
             residual=True, direction="forward"),
        dict(name="dropout_backward_5003x1501_fp32", op="dropout", rows=5003, cols=1501, dtype="fp32", p=0.25,
             residual=False, direction="backward"),
        # the medium workload's gate/up weights, once a training step
        dict(name="weights_E16_H2048_2I2816", op="weights", G=16, R=2048, C=2816),
        # a router-sized weight, odd columns
        dict(name="weights_G1_R608_C77", op="weights", G=1, R=608, C=77),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "tokens", "tokens", "dropout", "weights"])
    if op == "dropout":
        cols = _log(rng, 1, 8192)
        return dict(op=op, rows=min(_log(rng, 1, 65536), (1 << 26) // cols), cols=cols, dtype=rng.choice(["fp32", "bf16"]),
                    p=rng.choice([0.05, 0.1, 0.25, 0.5]), residual=rng.random() < 0.5,
                    direction=rng.choice(["forward", "backward"]))
    if op == "weights":
        G, R = _log(rng, 1, 64), 32 * _log(rng, 1, 128)
        return dict(op=op, G=G, R=R, C=min(_log(rng, 1, 8192), max(1, (1 << 27) // (G * R))))
    E = _log(rng, 1, 64)
    c = dict(op=op, H=32 * _log(rng, 2, 96), I=32 * _log(rng, 1, 64), E=E, K=rng.randint(1, min(E, 8)),
             affinity_on=rng.choice([ON_H, ON_I]), activation=rng.choice([SWIGLU, GEGLU]))
    c["bias"] = c["affinity_on"] == ON_H and rng.random() < 0.5
    c["residual"] = rng.random() < 0.5
    if op == "tokens":
        # pairs x weights: no more than the plain form can hold
        most = (1 << 31) // (c["K"] * 3 * c["H"] * c["I"])
        return dict(c, T=max(1, min(_log(rng, 1, 256), most)))
    return dict(c, T=max(c["E"], _log(rng, 32, 8192)), B=rng.choice([128, 256, 512]),
                ckpt=rng.choice(["none", "bf16", "mxfp8"]), p=rng.choice([0.0, 0.1]), dropped=rng.choice([0.0, 0.1]))


def work(case):
    c = case
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        return {"bytes": n * (4 if c["dtype"] == "fp32" else 2) * (3 if c["residual"] and c["direction"] == "forward" else 2),
                "flops": 2 * n}
    if c["op"] == "weights":
        n = c["G"] * c["R"] * c["C"]
        return {"bytes": n * (3 + 1 / 32), "flops": 2 * n}
    T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["K"]
    experts = min(E, T * K)   # with tokens
    b = T * H * (6 if c["residual"] else 4) + T * K * 8 + experts * 3 * H * I * (1 + 1 / 32)
    if c["bias"]:
        b += experts * (2 * I + H) * 2
    if c["op"] == "ffn":
        b += T * K * I * {"none": 0, "bf16": 4, "mxfp8": 2.0625}[c["ckpt"]]
    return {"bytes": b, "flops": 6 * T * K * H * I}


# ----------------------------------------------------------------------------- inputs
def _mx_encode(x):
    """fp32 values (groups of 32 along the last axis) -> (E4M3 code values, E8M0 bytes)."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = g.abs().amax(-1, keepdim=True)
    X = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - _EMAX, -127).clamp(-127, 127)
    y = (g * torch.exp2(-X.float())).clamp(-_MAX, _MAX)
    return y.to(torch.float8_e4m3fn).reshape(x.shape), (X.squeeze(-1) + 127).to(torch.uint8)


def _mx_values(codes, scales):
    """The fp32 values that codes (E4M3 or their bytes) and E8M0 bytes stand for."""
    v = codes.view(torch.float8_e4m3fn).float()
    s = torch.exp2(scales.float() - 127.0)
    return (v.reshape(*scales.shape, 32) * s.unsqueeze(-1)).reshape(v.shape)


def prepare(case, seed):
    c = case
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def rand(*shape, sigma=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * sigma).to(torch.bfloat16)

    if c["op"] == "weights":
        return dict(case=c, w=rand(c["G"], c["R"], c["C"], sigma=0.02))
    rng = torch.randint(0, 2 ** 62, (2,), generator=gen, device=dev, dtype=torch.int64)   # seed, offset
    if c["op"] == "dropout":
        shape = (c["rows"], c["cols"])
        x = torch.randn(shape, generator=gen, device=dev).to(_DT[c["dtype"]])
        r = torch.randn(shape, generator=gen, device=dev).to(_DT[c["dtype"]]) if c["residual"] else None
        return dict(case=c, x=x, residual=r, rng=rng)
    T, H, I, E, K = (c[k] for k in "THIEK")
    # the router's answer, with experts of uneven load
    z = torch.randn(T, E, generator=gen, device=dev) - 0.5 * torch.log(torch.arange(1.0, E + 1, device=dev))
    score, idx = torch.topk(torch.softmax(z, 1), K, dim=1)
    s = dict(case=c, x=rand(T, H), rng=rng, residual=rand(T, H) if c["residual"] else None, b1=None, b2=None)
    if c["bias"]:
        s["b1"], s["b2"] = rand(E, 2, I, sigma=0.1), rand(E, H, sigma=0.1)
    wgu, s["wgu_s"] = _mx_encode(rand(E, 2, I, H, sigma=1 / math.sqrt(H)).float())
    wd, s["wd_s"] = _mx_encode(rand(E, H, I, sigma=1 / math.sqrt(I)).float())
    s["wgu"], s["wd"] = wgu.view(torch.uint8), wd.view(torch.uint8)
    if c["op"] == "tokens":
        return dict(s, idx=idx.to(torch.int32).contiguous(), scores=score.contiguous())
    # over capacity: selections, and with them some tokens' last one, dropped
    live = torch.rand(T, K, generator=gen, device=dev) >= c["dropped"]
    s["aff"] = torch.zeros(T, E, device=dev).scatter_(1, idx, torch.where(live, score, 0.0)).reshape(-1)
    # blocks of B slots: expert after expert, tokens ascending, -1 in the padding
    B = c["B"]
    N = (max(T * K - (E - 1), 1) + B - 1) // B + E - 1
    flat = torch.where(live, idx, E).reshape(-1)
    order = torch.argsort(flat, stable=True)
    n = torch.bincount(flat, minlength=E + 1)
    nb = (n[:E] + B - 1) // B
    start = torch.cat([(torch.cumsum(nb, 0) - nb) * B, torch.tensor([N * B], device=dev)])   # the dropped ones: past the end
    at = start[flat[order]] + torch.arange(T * K, device=dev) - (torch.cumsum(n, 0) - n)[flat[order]]
    tpid = torch.full((N * B + T * K,), -1, dtype=torch.int32, device=dev)
    tpid[at] = (order // K).to(torch.int32)
    s["tpid"] = tpid[: N * B].clone()
    s["b2e"] = torch.full((N,), E - 1, dtype=torch.int32, device=dev)
    used = torch.repeat_interleave(torch.arange(E, device=dev), nb)
    s["b2e"][: used.numel()] = used.to(torch.int32)
    return s


# ----------------------------------------------------------------------------- plain forms
def _act(g, activation):
    if activation == SWIGLU:
        return g / (1 + torch.exp(-g))
    return g * 0.5 * torch.erfc(-g / math.sqrt(2.0))


def _requant(x):
    codes, scales = _mx_encode(x)
    return _mx_values(codes, scales)


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _keep(rows, cols, p, rng):
    """The mask [rows, cols]: 16 bits an element of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random
    numbers: as easy as 1, 2, 3", 2011), eight elements a counter, the counter (element / 8, offset), the key the seed."""
    low = 0xFFFFFFFF
    n = rows * cols
    g = torch.arange((n + 7) // 8, device=rng.device, dtype=torch.int64)
    x0, x1 = g & low, g >> 32
    x2, x3 = (rng[1] & low).expand_as(g), ((rng[1] >> 32) & low).expand_as(g)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        a, b = x0 * 0xD2511F53, x2 * 0xCD9E8D57     # products modulo 2^64
        x0, x1, x2, x3 = ((b >> 32) & low) ^ x1 ^ k0, b & low, ((a >> 32) & low) ^ x3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([x0, x1, x2, x3], 1)
    bits = torch.stack([words & 0xFFFF, words >> 16], 2).reshape(-1)[:n]
    return (bits >= _threshold(p)).reshape(rows, cols)


def _drop(x, p, rng):
    """x (fp32 or fp64 [rows, cols]) with its dropped elements 0 and the others scaled."""
    t = _threshold(p)
    return torch.where(_keep(*x.shape, p, rng), x * (65536.0 / (65536 - t)), 0.0)


def _plain_dropout(s):
    c = s["case"]
    y = _drop(s["x"].float(), c["p"], s["rng"])
    if s["residual"] is not None and c["direction"] == "forward":
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def _plain_weights(s):
    codes, scales = _mx_encode(s["w"].float().transpose(1, 2).contiguous())
    return codes, scales


def _plain_ffn(s):
    c = s["case"]
    T, H, I, E, B = (c[k] for k in "THIEB")
    N = s["b2e"].numel()
    e = s["b2e"].long()
    tok = s["tpid"].long().reshape(N, B)
    ok = (tok >= 0)[:, :, None]
    tok = tok.clamp(min=0)
    a = torch.where(ok, s["aff"].reshape(T, E)[tok, e[:, None]][:, :, None], 0.0)
    wgu = _mx_values(s["wgu"], s["wgu_s"]).reshape(E, 2 * I, H).transpose(1, 2).contiguous()
    x = torch.where(ok, _requant(s["x"].float())[tok], 0.0)
    gu = torch.bmm(x, wgu[e])                                                # [N, B, 2I]
    del wgu, x
    if c["bias"]:
        gu = gu + s["b1"].float().reshape(E, 1, 2 * I)[e]
    gu = torch.where(ok, gu, 0.0)
    out = []
    if c["ckpt"] != "none":
        ck = gu.reshape(N, B, 2, I).permute(0, 2, 3, 1).contiguous().to(torch.bfloat16)
        if c["ckpt"] == "bf16":
            out = [ck]
        else:
            codes, scales = _mx_encode(ck.float())
            out = [codes, scales.view(torch.float8_e8m0fnu)]
    inter = _act(gu[:, :, :I], c["activation"]) * gu[:, :, I:]
    del gu
    if c["affinity_on"] == ON_I:
        inter = inter * a
    wd = _mx_values(s["wd"], s["wd_s"]).transpose(1, 2).contiguous()         # [E, I, H]
    y = torch.bmm(_requant(inter), wd[e])
    del wd, inter
    if c["bias"]:
        y = y + s["b2"].float().reshape(E, 1, H)[e]
    if c["affinity_on"] == ON_H:
        y = y * a
    y = torch.where(ok, y, 0.0)
    y = torch.zeros(T, H, device=y.device).index_add_(0, tok.reshape(-1), y.reshape(N * B, H))
    if c["p"]:
        y = _drop(y, c["p"], s["rng"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.to(torch.bfloat16)] + out


def _plain_tokens(s):
    c = s["case"]
    T, H, I, E, K = (c[k] for k in "THIEK")
    e = s["idx"].long().reshape(-1)
    a = s["scores"].reshape(T * K, 1)
    x = _requant(s["x"].float())[:, None].expand(T, K, H).reshape(T * K, H, 1)
    gu = torch.bmm(_mx_values(s["wgu"].reshape(E, 2 * I, H)[e], s["wgu_s"].reshape(E, 2 * I, H // 32)[e]), x)[:, :, 0]
    if c["bias"]:
        gu = gu + s["b1"].float().reshape(E, 2 * I)[e]
    inter = _act(gu[:, :I], c["activation"]) * gu[:, I:]
    if c["affinity_on"] == ON_I:
        inter = inter * a
    y = torch.bmm(_mx_values(s["wd"][e], s["wd_s"][e]), _requant(inter)[:, :, None])[:, :, 0]
    if c["bias"]:
        y = y + s["b2"].float()[e]
    if c["affinity_on"] == ON_H:
        y = y * a
    y = y.reshape(T, K, H).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(torch.bfloat16)


# ----------------------------------------------------------------------------- one pass
def run(state):
    s = state
    c = s["case"]
    if own:
        import mxfp8_grouped_gemm_amd as mx
        if c["op"] == "dropout":
            if c["direction"] == "forward":
                return mx.dropout_add(s["x"], c["p"], s["rng"], residual=s["residual"])
            return mx.dropout_add_bwd(s["x"], c["p"], s["rng"])
        if c["op"] == "weights":
            codes, scales = mx.mxfp8_quantize_transposed(s["w"])
            return codes.view(torch.float8_e4m3fn), scales
        if c["op"] == "tokens":
            return mx.moe_tokens_fwd_mxfp8(s["x"], s["idx"], s["scores"], s["wgu"], s["wgu_s"], s["wd"], s["wd_s"],
                                           gate_up_bias=s["b1"], down_bias=s["b2"], affinity_on=c["affinity_on"],
                                           activation=c["activation"], residual=s["residual"])
        r = mx.moe_fwd_mxfp8(s["x"], s["aff"], s["wgu"], s["wgu_s"], s["wd"], s["wd_s"], s["tpid"], s["b2e"], c["B"],
                             gate_up_bias=s["b1"], down_bias=s["b2"], affinity_on=c["affinity_on"],
                             activation=c["activation"], checkpoint=None if c["ckpt"] == "none" else c["ckpt"],
                             residual=s["residual"], dropout_p=c["p"], dropout_rng=s["rng"])
        if c["ckpt"] == "none":
            return [r["out"]]
        if c["ckpt"] == "bf16":
            return [r["out"], r["checkpoint"]]
        codes, scales = r["checkpoint"]
        return [r["out"], codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)]
    return {"ffn": _plain_ffn, "tokens": _plain_tokens, "dropout": _plain_dropout, "weights": _plain_weights}[c["op"]](s)


# ----------------------------------------------------------------------------- in 64 bits
def _exact_scale(x):
    """2^X of each group of 32 (x float64, groups along the last axis), [..., n/32, 1]."""
    top = x.unflatten(-1, (-1, 32)).abs().max(-1, keepdim=True).values
    return torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))).clamp(min=-127.0 + _EMAX) - _EMAX)


def _exact_mx(x):
    """x (float64) through MXFP8: nearest-even to 4 significant bits, steps no finer than 2^-9, in units of the scale."""
    s = _exact_scale(x)
    y = x.unflatten(-1, (-1, 32)) / s
    q = torch.exp2(((torch.frexp(y).exponent - 1).clamp(min=-6) - 3).double())
    return ((torch.round(y / q) * q).clamp(-_MAX, _MAX) * s).flatten(-2)


def _exact_values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
    return (v * torch.exp2(scales.double() - 127).unsqueeze(-1)).flatten(-2)


def _exact_expert(s, q, xq, a):
    """Expert q on rows xq [n, H] with affinities a [n, 1]: (gate and up [n, 2, I], its share of y [n, H])."""
    c = s["case"]
    gu = (xq @ _exact_values(s["wgu"][q], s["wgu_s"][q]).flatten(0, 1).T).unflatten(1, (2, -1))
    if s["b1"] is not None:
        gu = gu + s["b1"][q].double()
    g, u = gu[:, 0], gu[:, 1]
    h = (g * torch.sigmoid(g) if c["activation"] == SWIGLU else g * torch.special.ndtr(g)) * u
    if c["affinity_on"] == ON_I:
        h = h * a
    y = _exact_mx(h) @ _exact_values(s["wd"][q], s["wd_s"][q]).T
    if s["b2"] is not None:
        y = y + s["b2"][q].double()
    return gu, (y * a if c["affinity_on"] == ON_H else y)


def _exact_keep(rows, cols, p, rng):
    """The mask, counter by counter of the generator's definition in numpy's unsigned arithmetic."""
    import numpy as np
    seed, off = (int(v) & (2 ** 64 - 1) for v in rng.tolist())
    n = rows * cols
    i = np.arange((n + 7) // 8, dtype=np.uint64)
    m32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [i & m32, i >> sh, np.full_like(i, off & 0xFFFFFFFF), np.full_like(i, off >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        hi0, lo0 = (c[0] * np.uint64(0xD2511F53)) >> sh, (c[0] * np.uint64(0xD2511F53)) & m32
        hi1, lo1 = (c[2] * np.uint64(0xCD9E8D57)) >> sh, (c[2] * np.uint64(0xCD9E8D57)) & m32
        c = [hi1 ^ c[1] ^ np.uint64(key[0]), lo1, hi0 ^ c[3] ^ np.uint64(key[1]), lo0]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    half = np.stack([w >> np.uint64(16 * h) & np.uint64(0xFFFF) for w in c for h in (0, 1)], 1).reshape(-1)[:n]
    return torch.from_numpy(half >= np.uint64(_threshold(p))).reshape(rows, cols).to(rng.device)


def _exact_drop(x, p, rng):
    t = _threshold(p)
    return torch.where(_exact_keep(*x.shape, p, rng), x / (1 - t / 65536), 0.0)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "weights":
        w = s["w"].double().transpose(1, 2).contiguous()
        return (_exact_mx(w).unflatten(-1, (-1, 32)) / _exact_scale(w)).flatten(-2), None
    if c["op"] == "dropout":
        y = _exact_drop(s["x"].double(), c["p"], s["rng"])
        return y + s["residual"].double() if s["residual"] is not None and c["direction"] == "forward" else y
    T, H, I, E, K = (c[k] for k in "THIEK")
    dev = s["x"].device
    xq = _exact_mx(s["x"].double())
    y = torch.zeros(T, H, dtype=torch.float64, device=dev)
    if c["op"] == "tokens":
        for q in torch.unique(s["idx"]).tolist():
            t, k = torch.nonzero(s["idx"] == q, as_tuple=True)
            y[t] += _exact_expert(s, q, xq[t], s["scores"][t, k].double()[:, None])[1]
        return y + s["residual"].double() if s["residual"] is not None else y
    B = c["B"]
    slots = s["tpid"].reshape(-1, B).long()
    keep = c["ckpt"] == "bf16"
    ck = torch.zeros(slots.shape[0], 2, I, B, dtype=torch.float64, device=dev) if keep else None
    for q in range(E):
        for part in torch.nonzero((s["b2e"] == q) & (slots >= 0).any(1))[:, 0].split(4096 // min(B, 4096)):
            t = slots[part].reshape(-1)
            ok = t >= 0
            gu, z = _exact_expert(s, q, xq[t[ok]], s["aff"].reshape(T, E)[t[ok], q].double()[:, None])
            y.index_add_(0, t[ok], z)
            if keep:
                full = torch.zeros(t.numel(), 2, I, dtype=torch.float64, device=dev)
                full[ok] = gu
                ck[part] = full.unflatten(0, (-1, B)).permute(0, 2, 3, 1)
    if c["p"]:
        y = _exact_drop(y, c["p"], s["rng"])
    if s["residual"] is not None:
        y = y + s["residual"].double()
    if c["ckpt"] == "none":
        return [y]
    if keep:
        return [y, ck]
    # the 8-bit checkpoint is taken from the bf16 one, whose rounding may move a group's scale to the next power of two
    # and a code to its neighbour: the formulas in 64 bits have no value in their place
    return [y, None, None]
