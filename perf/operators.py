"""What the operators beside the MoE backward are measured on: their plain forms,
the calls a user makes of them, and the cases.

  router    moe_router_fwd: top-k routing of a batch of router logits
  balance   moe_balance_loss (and moe_balance_loss_bwd): the load-balance and z
            losses, per-expert counts, and the logits' gradient
  act       mxfp8_gated_act_fwd / _bwd: the gated activation that keeps its
            gate/up checkpoint in MXFP8, and its backward from that checkpoint
  moe       moe_bwd_mxfp8 from an MXFP8 gate/up checkpoint

`own` False computes the plain form with elementary torch operations; True calls
the library.
"""
import math

import torch

own = False

SOFTMAX_OVER_TOPK, TOPK_OVER_SOFTMAX, TOPK = 0, 1, 2
SWIGLU, GEGLU = 0, 1
E4M3, E5M2 = 0, 1
_EMAX = (8, 15)
_MAX = (448.0, 57344.0)
_F8 = (torch.float8_e4m3fn, torch.float8_e5m2)
_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------- the cases
def listed():
    return [
        # the smallest MoE layer of the tests, one routing call: latency
        dict(name="router_tiny_T256_E4_top2", op="router", T=256, E=4, K=2, mode=SOFTMAX_OVER_TOPK, renorm=False,
             dtype="fp32", masked=0.0, closed=0.0),
        # the fine-grained workload's router, probabilities renormalised over the selection
        dict(name="router_fine_T32768_E128_top8", op="router", T=32768, E=128, K=8, mode=TOPK_OVER_SOFTMAX,
             renorm=True, dtype="fp32", masked=0.0, closed=0.0),
        # a padded bf16 batch, odd sizes, some experts closed to some tokens
        dict(name="router_ragged_T5003_E60_top6_bf16", op="router", T=5003, E=60, K=6, mode=TOPK_OVER_SOFTMAX,
             renorm=False, dtype="bf16", masked=0.1, closed=0.05),
        # the large workload's router: an evaluation step that only logs losses and loads
        dict(name="balance_forward_large_T16384_E8", op="balance", T=16384, E=8, K=2, S=1, dtype="fp32", masked=0.0,
             closed=0.0, direction="forward"),
        # a training step on packed sequences, the loss per sequence
        dict(name="balance_step_fine_T32768_E128_S16", op="balance", T=32768, E=128, K=8, S=16, dtype="fp32",
             masked=0.0, closed=0.0, direction="step"),
        # a training step on a padded bf16 batch
        dict(name="balance_step_ragged_T5003_E60_S7_bf16", op="balance", T=5003, E=60, K=6, S=7, dtype="bf16",
             masked=0.1, closed=0.05, direction="step"),
        # the dense FFN beside the 4096-wide dense backward: forward
        dict(name="act_forward_dense_M4096_I4096", op="act", R=4096, I=1, B=4096, pad=0.0, activation=SWIGLU,
             fmt=E4M3, direction="forward"),
        # the medium MoE workload's blocks, a tenth of the slots padding: forward
        dict(name="act_forward_moe_N76_I1408_B512", op="act", R=76, I=1408, B=512, pad=0.1, activation=SWIGLU,
             fmt=E4M3, direction="forward"),
        # the fine-grained MoE workload's blocks: backward
        dict(name="act_backward_moe_N2175_I256_B128", op="act", R=2175, I=256, B=128, pad=0.05, activation=SWIGLU,
             fmt=E4M3, direction="backward"),
        # a short GeGLU batch with odd sizes and the wide-range format: backward, latency
        dict(name="act_backward_dense_M77_I352_geglu", op="act", R=77, I=1, B=352, pad=0.0, activation=GEGLU,
             fmt=E5M2, direction="backward"),
        # the whole layer's backward from the 8-bit checkpoint: the smallest layer, and the medium workload
        dict(name="moe_tiny_T256_H128_I256_E4", op="moe", T=256, H=128, I=256, E=4, K=2, B=128, affinity_on=0,
             activation=SWIGLU),
        dict(name="moe_medium_T8192_H2048_I1408_E16", op="moe", T=8192, H=2048, I=1408, E=16, K=4, B=512,
             affinity_on=0, activation=SWIGLU),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "balance", "act", "moe"])
    if op in ("router", "balance"):
        E = _log(rng, 2, 256)
        # tokens x experts up to the fine-grained workload's
        T = min(_log(rng, 1, 65536), 32768 * 128 // E)
        K = rng.randint(1, min(E, 8))
        c = dict(op=op, T=T, E=E, K=K, dtype=rng.choice(["fp32", "bf16"]), masked=rng.choice([0.0, 0.1, 0.5]),
                 closed=rng.choice([0.0, 0.05]))
        if op == "router":
            c["mode"] = rng.choice([SOFTMAX_OVER_TOPK, TOPK_OVER_SOFTMAX, TOPK])
            c["renorm"] = c["mode"] == TOPK_OVER_SOFTMAX and rng.random() < 0.5
        else:
            c["S"] = min(_log(rng, 1, 64), T)
            c["direction"] = rng.choice(["forward", "step"])
        return c
    if op == "act":
        c = dict(op=op, activation=rng.choice([SWIGLU, GEGLU]), fmt=rng.choice([E4M3, E5M2]),
                 direction=rng.choice(["forward", "backward"]))
        if rng.random() < 0.5:   # a dense FFN's rows
            c.update(R=_log(rng, 1, 8192), I=1, B=32 * _log(rng, 1, 128), pad=0.0)
        else:                    # a MoE layer's blocks
            c.update(I=32 * _log(rng, 1, 44), B=rng.choice([128, 256, 512, 1024]), pad=rng.choice([0.0, 0.1, 0.5]))
            c["R"] = _log(rng, 1, max(1, min(2048, (1 << 26) // (c["I"] * c["B"]))))
        return c
    E = _log(rng, 2, 16)
    H, I = 32 * _log(rng, 4, 64), 32 * _log(rng, 2, 44)
    return dict(op="moe", T=_log(rng, 32, 4096), H=H, I=I, E=E, K=rng.randint(1, min(E, 4)),
                B=rng.choice([128, 256, 512]), affinity_on=rng.randint(0, 1), activation=rng.choice([SWIGLU, GEGLU]))


def work(case):
    c = case
    if c["op"] in ("router", "balance"):
        T, E, K = c["T"], c["E"], c["K"]
        size = 4 if c["dtype"] == "fp32" else 2
        mask = T if c["masked"] else 0
        if c["op"] == "router":   # logits in; ids, scores and the masked affinities out
            return {"bytes": T * E * size + mask + T * K * 8 + T * E * 4, "flops": 4 * T * E}
        b = T * E * size + mask + T * K * 4 + c["S"] * E * 4
        if c["direction"] == "step":
            b += T * E * 4
        return {"bytes": b, "flops": (4 if c["direction"] == "forward" else 10) * T * E}
    if c["op"] == "act":   # forward: 4 in, 2 + 2 + 2/32 out; backward: 2 + 2/32 + 2 in, 4 out
        n = c["R"] * c["I"] * c["B"]
        return {"bytes": n * 8.0625 + (4 * c["R"] * c["B"] if c["I"] > 1 else 0), "flops": 12 * n}
    T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["K"]
    slots = T * K
    return {"bytes": 3 * T * H * 2 + T * E * 6 + E * H * 3 * I * (1 + 1 / 32 + 2) + slots * 2 * I * (1 + 1 / 32),
            "flops": 12 * slots * H * I}


# ----------------------------------------------------------------------------- inputs
def _mx_encode(x, fmt):
    """fp32 values (groups of 32 along the last axis) -> (code values, E8M0 bytes)."""
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = g.abs().amax(-1, keepdim=True)
    X = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - _EMAX[fmt], -127).clamp(-127, 127)
    y = (g * torch.exp2(-X.float())).clamp(-_MAX[fmt], _MAX[fmt])
    return y.to(_F8[fmt]).reshape(x.shape), (X.squeeze(-1) + 127).to(torch.uint8)


def _mx_values(codes, scales, fmt):
    """The fp32 values that codes (a uint8 tensor) and their E8M0 bytes stand for."""
    v = codes.view(_F8[fmt]).float()
    s = torch.exp2(scales.float() - 127.0)
    return (v.reshape(*scales.shape, 32) * s.unsqueeze(-1)).reshape(v.shape)


def _logits(c, gen, dev):
    T, E = c["T"], c["E"]
    z = torch.randn(T, E, generator=gen, device=dev) * 1.5 + torch.randn(E, generator=gen, device=dev) * 0.5
    if c["closed"]:   # experts closed to a token; a token in 50 has none open
        shut = torch.rand(T, E, generator=gen, device=dev) < c["closed"]
        shut |= torch.rand(T, 1, generator=gen, device=dev) < 0.02
        z = z.masked_fill(shut, -math.inf)
    mask = None
    if c["masked"]:
        mask = torch.rand(T, generator=gen, device=dev) >= c["masked"]
        z = torch.where(mask[:, None], z, z * 100)   # padding tokens hold whatever was left there
    return z.to(_DT[c["dtype"]]), mask


def _tokens_of_blocks(R, B, pad, gen, dev):
    """[R*B] int32 slot -> token ids in turn; a share `pad` of the slots, at the
    blocks' ends, are padding (-1)."""
    live = (B * (1 - 2 * pad * torch.rand(R, 1, generator=gen, device=dev))).ceil().long()
    ok = (torch.arange(B, device=dev)[None, :] < live).reshape(-1)
    ids = torch.cumsum(ok.to(torch.int32), 0, dtype=torch.int32) - 1
    return torch.where(ok, ids, torch.full_like(ids, -1)), R * B


def prepare(case, seed):
    c = case
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    if c["op"] in ("router", "balance"):
        z, mask = _logits(c, gen, dev)
        s = dict(case=c, logits=z, mask=mask)
        if c["op"] == "balance":
            T, S = c["T"], c["S"]
            v, i = torch.topk(z.float(), c["K"], dim=1)
            i = torch.where(v > -math.inf, i, -1)
            i = torch.where(torch.rand(i.shape, generator=gen, device=dev) < 0.02, -1, i)   # over capacity: dropped
            s["idx"] = i.to(torch.int32).contiguous()
            s["seq"] = None
            if S > 1:
                cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), generator=gen, device=dev)).values
                ends = torch.tensor([T - T // 100], device=dev)   # the last hundredth lies behind the last sequence
                s["seq"] = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), cuts, ends]).clamp(max=int(ends)).to(torch.int32)
            s["dloss"] = torch.rand(2, generator=gen, device=dev) + 0.5
            s["coef"] = (0.01, 0.001)
        return s
    if c["op"] == "act":
        R, I, B = c["R"], c["I"], c["B"]
        shape = (R, 2, B) if I == 1 else (R, 2, I, B)
        s = dict(case=c, tpid=None, T=0)
        if I > 1:
            s["tpid"], s["T"] = _tokens_of_blocks(R, B, c["pad"], gen, dev)
        x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
        if c["direction"] == "forward":
            return dict(s, gate_up=x)
        codes, scales = _mx_encode(_masked(x.float(), s["tpid"], s["T"]), c["fmt"])
        d = torch.randn((R,) + shape[2:], generator=gen, device=dev, dtype=torch.bfloat16)
        return dict(s, codes=codes.view(torch.uint8), scales=scales, dinter=d)
    T, H, I, E, K, B = (c[k] for k in "THIEKB")
    z = torch.randn(T, E, generator=gen, device=dev) - 0.5 * torch.log(torch.arange(1.0, E + 1, device=dev))
    p, idx = torch.topk(torch.softmax(z, 1), K, dim=1)
    # blocks of B slots: expert after expert, tokens ascending, -1 in the padding
    flat = idx.reshape(-1)
    order = torch.argsort(flat, stable=True)
    n = torch.bincount(flat, minlength=E)
    nb = (n + B - 1) // B
    N = (max(T * K - (E - 1), 1) + B - 1) // B + E - 1
    first = torch.cumsum(nb, 0) - nb
    at = first[flat[order]] * B + torch.arange(T * K, device=dev) - (torch.cumsum(n, 0) - n)[flat[order]]
    tpid = torch.full((N * B,), -1, dtype=torch.int32, device=dev)
    tpid[at] = (order // K).to(torch.int32)
    b2e = torch.full((N,), E - 1, dtype=torch.int32, device=dev)
    used = torch.repeat_interleave(torch.arange(E, device=dev), nb)
    b2e[: used.numel()] = used.to(torch.int32)
    aff = torch.zeros(T, E, device=dev).scatter_(1, idx, p).reshape(-1)

    def rand(*shape, sigma=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * sigma).to(torch.bfloat16)

    wgu, wgu_s = _mx_encode(rand(E, H, 2, I, sigma=0.02).float(), E4M3)
    wd, wd_s = _mx_encode(rand(E, I, H, sigma=0.02).float(), E4M3)
    ck, ck_s = _mx_encode(_masked(rand(N, 2, I, B, sigma=0.02 * math.sqrt(H)).float(), tpid, T), E4M3)
    u8 = torch.uint8
    return dict(case=c, x=rand(T, H), aff=aff, wgu=wgu.view(u8), wgu_s=wgu_s, wd=wd.view(u8), wd_s=wd_s, tpid=tpid,
                b2e=b2e, dy=rand(T, H), ck=ck.view(u8), ck_s=ck_s)


# ----------------------------------------------------------------------------- plain forms
def _masked(x, tpid, T):
    """x [R, ..., B] with the slots of no token set to zero."""
    if tpid is None:
        return x
    B = x.shape[-1]
    ok = ((tpid >= 0) & (tpid < T)).reshape(-1, *([1] * (x.dim() - 2)), B)
    return torch.where(ok, x, torch.zeros((), device=x.device))


def _plain_router(z, mask, mode, renorm, K):
    z = z.float()
    if mask is not None:
        z = torch.where(mask[:, None], z, torch.full_like(z, -math.inf))
    v, idx = torch.sort(z, dim=1, descending=True, stable=True)   # ties: the lowest expert first
    v, idx = v[:, :K], idx[:, :K]
    open_ = v > -math.inf
    m = torch.where(open_[:, :1], v[:, :1], torch.zeros_like(v[:, :1]))
    e = torch.exp(v - m)
    if mode == SOFTMAX_OVER_TOPK or renorm:
        y = e / e.sum(1, keepdim=True)
    elif mode == TOPK_OVER_SOFTMAX:
        y = e / torch.exp(z - m).sum(1, keepdim=True)
    else:
        y = v
    y = torch.where(open_, y, torch.zeros_like(y))
    aff = torch.zeros_like(z).scatter_(1, idx, y)
    return torch.where(open_, idx, -1).to(torch.int32), y, aff.reshape(-1)


def _plain_balance(s):
    c = s["case"]
    T, E, K, S = c["T"], c["E"], c["K"], c["S"]
    z = s["logits"].float()
    dev = z.device
    seq = s["seq"] if s["seq"] is not None else torch.tensor([0, T], dtype=torch.int32, device=dev)
    seg = torch.searchsorted(seq, torch.arange(T, dtype=torch.int32, device=dev), right=True) - 1
    m = z.amax(1, keepdim=True)
    ok = (seg >= 0) & (seg < S) & (m[:, 0] > -math.inf)
    if s["mask"] is not None:
        ok = ok & s["mask"]
    z = torch.where(ok[:, None], z, torch.zeros_like(z))
    m = torch.where(ok[:, None], m, torch.zeros_like(m))
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    p = torch.where(ok[:, None], e / total, torch.zeros_like(e))
    lse = torch.where(ok, m[:, 0] + torch.log(total[:, 0]), torch.zeros_like(m[:, 0]))
    # sums over a sequence's tokens: differences of running sums, in 64 bits (whole numbers exactly)
    hit = (s["idx"][:, :, None] == torch.arange(E, device=dev)).sum(1)     # [T, E]: ids outside [0, E) count nowhere
    terms = torch.cat([p.double(), torch.where(ok[:, None], hit, 0).double(), ok[:, None].double()], 1)
    running = torch.cumsum(terms.t().contiguous(), 1)                      # [2E + 1, T]
    running = torch.cat([torch.zeros_like(running[:, :1]), running], 1)
    sums = (running[:, seq[1:].long()] - running[:, seq[:-1].long()]).t()
    psum, counts, n = sums[:, :E], sums[:, E:2 * E].to(torch.int32), sums[:, 2 * E].to(torch.int32)
    live, every = (n > 0).sum(), n.sum()
    num = torch.cat([n, live.reshape(1).to(torch.int32), every.reshape(1).to(torch.int32)])
    bal, zc = s["coef"]
    per = n.clamp(min=1).double()[:, None]
    w = bal * E * counts.double() / (K * per * per * live.clamp(min=1))
    loss = torch.stack([(w * psum).sum(), zc * lse.double().square().sum() / every.clamp(min=1)]).float()
    if c["direction"] == "forward":
        return loss, counts, num
    w = w.float()[torch.where(ok, seg, torch.zeros_like(seg))]
    d = p * (w - (w * p).sum(1, keepdim=True)) * s["dloss"][0]
    d = d + p * (2 * zc * s["dloss"][1] / every.clamp(min=1) * lse)[:, None]
    return loss, counts, num, d


def _act(g, activation):
    """act(g) and act'(g)."""
    if activation == SWIGLU:
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    cdf = 0.5 * torch.erfc(-g / math.sqrt(2.0))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _plain_act(s):
    c = s["case"]
    if c["direction"] == "forward":
        x = _masked(s["gate_up"].float(), s["tpid"], s["T"])
        a, _ = _act(x[:, 0], c["activation"])
        codes, scales = _mx_encode(x, c["fmt"])
        return (a * x[:, 1]).to(torch.bfloat16), codes, scales
    x = _mx_values(s["codes"], s["scales"], c["fmt"])
    d = _masked(s["dinter"].float(), s["tpid"], s["T"])
    a, da = _act(x[:, 0], c["activation"])
    return torch.stack([d * x[:, 1] * da, d * a], 1).to(torch.bfloat16)


def _bf(x):
    return x.to(torch.bfloat16).float()


def _requant(x, fmt):
    """x through MXFP8 (groups of 32 along the last axis) and back."""
    codes, scales = _mx_encode(x, fmt)
    return _mx_values(codes.view(torch.uint8), scales, fmt)


def _plain_moe(s):
    c = s["case"]
    T, H, I, E, B = (c[k] for k in "THIEB")
    N = s["b2e"].numel()
    e = s["b2e"].long()
    tok = s["tpid"].long().reshape(N, B)
    ok = (tok >= 0).float()[:, :, None]
    tok = tok.clamp(min=0)
    a = s["aff"].reshape(T, E)[tok, e[:, None]][:, :, None] * ok            # [N, B, 1]
    dy = s["dy"].float()
    wd = _mx_values(s["wd"], s["wd_s"], E4M3)                               # [E, I, H]
    wgu = _mx_values(s["wgu"], s["wgu_s"], E4M3)                            # [E, H, 2, I]
    ck = _mx_values(s["ck"], s["ck_s"], E4M3).permute(0, 1, 3, 2)           # [N, 2, B, I]
    ds = torch.bmm(_requant(dy, E5M2)[tok] * ok, wd[e].transpose(1, 2).contiguous())
    g, u = ck[:, 0] * ok, ck[:, 1] * ok
    act, dact = _act(g, c["activation"])
    act = _bf(act)
    inter = _bf(act * u)
    daff = (ds * inter).sum(2, keepdim=True)
    di = a * ds
    dgu = torch.stack([_bf(di * u * dact), _bf(di * act)], 2)               # [N, B, 2, I]
    dx_slot = torch.bmm(_requant(dgu, E5M2).reshape(N, B, 2 * I),
                        wgu[e].reshape(N, H, 2 * I).transpose(1, 2).contiguous())
    dx = torch.zeros(T, H, device=dy.device).index_add_(0, tok.reshape(-1), (dx_slot * ok).reshape(N * B, H))
    da = torch.zeros(T, E, device=dy.device).index_put_((tok, e[:, None].expand(N, B)), daff[:, :, 0], accumulate=True)
    xq = _requant((s["x"].float()[tok] * ok).transpose(1, 2), E4M3)         # [N, H, B]: groups along the slots
    gq = _requant(dgu.reshape(N, B, 2 * I).transpose(1, 2), E5M2)
    on_i = c["affinity_on"] == 1
    iq = _requant((_bf(a * inter) if on_i else inter).transpose(1, 2), E4M3)
    yq = _requant(((dy[tok] * ok) if on_i else _bf(a * dy[tok])).transpose(1, 2), E5M2)
    dwgu = torch.zeros(E, H, 2 * I, device=dy.device).index_add_(0, e, torch.bmm(xq, gq.transpose(1, 2).contiguous()))
    dwd = torch.zeros(E, I, H, device=dy.device).index_add_(0, e, torch.bmm(iq, yq.transpose(1, 2).contiguous()))
    b16 = torch.bfloat16
    return dx.to(b16), da.reshape(-1).to(b16), dwgu.reshape(E, H, 2, I).to(b16), dwd.to(b16)


# ----------------------------------------------------------------------------- one pass
def run(state):
    s = state
    c = s["case"]
    if own:
        import mxfp8_grouped_gemm_amd as mx
        if c["op"] == "router":
            return mx.moe_router_fwd(c["mode"], s["logits"], c["K"], renorm=c["renorm"], token_mask=s["mask"])
        if c["op"] == "balance":
            bal, zc = s["coef"]
            loss, counts, num = mx.moe_balance_loss(s["logits"], s["idx"], bal, zc, token_mask=s["mask"],
                                                    seq_starts=s["seq"])
            if c["direction"] == "forward":
                return loss, counts, num
            d = mx.moe_balance_loss_bwd(s["logits"], counts, num, c["K"], bal, zc, dloss=s["dloss"],
                                        token_mask=s["mask"], seq_starts=s["seq"])
            return loss, counts, num, d
        if c["op"] == "act":
            kw = dict(activation=c["activation"], fmt=c["fmt"], token_position_to_id=s["tpid"], T=s["T"])
            if c["direction"] == "forward":
                inter, codes, scales = mx.mxfp8_gated_act_fwd(s["gate_up"], **kw)
                return inter, codes.view(_F8[c["fmt"]]), scales
            return mx.mxfp8_gated_act_bwd(s["dinter"], s["codes"], s["scales"], **kw)
        g = mx.moe_bwd_mxfp8(s["x"], s["aff"], s["wgu"], s["wgu_s"], s["wd"], s["wd_s"], s["tpid"], s["b2e"], s["dy"],
                             c["B"], None, affinity_on=c["affinity_on"], activation=c["activation"],
                             gate_up_checkpoint=(s["ck"], s["ck_s"]))
        return g["dx"], g["daff"], g["dwgu"], g["dwd"]
    if c["op"] == "router":
        return _plain_router(s["logits"], s["mask"], c["mode"], c["renorm"], c["K"])
    if c["op"] == "balance":
        return _plain_balance(s)
    if c["op"] == "act":
        return _plain_act(s)
    return _plain_moe(s)


# ----------------------------------------------------------------------------- in 64 bits
def _round_to(x, bits, emin):
    """x (float64) rounded to nearest-even with `bits` significant bits, steps no finer than those of 2^emin."""
    e = torch.frexp(x).exponent - 1
    q = torch.exp2((e.clamp(min=emin) - (bits - 1)).double())
    return torch.round(x / q) * q


def _exact_mx(x, fmt):
    """x (float64) through MXFP8, groups of 32 along the last axis."""
    parts = x.unflatten(-1, (-1, 32))
    top = parts.abs().max(-1, keepdim=True).values
    X = torch.floor(torch.log2(top.clamp(min=1e-300))).clamp(min=-127 + _EMAX[fmt]) - _EMAX[fmt]
    s = torch.exp2(X)
    bits, emin = ((4, -6), (3, -14))[fmt]
    y = _round_to(parts / s, bits, emin).clamp(-_MAX[fmt], _MAX[fmt])
    return (y * s).flatten(-2)


def _exact_act(g, activation):
    return g * torch.sigmoid(g) if activation == SWIGLU else g * torch.special.ndtr(g)


def _exact_router(s):
    c = s["case"]
    z = s["logits"].double()
    if s["mask"] is not None:
        z = z.masked_fill(~s["mask"][:, None], -math.inf)
    top = torch.argsort(z, dim=1, descending=True, stable=True)[:, : c["K"]]
    chosen = torch.zeros_like(z, dtype=torch.bool).scatter_(1, top, True) & (z > -math.inf)
    if c["mode"] == TOPK:
        y = z
    elif c["mode"] == TOPK_OVER_SOFTMAX and not c["renorm"]:
        y = torch.softmax(z, 1)
    else:
        y = torch.softmax(z.masked_fill(~chosen, -math.inf), 1)
    y = torch.where(chosen, y, 0.0)
    return None, y.gather(1, top), y.reshape(-1)


def _exact_balance(s):
    c = s["case"]
    T, E, K, S = c["T"], c["E"], c["K"], c["S"]
    z = s["logits"].double()
    keep = (z > -math.inf).any(1)
    if s["mask"] is not None:
        keep = keep & s["mask"]
    bounds = [0, T] if s["seq"] is None else s["seq"].tolist()
    d = torch.zeros_like(z)
    total, rows = 0, []
    for q in range(S):
        r = torch.nonzero(keep[bounds[q]:bounds[q + 1]])[:, 0] + bounds[q]
        if r.numel():
            rows.append(r)
            total += r.numel()
    bal, zc = s["coef"]
    b, zz = torch.zeros((), dtype=torch.float64, device=z.device), torch.zeros((), dtype=torch.float64, device=z.device)
    for r in rows:
        x = z[r].requires_grad_(True)
        i = s["idx"][r].long()
        f = torch.bincount(i[(i >= 0) & (i < E)], minlength=E).double() / (K * r.numel())
        lb = bal * E * (f * torch.softmax(x, 1).mean(0)).sum() / len(rows)
        lz = zc * torch.logsumexp(x, 1).square().sum() / total
        (lb * s["dloss"][0].double() + lz * s["dloss"][1].double()).backward()
        d[r] = x.grad
        b, zz = b + lb.detach(), zz + lz.detach()
    out = (torch.stack([b, zz]), None, None)
    return out if c["direction"] == "forward" else out + (d,)


def _exact_of_act(s):
    c = s["case"]
    if c["direction"] == "forward":
        x = _masked(s["gate_up"].double(), s["tpid"], s["T"])
        parts = x.unflatten(-1, (-1, 32))
        top = parts.abs().max(-1, keepdim=True).values
        X = torch.where(top > 0, torch.floor(torch.log2(top.clamp(min=1e-300))) - _EMAX[c["fmt"]], -127.0).clamp(min=-127)
        bits, emin = ((4, -6), (3, -14))[c["fmt"]]
        y = _round_to(parts / torch.exp2(X), bits, emin).clamp(-_MAX[c["fmt"]], _MAX[c["fmt"]])
        return _exact_act(x[:, 0], c["activation"]) * x[:, 1], y.flatten(-2), None
    v = s["codes"].view(_F8[c["fmt"]]).double().unflatten(-1, (-1, 32))
    x = (v * torch.exp2(s["scales"].double() - 127).unsqueeze(-1)).flatten(-2).requires_grad_(True)
    d = _masked(s["dinter"].double(), s["tpid"], s["T"])
    (_exact_act(x[:, 0], c["activation"]) * x[:, 1] * d).sum().backward()
    return x.grad


def _exact_moe(s):
    """Expert by expert, the operands' roundings as the operator defines them."""
    c = s["case"]
    T, H, I, E, B = (c[k] for k in "THIEB")
    dev = s["dy"].device
    f64 = torch.float64

    def values(codes, scales):
        v = codes.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
        return (v * torch.exp2(scales.double() - 127).unsqueeze(-1)).flatten(-2)

    def b16(x):
        return _round_to(x, 8, -126)

    dy = s["dy"].double()
    dyq = _exact_mx(dy, E5M2)
    x = s["x"].double()
    dx = torch.zeros(T, H, dtype=f64, device=dev)
    da = torch.zeros(T, E, dtype=f64, device=dev)
    dwgu = torch.zeros(E, H, 2 * I, dtype=f64, device=dev)
    dwd = torch.zeros(E, I, H, dtype=f64, device=dev)
    slots = s["tpid"].reshape(-1, B).long()
    for q in range(E):
        blocks = torch.nonzero((s["b2e"] == q) & (slots >= 0).any(1))[:, 0]
        if not blocks.numel():
            continue
        t = slots[blocks].reshape(-1)
        ok = t >= 0
        t = t.clamp(min=0)
        a = torch.where(ok, s["aff"].reshape(T, E)[t, q].double(), 0.0)[:, None]
        ok = ok.double()[:, None]
        w_down, w_up = values(s["wd"][q], s["wd_s"][q]), values(s["wgu"][q], s["wgu_s"][q]).reshape(H, 2 * I)
        ck = values(s["ck"][blocks], s["ck_s"][blocks]).permute(1, 0, 3, 2).reshape(2, -1, I) * ok
        g, u = ck[0].clone().requires_grad_(True), ck[1]
        act = _exact_act(g, c["activation"])
        slope = torch.autograd.grad(act.sum(), g)[0]
        act = b16(act.detach())
        inter = b16(act * u)
        ds = (dyq[t] * ok) @ w_down.T
        da.index_put_((t, torch.full_like(t, q)), (ds * inter).sum(1), accumulate=True)
        dgu = torch.cat([b16(a * ds * u * slope), b16(a * ds * act)], 1)
        dx.index_add_(0, t, (_exact_mx(dgu, E5M2) @ w_up.T) * ok)
        left = _exact_mx((x[t] * ok).T.contiguous(), E4M3)
        dwgu[q] = left @ _exact_mx(dgu.T.contiguous(), E5M2).T
        if c["affinity_on"] == 1:
            dwd[q] = _exact_mx(b16(a * inter).T.contiguous(), E4M3) @ _exact_mx((dy[t] * ok).T.contiguous(), E5M2).T
        else:
            dwd[q] = _exact_mx(inter.T.contiguous(), E4M3) @ _exact_mx(b16(a * dy[t]).T.contiguous(), E5M2).T
    return dx, da.reshape(-1), dwgu.reshape(E, H, 2, I), dwd


def exact(case, seed):
    s = prepare(case, seed)
    return {"router": _exact_router, "balance": _exact_balance, "act": _exact_of_act, "moe": _exact_moe}[case["op"]](s)
