"""Layers of the MoE forward whose launches come near what a launch takes (2^32 threads: the runtime runs more of them
modulo 2^32, without an error), or near the documented limits of their sizes."""
import pytest
import torch

import mxfp8_grouped_gemm_amd as mx

pytestmark = pytest.mark.gpu


def test_small_layer_over_many_weight_rows():
    """Eight tokens of one block, and so many rows of weight scales that workgroups of 1024 threads would pass 2^32 threads:
    the last expert gives what it gives alone."""
    T, H, I, E, B = 8, 32, 2 ** 18, 512, 128
    print("small layer", T, H, I, E, flush=True)
    g = torch.Generator("cuda").manual_seed(4)

    def codes(*shape):
        c = torch.empty(shape, dtype=torch.uint8, device="cuda")
        for e in range(shape[0]):   # E4M3 of magnitude 0.5 to 0.94
            c[e] = torch.randint(0x30, 0x38, shape[1:], generator=g, device="cuda", dtype=torch.uint8)
        return c
    wgu, wd = codes(E, 2, I, H), codes(E, H, I)
    sgu = torch.randint(115, 120, (E, 2, I, H // 32), generator=g, device="cuda", dtype=torch.uint8)
    sd = torch.randint(115, 120, (E, H, I // 32), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    tpid = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    tpid[:T] = torch.arange(T, device="cuda")
    aff = torch.zeros(T, E, device="cuda")
    aff[:, -1] = 0.75

    def run(aff, weights, e):
        op = mx.MoeFwd(x, aff.reshape(-1), *weights, tpid, torch.full((1,), e, dtype=torch.int32, device="cuda"), B)
        op.workspace.fill_(255)      # scales of NaN where nothing is written
        return op.run()["out"]
    many = run(aff, (wgu, sgu, wd, sd), E - 1)
    one = run(aff[:, -1].contiguous(), [t[-1:].contiguous() for t in (wgu, sgu, wd, sd)], 0)
    torch.cuda.synchronize()
    assert not one.isnan().any() and one.float().norm() > 0 and torch.equal(many, one)


def test_tokens_of_the_longest_rows():
    """The most tokens of the longest rows (X of 2^30 elements, 2^17 workgroups of its quantisation): what each 64 of them
    give alone."""
    T, H, I = 256, 2 ** 22, 32
    print("tokens", T, H, I, flush=True)
    g = torch.Generator("cuda").manual_seed(6)
    w = [torch.randint(0x30, 0x38, s, generator=g, device="cuda", dtype=torch.uint8) for s in ((1, 2, I, H), (1, H, I))]
    for c in w:
        c |= torch.randint(0, 2, c.shape, generator=g, device="cuda", dtype=torch.uint8) << 7
    sgu = torch.randint(112, 118, (1, 2, I, H // 32), generator=g, device="cuda", dtype=torch.uint8)
    sd = torch.randint(120, 125, (1, H, I // 32), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    a = torch.rand(T, 1, generator=g, device="cuda")

    def run(r):
        return mx.moe_tokens_fwd_mxfp8(x[r], ids[r], a[r], w[0], sgu, w[1], sd)
    y = run(slice(0, T))
    for t in range(0, T, 64):
        part = run(slice(t, t + 64))
        assert part.any(1).all() and not part.isnan().any() and torch.equal(y[t:t + 64], part), t


def _weights(E, H, I, seed):
    """E experts with the codes of one."""
    g = torch.Generator("cuda").manual_seed(seed)

    def codes(*s):
        c = torch.randint(0x28, 0x38, s, generator=g, device="cuda", dtype=torch.uint8)
        return c | torch.randint(0, 2, s, generator=g, device="cuda", dtype=torch.uint8) << 7

    def scales(*s):
        return torch.randint(118, 122, s, generator=g, device="cuda", dtype=torch.uint8)
    one = codes(2, I, H), scales(2, I, H // 32), codes(H, I), scales(H, I // 32)
    return [t.unsqueeze(0).expand(E, *t.shape).contiguous() for t in one]


def test_most_tokens():
    """T just below 2^24 and T * 128 below 2^31: a range of the tokens by itself gives the same bits."""
    T, H, I, B = 16_700_000, 32, 32, 128
    print("tokens", T, H, I, flush=True)
    g = torch.Generator("cuda").manual_seed(7)
    x = torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16)
    aff = torch.rand(T, generator=g, device="cuda")
    w = _weights(1, H, I, 8)

    def run(a, b):
        n = b - a
        N = -(-n // B)
        tpid = torch.full((N * B,), -1, dtype=torch.int32, device="cuda")
        tpid[:n] = torch.arange(n, dtype=torch.int32, device="cuda")
        op = mx.MoeFwd(x[a:b].contiguous(), aff[a:b].contiguous(), *w, tpid,
                       torch.zeros(N, dtype=torch.int32, device="cuda"), B, checkpoint="mxfp8")
        for t in (op.out["out"], *op.out["checkpoint"]):
            t.fill_(77)
        return op.run()
    whole = run(0, T)
    n = 1 << 18
    for a in (0, T // 2 // B * B, (T - n) // B * B):   # the last one to the end, with a block partly filled
        b = min(a + n + B, T)
        part = run(a, b)
        torch.cuda.synchronize()
        assert part["out"].any() and torch.equal(part["out"], whole["out"][a:b]), a
        for p, q in zip(part["checkpoint"], whole["checkpoint"]):
            assert torch.equal(p, q[a // B:-(-b // B)]), a


# name: sizes of a layer in which every token goes to all of 8 experts, and which operand passes 2^32 bytes
FAR = {
    "s_short_contraction": (64, 2176, 2 ** 18),      # fp16 rows
    "s_long_contraction": (64, 4224, 2 ** 17),       # fp32 rows, Phase 3's kernel
    "x_by_slot": (4224, 8224, 2 ** 17),              # X in the slots' order, s and the fp16 rows as well
}


@pytest.mark.parametrize("name", FAR)
def test_operands_past_32_bits(name):
    """The same 1024 tokens over and over: what they give once."""
    H, I, T = FAR[name]
    E, B, n = 8, 1024, 1024
    print(name, T, H, I, flush=True)
    assert T * E * (H if name == "x_by_slot" else I) > 1 << 32
    g = torch.Generator("cuda").manual_seed(9)
    x = torch.randn(n, H, generator=g, device="cuda", dtype=torch.bfloat16)
    aff = torch.rand(n, E, generator=g, device="cuda")
    w = _weights(E, H, I, 10)

    def run(times):
        t = n * times
        tpid = torch.arange(t, dtype=torch.int32, device="cuda").repeat(E)
        b2e = torch.arange(E, dtype=torch.int32, device="cuda").repeat_interleave(t // B)
        y = mx.moe_fwd_mxfp8(x.repeat(times, 1), aff.repeat(times, 1).view(-1), *w, tpid, b2e, B)["out"]
        torch.cuda.synchronize()
        return y.view(times, n, H)
    one, many = run(1), run(T // n)
    assert one.float().norm() > 0 and not one.isnan().any()
    if name == "s_long_contraction":     # how the last tiles are cut along I goes by their number
        d = (many.float() - one.float()).norm(dim=(1, 2)) / one.float().norm()
        assert float(d.max()) <= 2.0 ** -8
    else:
        assert (many == one).all()
