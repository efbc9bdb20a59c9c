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
