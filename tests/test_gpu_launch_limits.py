"""Problems whose kernels would need 2^32 threads or more in one launch.

The runtime takes such a grid and runs its thread count modulo 2^32: no error,
and most outputs never written."""
import pytest
import torch

import mxfp8_grouped_gemm_amd as mx

pytestmark = pytest.mark.gpu


def _layer(T, x, dy, ck, aff, weights, B=128):
    """One expert, every token in its slot."""
    N = -(-T // B)
    tpid = torch.full((N * B,), -1, dtype=torch.int32, device="cuda")
    tpid[:T] = torch.arange(T, dtype=torch.int32, device="cuda")
    op = mx.MoeBwd(x, aff, *weights, tpid, torch.zeros(N, dtype=torch.int32, device="cuda"), dy, B, ck)
    for v in op.out.values():
        if v is not None:
            v.fill_(torch.nan)
    return op.run()


def test_finalisation_past_2_32_threads():
    """A workgroup of 256 per token and per 64 slots: 16.96 million of them.  dX and
    d(affinity) of a token depend on its own rows alone (one expert), so a layer of a
    range of the tokens gives the same bits."""
    T, H, I, B = 16_700_000, 32, 32, 128
    assert T < 2 ** 24 < T + -(-T // B) * B // 64
    print("finalisation", T, H, I, flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.randn(T, H, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ck = torch.randn(-(-T // B), 2, I, B, generator=g, device="cuda", dtype=torch.bfloat16)
    aff = torch.rand(T, generator=g, device="cuda")
    u8 = dict(dtype=torch.uint8, device="cuda")
    weights = (torch.randint(0, 120, (1, H, 2, I), generator=g, **u8), torch.full((1, H, 2, I // 32), 120, **u8),
               torch.randint(0, 120, (1, I, H), generator=g, **u8), torch.full((1, I, H // 32), 120, **u8))
    out = _layer(T, x, dy, ck, aff, weights)
    torch.cuda.synchronize()
    assert not out["dx"].isnan().any() and not out["daff"].isnan().any()
    n = 1 << 18
    for a in (0, T // 2 // B * B, (T - n) // B * B):   # the last one to the end, with a block partly filled
        b = min(a + n + B, T)
        part = _layer(b - a, x[a:b].contiguous(), dy[a:b].contiguous(), ck[a // B:-(-b // B)].contiguous(),
                      aff[a:b].contiguous(), weights)
        torch.cuda.synchronize()
        for k, rows in (("dx", out["dx"][a:b]), ("daff", out["daff"][a:b])):
            assert torch.equal(part[k].view(torch.int16), rows.view(torch.int16)), (k, a)


def test_router_backward_past_2_32_threads():
    """8 lanes a token: 2^29 tokens and some.  Top-1 of one expert: d(logit) = d(score), 0 without a selection."""
    T = 2 ** 29 + 1000
    print("router backward", T, flush=True)
    idx = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    idx[3::5] = -1
    g = torch.empty(T, 1, device="cuda")
    g.uniform_(1, 2)
    out = torch.full((T, 1), torch.nan, device="cuda")
    mx.moe_router_bwd(mx.ROUTER_TOPK, idx, dscores=g, num_experts=1, out=out)
    torch.cuda.synchronize()
    g[3::5] = 0
    assert torch.equal(out, g)
