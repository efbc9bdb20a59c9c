"""moe_tokens_fwd_mxfp8 on the GPU against the layer in 64 bits (oracle/ffn.py, whose bounds the tolerances are), and
against moe_fwd_mxfp8."""
import numpy as np
import pytest
import torch

from ffn_common import Problem, check_rows

pytestmark = pytest.mark.gpu

CASES = {
    "one": dict(T=1, H=128, I=128, E=1, K=1),
    "smallest": dict(T=1, H=32, I=32, E=2, K=1, bias=True, residual=True),
    "one_token": dict(T=1, H=1536, I=256, E=40, K=8, bias=True, residual=True),
    "one_token_long": dict(T=1, H=1024, I=4352, E=4, K=2, on_i=True, residual=True),
    "two_tokens_few_experts": dict(T=2, H=256, I=96, E=3, K=3, geglu=True),
    "eight": dict(T=8, H=640, I=160, E=7, K=2, bias=True),
    "nine": dict(T=9, H=160, I=128, E=30, K=3, residual=True),
    "ragged": dict(T=29, H=608, I=352, E=6, K=3, bias=True, geglu=True, residual=True, dropped=0.2),
    "one_expert": dict(T=70, H=128, I=64, E=1, K=1),
    "dense_loads": dict(T=130, H=256, I=128, E=2, K=2, residual=True),
    "ragged_dense": dict(T=100, H=96, I=224, E=3, K=2, on_i=True),
    "most": dict(T=256, H=128, I=128, E=24, K=8, bias=True, residual=True, dropped=0.3),
    "long_split": dict(T=3, H=128, I=8320, E=2, K=1, residual=True),
    "four": dict(T=4, H=352, I=256, E=12, K=5, bias=True, residual=True),
    "four_whole_tiles": dict(T=4, H=128, I=1088, E=40, K=32, residual=True),       # 1360 tiles of the gate/up product
    "four_wide": dict(T=4, H=2144, I=160, E=32, K=32, bias=True),                  # 1088 of the down projection, a half one last
    "five": dict(T=5, H=192, I=128, E=9, K=3, on_i=True),
    "whole_tiles": dict(T=40, H=2208, I=1120, E=32, K=2, geglu=True),
    "whole_tiles_64": dict(T=200, H=2112, I=96, E=32, K=3, residual=True, bias=True),
    "large_values": dict(T=20, H=128, I=128, E=2, K=1, sigma=40.0),
}


def _run(p, **more):
    import mxfp8_grouped_gemm_amd as mx
    pos, kw = p.tokens_on()
    out = mx.moe_tokens_fwd_mxfp8(*pos, **{**kw, **more})
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("name", CASES)
def test_tokens(name):
    p = Problem(**CASES[name], seed=sum(map(ord, name)))
    y, dy, _ = p.exact(blocks=False)
    out = _run(p)
    check_rows(out, y, dy, name)
    assert torch.equal(_run(p), out)       # the same bits again


def test_ids_out_of_range_and_no_selection():
    """Ids outside [0, E) are dropped; a token without any keeps its residual, or gets zeros."""
    p = Problem(T=12, H=128, I=64, E=4, K=2, residual=True, seed=3)
    p.idx[5] = (-1, 4)
    p.idx[7] = (2 ** 31 - 1, -2 ** 31)
    p.idx[8, 0] = -7
    p.pairs = {}
    for e in range(4):
        t, k = np.nonzero(p.idx == e)
        if t.size:
            p.pairs[e] = (t, p.scores[t, k])
    y, dy, _ = p.exact(blocks=False)
    out = _run(p)
    check_rows(out, y, dy)
    assert torch.equal(out[[5, 7]].cpu(), p.residual[[5, 7]])
    assert not _run(p, residual=None)[[5, 7]].any()
    p.idx[:] = -1
    assert torch.equal(_run(p).cpu(), p.residual)


def test_an_id_twice_counts_twice():
    p = Problem(T=3, H=128, I=64, E=4, K=2, seed=4)
    p.idx[1] = 2
    p.pairs = {}
    for e in range(4):
        t, k = np.nonzero(p.idx == e)
        if t.size:
            p.pairs[e] = (t, p.scores[t, k])
    y, dy, _ = p.exact(blocks=False)
    check_rows(_run(p), y, dy)


def test_many_of_one_expert_twice():
    """More selections of one expert than tokens: every one counts."""
    T, K = 256, 2
    p = Problem(T=T, H=64, I=32, E=3, K=K, idx=np.ones((T, K), np.int32), seed=5)
    p.pairs = {1: (np.repeat(np.arange(T), K), p.scores.reshape(-1))}
    y, dy, _ = p.exact(blocks=False)
    check_rows(_run(p), y, dy)


def test_same_layer_as_the_block_form():
    """The two forms round alike: what they differ by is the order of sums."""
    import mxfp8_grouped_gemm_amd as mx
    p = Problem(T=100, H=256, I=256, E=8, K=2, bias=True, residual=True, seed=6)
    pos, kw = p.on()
    block = mx.moe_fwd_mxfp8(*pos, **kw)["out"].float()
    tok = _run(p).float()
    assert float((block - tok).norm() / block.norm()) <= 4e-3


def test_in_place_empty_and_workspace():
    import mxfp8_grouped_gemm_amd as mx
    p = Problem(T=10, H=128, I=64, E=4, K=2, residual=True, seed=7)
    want = _run(p)
    pos, kw = p.tokens_on()
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")     # NaN everywhere
    assert torch.equal(mx.moe_tokens_fwd_mxfp8(*pos, **kw, workspace=ws, out=kw["residual"]), want)
    none = [pos[0][:0], pos[1][:0], pos[2][:0], *pos[3:]]
    assert mx.moe_tokens_fwd_mxfp8(*none).shape == (0, 128)


def test_stream_and_graph():
    """A captured decode step, replayed on other tokens, selections and scores with eager work in between."""
    import mxfp8_grouped_gemm_amd as mx
    a, b = (Problem(T=4, H=512, I=128, E=16, K=4, residual=True, seed=s) for s in (8, 9))
    pos, kw = a.tokens_on()
    other, okw = b.tokens_on()
    out = torch.empty(4, 512, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mx.moe_tokens_fwd_mxfp8(*pos, **kw, workspace=ws, out=out)
    s.synchronize()
    assert torch.equal(out, _run(a))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.moe_tokens_fwd_mxfp8(*pos, **kw, workspace=ws, out=out)
    first = [t.clone() for t in pos[:3]]
    for k in range(4):
        for dst, x, y in zip(pos[:3], first, other[:3]):
            dst.copy_(y if k % 2 else x)
        want = mx.moe_tokens_fwd_mxfp8(*pos, **kw)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_router_to_tokens():
    """A decode step as a user makes it: router, then the layer, with masked tokens."""
    import mxfp8_grouped_gemm_amd as mx
    p = Problem(T=6, H=128, I=128, E=16, K=4, seed=10)
    pos, kw = p.tokens_on()
    logits = torch.randn(6, 16, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    mask = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.bool, device="cuda")
    idx, scores, _ = mx.moe_router_fwd(mx.ROUTER_SOFTMAX_OVER_TOPK, logits, 4, token_mask=mask)
    out = mx.moe_tokens_fwd_mxfp8(pos[0], idx, scores, *pos[3:], **kw)
    p.idx, p.scores = idx.cpu().numpy(), scores.cpu().numpy()
    p.pairs = {}
    for e in range(16):
        t, k = np.nonzero(p.idx == e)
        if t.size:
            p.pairs[e] = (t, p.scores[t, k])
    y, dy, _ = p.exact(blocks=False)
    check_rows(out, y, dy)
    assert not out[2].any()
