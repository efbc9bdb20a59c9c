"""What the MoE forward's documentation allows, over every way it sets a layer up: counts of valid tokens, blocks of no
expert, rows that hold NaN and infinity, captured calls, and graphs that share a workspace."""
import numpy as np
import pytest
import torch

from ffn_common import Problem, check_rows

pytestmark = pytest.mark.gpu

# name: the problem, and how many blocks its list has (None: its own and one without a token)
KINDS = {
    "one_workgroup": (dict(T=200, H=128, I=128, E=3, K=2, B=128), None),
    "exact_products": (dict(T=200, H=160, I=96, E=3, K=2, B=128), 80),
    "scaled_128": (dict(T=200, H=128, I=256, E=3, K=2, B=128), 300),
    "many_blocks": (dict(T=200, H=128, I=64, E=3, K=2, B=128), 1100),
    "scaled_256": (dict(T=200, H=1536, I=384, E=3, K=2, B=256), 60),
    "by_slot": (dict(T=200, H=1536, I=8192, E=2, K=1, B=256), 6),
}


def _problem(name, seed, **more):
    args, N = KINDS[name]
    p = Problem(**args, residual=True, seed=seed, **more)
    if N is not None:
        assert p.N <= N
        p.tpid = np.concatenate([p.tpid, np.full((N - p.N) * p.B, -1, np.int32)])
        p.b2e = np.concatenate([p.b2e, np.full(N - p.N, p.E - 1, np.int32)])
        p.N = N
    return p


def _fwd(p, checkpoint=None, **more):
    import mxfp8_grouped_gemm_amd as mx
    pos, kw = p.on()
    r = mx.moe_fwd_mxfp8(*pos, **{**kw, **more}, checkpoint=checkpoint)
    torch.cuda.synchronize()
    return r


@pytest.mark.parametrize("kind", KINDS)
def test_valid_tokens_and_blocks_of_no_expert(kind):
    """Tokens from the count on are in no slot, blocks of an expert outside [0, E) hold none, wherever they stand."""
    p = _problem(kind, 61)
    # the last block, of no expert; the first too, whose tokens go with it
    p.b2e[-1] = p.E
    p.tpid[-p.B:-p.B + 5] = np.arange(5)
    lost = set(p.tpid[:p.B].tolist())
    e0 = int(p.b2e[0])
    p.b2e[0] = -1
    count = lambda n: torch.tensor([n], dtype=torch.int32, device="cuda")   # noqa: E731
    whole = dict(p.pairs)
    for n in (150, 0, -7, p.T + 9):
        p.pairs = {}
        for e, (t, a) in whole.items():
            keep = (t < n) & ~(np.isin(t, list(lost)) if e == e0 else np.zeros(t.size, bool))
            if keep.any():
                p.pairs[e] = (t[keep], a[keep])
        r = _fwd(p, "bf16", num_valid_tokens=count(n))
        if n <= 0:
            assert torch.equal(r["out"].cpu(), p.residual) and not r["checkpoint"].any()
            continue
        y, dy, _ = p.exact()
        check_rows(r["out"], y, dy, (kind, n))
        owner = np.repeat(p.b2e, p.B)
        live = (p.tpid >= 0) & (p.tpid < n) & (owner >= 0) & (owner < p.E)
        gu = r["checkpoint"].view(p.N, 2, p.I, p.B)
        dead = torch.from_numpy(~live.reshape(p.N, 1, 1, p.B)).cuda()
        assert not (gu.view(torch.int16).bool() & dead).any() and (gu.bool() & ~dead).any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("kind", KINDS)
def test_a_row_of_nan_or_infinity_stays_in_its_row(kind, bad):
    p = _problem(kind, 62)
    clean = _fwd(p)["out"]
    p.x[77, 5] = bad
    p.x[123] = bad
    out = _fwd(p, "mxfp8")["out"]
    rows = torch.ones(p.T, dtype=torch.bool, device="cuda")
    rows[[77, 123]] = False
    assert torch.equal(out[rows], clean[rows])


@pytest.mark.parametrize("T", [1, 4, 8, 30, 200])
def test_few_tokens_of_nan_or_infinity_stay_in_their_rows(T):
    import mxfp8_grouped_gemm_amd as mx
    p = Problem(T=T + 1, H=160, I=128, E=3, K=2, bias=True, seed=63)
    pos, kw = p.tokens_on()
    T += 1
    for bad in (float("nan"), float("inf")):
        clean = mx.moe_tokens_fwd_mxfp8(*pos, **kw)
        x = pos[0].clone()
        x[T // 2, 3] = bad
        out = mx.moe_tokens_fwd_mxfp8(x, *pos[1:], **kw)
        rows = torch.arange(T, device="cuda") != T // 2
        assert torch.equal(out[rows], clean[rows])


@pytest.mark.parametrize("kind", KINDS)
def test_captured_calls_that_share_a_workspace(kind):
    """Two layers' calls in graphs of their own, one workspace: replayed in any order on changed inputs, with eager work
    between, each gives what an eager call gives."""
    import mxfp8_grouped_gemm_amd as mx
    ps = [_problem(kind, 64 + k, p=0.25 * k) for k in range(2)]
    args = [p.on() for p in ps]
    eager = [mx.MoeFwd(*pos, **kw, checkpoint="mxfp8") for pos, kw in args]
    ws = torch.full((max(op.workspace.numel() for op in eager),), 255, dtype=torch.uint8, device="cuda")
    ops = [mx.MoeFwd(*pos, **kw, checkpoint="mxfp8", workspace=ws) for pos, kw in args]
    graphs = []
    for op in ops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            op.run()
        graphs.append(g)
    x0 = [pos[0].clone() for pos, _ in args]
    for k, order in enumerate([(0, 1), (1, 0), (0, 0), (1, 1)]):
        want = []
        for (pos, kw), x, op in zip(args, x0, eager):
            pos[0].copy_(x * (1 + 0.5 * k))
            if kw["dropout_rng"] is not None:
                kw["dropout_rng"][1] = 50 + k
            r = op.run()
            want.append([t.clone() for t in (r["out"], *r["checkpoint"])])
        for i in order:
            outs = (ops[i].out["out"], *ops[i].out["checkpoint"])
            for t in outs:
                t.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            for got, w in zip(outs, want[i]):
                assert torch.equal(got, w), (kind, k, i)


@pytest.mark.parametrize("T", [1, 4, 8, 40, 200])
def test_captured_decode_steps_that_share_a_workspace(T):
    import mxfp8_grouped_gemm_amd as mx
    ps = [Problem(T=T, H=256, I=128, E=8, K=2, residual=True, seed=70 + k) for k in range(2)]
    args = [p.tokens_on() for p in ps]
    ws = torch.full((1 << 23,), 255, dtype=torch.uint8, device="cuda")
    outs = [torch.empty(T, 256, dtype=torch.bfloat16, device="cuda") for _ in ps]
    graphs = []
    for (pos, kw), out in zip(args, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mx.moe_tokens_fwd_mxfp8(*pos, **kw, workspace=ws, out=out)
        graphs.append(g)
    first = [[t.clone() for t in pos[:3]] for pos, _ in args]
    for k, order in enumerate([(0, 1), (1, 0), (0, 0), (1, 1)]):
        for (pos, _), own, other in zip(args, first, first[::-1]):
            for dst, a, b in zip(pos[:3], own, other):
                dst.copy_(b if k % 2 else a)
        want = [mx.moe_tokens_fwd_mxfp8(*pos, **kw) for pos, kw in args]
        for i in order:
            outs[i].zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(outs[i], want[i]), (T, k, i)


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(kind):
    """Two calls in flight, each with a workspace of its own."""
    import mxfp8_grouped_gemm_amd as mx
    ps = [_problem(kind, 80 + k) for k in range(2)]
    args = [p.on() for p in ps]
    want = [_fwd(p, "bf16") for p in ps]
    ops = [mx.MoeFwd(*pos, **kw, checkpoint="bf16") for pos, kw in args]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(3):
        for op, s in zip(ops, streams):
            with torch.cuda.stream(s):
                op.run()
    torch.cuda.synchronize()
    for op, w in zip(ops, want):
        assert torch.equal(op.out["out"], w["out"]) and torch.equal(op.out["checkpoint"], w["checkpoint"])
