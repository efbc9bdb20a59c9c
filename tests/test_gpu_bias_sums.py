"""The bias gradients' sums of moe_bwd_mxfp8: what the documented workspace regions hold after a call, and that the order
of the blocks' atomics does not show."""
import numpy as np
import pytest
import torch

import synthetic as S
from moe_gpu_common import gpu_problem

pytestmark = pytest.mark.gpu

CFGS = {
    # db2 beside the gather of dY (H % 128 == 0): Phase 1 apart from its epilogue and with it; H % 128 != 0, db2 on its own
    "gathered": S.scaled(S.FINE, T=4096, H=256, I=128, E=3, K=2, B=256),
    "gathered_fused": S.scaled(S.FINE, T=20000, H=128, I=128, E=3, K=2, B=128),
    "own_kernel": S.scaled(S.FINE, T=4096, H=160, I=96, E=3, K=2, B=128),
    "smallest": S.scaled(S.FINE, T=40, H=32, I=32, E=4, K=2, B=128),
}


def _sums(op, cfg):
    """db1_acc [E, 2, I] and db2_acc [E, H] as the header describes them: fp32."""
    torch.cuda.synchronize()
    ws, L = op.workspace.cpu().numpy(), op.layout
    return {k: ws[L[k + "_acc"]:][:4 * n].view(np.float32).copy()
            for k, n in (("db1", cfg.E * 2 * cfg.I), ("db2", cfg.E * cfg.H))}


@pytest.mark.parametrize("name", CFGS)
def test_workspace_holds_the_fp32_sums(name):
    """The regions' values, rounded to bf16, are the returned gradients."""
    cfg = CFGS[name]
    assert cfg.has_bias
    op = gpu_problem(cfg)["op"]
    op.workspace.fill_(0xC3)
    out = op.run()
    for k, v in _sums(op, cfg).items():
        want = torch.from_numpy(v).to(torch.bfloat16)
        assert np.isfinite(v).all() and v.any()
        assert torch.equal(out[k].cpu().reshape(-1).view(torch.int16), want.view(torch.int16)), k


@pytest.mark.parametrize("name", CFGS)
def test_repeated_runs_give_the_same_bits(name):
    """Dozens of blocks an expert: fp32 atomics would give other sums, in the last bits at least, on every run."""
    cfg = CFGS[name]
    op = gpu_problem(cfg)["op"]
    first, sums = {k: v.clone() for k, v in op.run().items() if v is not None}, _sums(op, cfg)
    for _ in range(6):
        again = op.run()
        for k, v in _sums(op, cfg).items():
            assert np.array_equal(v.view(np.int32), sums[k].view(np.int32)), k
        for k, v in first.items():
            assert torch.equal(again[k].view(torch.int16), v.view(torch.int16)), k


@pytest.mark.parametrize("name", CFGS)
def test_accumulated_gradients_leave_the_sums_alone(name):
    """With accumulate the regions hold this call's sums, and the outputs what they held plus those, rounded once."""
    cfg = CFGS[name]
    op = gpu_problem(cfg)["op"]
    op.run()
    sums = _sums(op, cfg)
    g = torch.Generator("cuda").manual_seed(1)
    for v in op.out.values():
        if v is not None:
            v.copy_(torch.randn(v.shape, generator=g, device="cuda"))
    before = {k: op.out[k].cpu().reshape(-1).float() for k in sums}
    op.args.accumulate = 1
    op.workspace.fill_(0xC3)
    op.run()
    for k, v in _sums(op, cfg).items():
        assert np.array_equal(v.view(np.int32), sums[k].view(np.int32)), k
        want = (before[k] + torch.from_numpy(v)).to(torch.bfloat16)
        assert torch.equal(op.out[k].cpu().reshape(-1).view(torch.int16), want.view(torch.int16)), k
