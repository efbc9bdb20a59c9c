"""What the router forward, the balance losses and the gated activation refuse,
without a GPU: every check comes before any launch (the pointers here are never
dereferenced), and the bindings check shapes, types and devices first."""
import ctypes as C
import math

import pytest
import torch

import mxfp8_grouped_gemm_amd as mx
from test_abi import test_binding_structs_match_the_header as _structs_match

F = C.c_void_p(0x10000)
ODD = C.c_void_p(0x10004)


@pytest.mark.parametrize("cls,ctype", [("BalanceArgs", "moe_balance_args"), ("GatedActArgs", "mxfp8_gated_act_args")])
def test_binding_structs_match_the_header(cls, ctype, tmp_path):
    _structs_match(cls, ctype, tmp_path)


def test_router_fwd_refusals():
    f = mx.lib().moe_router_fwd
    ok = dict(mode=0, T=4, E=8, K=2, logits=F, typ=0, mask=None, renorm=0, idx=F, scores=F, aff=F)

    def run(**kw):
        a = {**ok, **kw}
        return f(a["mode"], a["T"], a["E"], a["K"], a["logits"], a["typ"], a["mask"], a["renorm"], a["idx"],
                 a["scores"], a["aff"], None)

    assert run(mode=3) == 1 and "mode" in mx.last_error()
    assert run(typ=2) == 1 and "logits_type" in mx.last_error()
    for bad in (dict(T=-1), dict(E=0), dict(K=0), dict(K=9), dict(E=64, K=33)):
        assert run(**bad) == 1, bad
    assert run(E=4097) == 2 and "4096" in mx.last_error()
    assert run(T=2 ** 30) == 2
    assert run(T=2 ** 26 - 1023, E=257, K=1) == 2 and "one launch" in mx.last_error()
    assert run(renorm=1) == 1 and "renorm" in mx.last_error()
    assert run(mode=1, renorm=2) == 1
    for k in ("logits", "idx", "scores"):
        assert run(**{k: None}) == 1 and "null" in mx.last_error()
        assert run(**{k: ODD}) == 1 and "aligned" in mx.last_error()
    assert run(aff=ODD) == 1
    assert run(T=0, logits=None, idx=None, scores=None, aff=None) == 0


def _balance_args(**kw):
    a = mx.BalanceArgs(64, 8, 2, 1, F, 0, F, None, None, 0.01, 0.001, F, F, F, None, F, 0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_balance_refusals():
    L = mx.lib()
    need = L.moe_balance_loss_workspace_size(64, 8, 1)
    assert need > 0 and need % 256 == 0

    def fwd(ws=F, nbytes=1 << 40, **kw):
        return L.moe_balance_loss(C.byref(_balance_args(**kw)), ws, nbytes, None)

    def bwd(**kw):
        return L.moe_balance_loss_bwd(C.byref(_balance_args(**kw)), None)

    for f in (fwd, bwd):
        for bad in (dict(T=-1), dict(E=0), dict(K=0), dict(K=9), dict(S=0), dict(S=2), dict(logits_type=5),
                    dict(balance_coef=math.inf), dict(z_coef=math.nan), dict(logits=None), dict(counts=None),
                    dict(num_tokens=None), dict(counts=0x10004), dict(logits=0x10002), dict(seq_starts=0x10002)):
            assert f(**bad) == 1, bad
        assert f(E=4097, K=1) == 2
        assert f(T=2 ** 30) == 2
        assert f(S=2 ** 28, seq_starts=F) == 2 and f(S=2 ** 20 + 1, seq_starts=F) == 2
    assert fwd(loss=None) == 1 and fwd(topk_idx=None) == 1 and fwd(topk_idx=0x10004) == 1 and fwd(loss=0x10002) == 1
    assert bwd(dlogits=None) == 1 and bwd(dlogits=0x10004) == 1 and bwd(dloss=0x10002) == 1
    assert bwd(accumulate=2) == 1 and "accumulate" in mx.last_error()
    assert bwd(T=0, logits=None, dlogits=None) == 0
    assert fwd(nbytes=need - 1) == 3 and "workspace" in mx.last_error()
    assert fwd(ws=None) == 1 and fwd(ws=C.c_void_p(0x10010)) == 1
    assert L.moe_balance_loss(None, F, 1 << 40, None) == 1 and L.moe_balance_loss_bwd(None, None) == 1
    for bad in ((-1, 8, 1), (64, 0, 1), (64, 4097, 1), (64, 8, 0), (64, 8, 2 ** 29)):
        assert L.moe_balance_loss_workspace_size(*bad) == 0


def test_gated_act_refusals():
    L = mx.lib()

    def args(**kw):
        a = mx.GatedActArgs(4, 128, 0, 0, None, 0, 0)
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    def fwd(x=F, inter=F, codes=F, scales=F, **kw):
        return L.mxfp8_gated_act_fwd(C.byref(args(**kw)), x, inter, codes, scales, None)

    def bwd(d=F, codes=F, scales=F, out=F, **kw):
        return L.mxfp8_gated_act_bwd(C.byref(args(**kw)), d, codes, scales, out, None)

    for f in (fwd, bwd):
        for bad in (dict(rows=-1), dict(cols=-32), dict(cols=48), dict(activation=2), dict(fmt=2),
                    dict(token_position_to_id=F, period=0), dict(token_position_to_id=F, period=48),
                    dict(token_position_to_id=F, period=96), dict(token_position_to_id=F, period=64, T=-1),
                    dict(token_position_to_id=0x10004, period=64, T=3), dict(codes=None), dict(codes=ODD),
                    dict(scales=None)):
            assert f(**bad) == 1, bad
        assert f(rows=2 ** 34, cols=64) == 2
        assert f(rows=0, codes=None, scales=None) == 0
        assert f(cols=0) == 0
    assert fwd(x=None) == 1 and fwd(inter=ODD) == 1 and bwd(d=None) == 1 and bwd(out=ODD) == 1
    assert L.mxfp8_gated_act_fwd(None, F, F, F, F, None) == 1 and L.mxfp8_gated_act_bwd(None, F, F, F, F, None) == 1


def test_bindings_check_their_tensors():
    z = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        mx.moe_router_fwd(0, z, 2)
    with pytest.raises(TypeError):
        mx.moe_router_fwd(0, z.double(), 2)
    with pytest.raises(ValueError, match="logits"):
        mx.moe_router_fwd(0, z[0], 2)
    with pytest.raises(ValueError, match="device tensor"):
        mx.moe_balance_loss(z, torch.zeros(4, 2, dtype=torch.int32), 0.1)
    with pytest.raises(ValueError, match="device tensor"):
        mx.moe_balance_loss_bwd(z, torch.zeros(1, 8, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 2, 0.1)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        mx.mxfp8_gated_act_fwd(x)
    c, s = torch.zeros(2, 2, 64, dtype=torch.uint8), torch.zeros(2, 2, 2, dtype=torch.uint8)
    for bad in (c[:, :1], c[:, :, :48], c[0]):
        with pytest.raises(ValueError):
            mx.mxfp8_gated_act_bwd(x[:, 0].contiguous(), bad, s)
    with pytest.raises(ValueError, match="shape"):
        mx.mxfp8_gated_act_bwd(x, c, s)
    with pytest.raises(ValueError, match="needs T"):
        mx.mxfp8_gated_act_bwd(x[:, 0].contiguous(), c, s, token_position_to_id=torch.zeros(128, dtype=torch.int32))
    with pytest.raises(ValueError, match="token_position_to_id"):
        mx.mxfp8_gated_act_bwd(x[:, 0].contiguous(), c, s, token_position_to_id=torch.zeros(64, dtype=torch.int32), T=1)


def test_moe_bwd_checkpoint_refusals():
    """The MXFP8 gate/up checkpoint of moe_bwd_mxfp8: in validation, before any device access."""
    from test_abi import _fake_args
    L = mx.lib()
    f = 0x10000

    def run(**kw):
        a = _fake_args(mx, L)
        for k, v in kw.items():
            setattr(a, k, v)
        return L.moe_bwd_mxfp8(C.byref(a), C.c_void_p(f), 1024, None)

    ck = dict(gate_up_proj_act_checkpoint_T=None, gate_up_checkpoint_codes=f, gate_up_checkpoint_scales=f)
    assert run(**ck) == 3                                     # accepted up to the workspace
    assert run(gate_up_proj_act_checkpoint_T=None) == 1
    assert run(**{**ck, "gate_up_proj_act_checkpoint_T": f}) == 1 and "not both" in mx.last_error()
    assert run(**{**ck, "gate_up_checkpoint_scales": None}) == 1 and "together" in mx.last_error()
    assert run(gate_up_checkpoint_scales=f) == 1 and "together" in mx.last_error()
    assert run(**ck, fmt_checkpoint=2) == 1 and "fmt_checkpoint" in mx.last_error()
    assert run(**{**ck, "gate_up_checkpoint_codes": f + 8}) == 1 and "aligned" in mx.last_error()
    assert run(**{**ck, "gate_up_checkpoint_scales": f + 4}) == 1 and "aligned" in mx.last_error()
    assert run(**ck, gate_act_checkpoint_T=f) == 2 and run(**ck, intermediate_checkpoint_T=f) == 2
    # the workspace of an E5M2 checkpoint holds the product that its epilogue reads
    a, b = _fake_args(mx, L), _fake_args(mx, L)
    a.N = b.N = 300   # tiles enough for the fused kernel, which needs no such region
    b.gate_up_checkpoint_codes, b.fmt_checkpoint = f, mx.E5M2
    assert L.moe_bwd_mxfp8_workspace_size(C.byref(b)) > L.moe_bwd_mxfp8_workspace_size(C.byref(a))
