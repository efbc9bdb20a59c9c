"""What the MoE forward, dropout and the transposed quantiser refuse, without a GPU: every check comes before any launch
(the pointers here are never dereferenced), and the bindings check shapes, types and devices first."""
import ctypes as C
import math

import pytest
import torch

import mxfp8_grouped_gemm_amd as mx
from test_abi import test_binding_structs_match_the_header as _structs_match

F = 0x10000
ODD = 0x10004


@pytest.mark.parametrize("cls,ctype", [("DropoutAddArgs", "dropout_add_args"), ("MoeFwdArgs", "moe_fwd_mxfp8_args"),
                                       ("MoeTokensFwdArgs", "moe_tokens_fwd_mxfp8_args")])
def test_binding_structs_match_the_header(cls, ctype, tmp_path):
    _structs_match(cls, ctype, tmp_path)


def test_quantize_transposed_refusals():
    f = mx.lib().mxfp8_quantize_transposed

    def run(x=F, G=2, R=64, N=5, fmt=0, codes=F, scales=F):
        return f(x, G, R, N, fmt, codes, scales, None)

    for bad in (dict(G=-1), dict(R=-32), dict(N=-1), dict(R=48), dict(fmt=2), dict(x=None), dict(codes=None),
                dict(scales=None), dict(x=ODD), dict(codes=ODD)):
        assert run(**bad) == 1, bad
    assert run(G=2 ** 24) == 2 and run(R=2 ** 36) == 2 and run(N=2 ** 40) == 2 and run(R=2 ** 62, N=2 ** 62) == 2
    for empty in (dict(G=0), dict(R=0), dict(N=0)):
        assert run(x=None, codes=None, scales=None, **empty) == 0


def _drop(**kw):
    a = mx.DropoutAddArgs(4, 40, 40, 40, 40, 0, 0.5, F, F, F, F)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_dropout_refusals():
    L = mx.lib()
    fwd = lambda **kw: L.dropout_add_fwd(C.byref(_drop(**kw)), None)                    # noqa: E731
    bwd = lambda **kw: L.dropout_add_bwd(C.byref(_drop(**{"residual": None, **kw})), None)   # noqa: E731
    for f in (fwd, bwd):
        for bad in (dict(rows=-1), dict(cols=-1), dict(type=2), dict(p=-0.1), dict(p=1.5), dict(p=math.nan), dict(ldx=39),
                    dict(ldy=0), dict(ldx=2 ** 60), dict(x=None), dict(y=None), dict(rng=None), dict(x=ODD), dict(y=ODD),
                    dict(rng=0x10004)):
            assert f(**bad) == 1, bad
        assert f(rows=2 ** 33, cols=40) == 2
        assert f(rows=0, x=None, y=None, rng=None) == 0 and f(cols=0) == 0
    assert fwd(ldr=39) == 1 and fwd(residual=ODD) == 1
    assert bwd(residual=F) == 1 and "residual" in mx.last_error()
    assert L.dropout_add_fwd(None, None) == 1 and L.dropout_add_bwd(None, None) == 1


def _fwd(**kw):
    a = mx.MoeFwdArgs(256, 128, 256, 4, 7, 128, *([F] * 8), None, None, None, 0, 0, F)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_moe_fwd_refusals():
    L = mx.lib()
    need = L.moe_fwd_mxfp8_workspace_size(C.byref(_fwd()))
    assert need > 0 and need % 256 == 0

    def run(ws=F, nbytes=1 << 60, **kw):
        return L.moe_fwd_mxfp8(C.byref(_fwd(**kw)), ws, nbytes, None)

    shapes = [dict(T=0), dict(H=0), dict(I=-32), dict(E=0), dict(N=0), dict(block_size=0), dict(H=48), dict(I=40)]
    large = [dict(block_size=64), dict(block_size=2048), dict(T=2 ** 24, H=128), dict(T=2 ** 29), dict(N=2 ** 17 + 1),
             dict(H=2 ** 20, I=2 ** 10), dict(I=2 ** 23, H=32), dict(N=2 ** 16, I=2 ** 13), dict(T=2 ** 40), dict(N=2 ** 40)]
    for bad in shapes:
        assert run(**bad) == 1, bad
        assert L.moe_fwd_mxfp8_workspace_size(C.byref(_fwd(**bad))) == 0
    for bad in large:
        assert run(**bad) == 2, bad
        assert L.moe_fwd_mxfp8_workspace_size(C.byref(_fwd(**bad))) == 0
    for name in ("hidden_states", "expert_affinities_masked", "gate_up_codes", "gate_up_scales", "down_codes", "down_scales",
                 "token_position_to_id", "block_to_expert", "output_hidden_states"):
        assert run(**{name: None}) == 1 and run(**{name: ODD}) == 1, name
    for name in ("gate_up_proj_bias", "down_proj_bias", "gate_up_proj_act_checkpoint_T", "residual"):
        assert run(**{name: ODD}) == 1, name
    for bad in (dict(affinity_on=2), dict(activation=2), dict(dropout_p=-1.0), dict(dropout_p=math.nan),
                dict(dropout_p=0.5), dict(gate_up_checkpoint_codes=F), dict(gate_up_checkpoint_scales=F),
                dict(gate_up_checkpoint_codes=F, gate_up_checkpoint_scales=F, gate_up_proj_act_checkpoint_T=F),
                dict(gate_up_checkpoint_codes=F, gate_up_checkpoint_scales=F, fmt_checkpoint=2),
                dict(num_valid_tokens=0x10002), dict(dropout_rng=ODD), dict(ws=None), dict(ws=0x10010)):
        assert run(**bad) == 1, bad
    for bias in ("gate_up_proj_bias", "down_proj_bias"):
        assert run(affinity_on=1, **{bias: F}) == 2
    assert run(nbytes=need - 1) == 3 and "workspace" in mx.last_error()
    assert L.moe_fwd_mxfp8(None, F, 1 << 60, None) == 1 and L.moe_fwd_mxfp8_workspace_size(None) == 0


def _tok(**kw):
    a = mx.MoeTokensFwdArgs(8, 128, 256, 4, 2, *([F] * 7), None, None, 0, 0, None, F)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_moe_tokens_fwd_refusals():
    L = mx.lib()
    need = L.moe_tokens_fwd_mxfp8_workspace_size(C.byref(_tok()))
    assert need > 0 and need % 256 == 0

    def run(ws=F, nbytes=1 << 60, **kw):
        return L.moe_tokens_fwd_mxfp8(C.byref(_tok(**kw)), ws, nbytes, None)

    for bad in (dict(T=-1), dict(H=0), dict(I=-32), dict(E=0), dict(K=0), dict(K=33), dict(H=48), dict(I=40)):
        assert run(**bad) == 1, bad
        assert L.moe_tokens_fwd_mxfp8_workspace_size(C.byref(_tok(**bad))) == 0
    for large in (dict(T=257), dict(H=2 ** 20, I=2 ** 10), dict(H=2 ** 23, I=32), dict(I=2 ** 23, H=32), dict(E=4097),
                  dict(T=256, K=32, I=2 ** 18, H=32)):
        assert run(**large) == 2, large
        assert L.moe_tokens_fwd_mxfp8_workspace_size(C.byref(_tok(**large))) == 0
    for name in ("hidden_states", "topk_idx", "topk_scores", "gate_up_codes", "gate_up_scales", "down_codes", "down_scales",
                 "output_hidden_states"):
        assert run(**{name: None}) == 1 and run(**{name: ODD}) == 1, name
    for bad in (dict(gate_up_proj_bias=ODD), dict(down_proj_bias=ODD), dict(residual=ODD), dict(affinity_on=2),
                dict(activation=-1), dict(ws=None), dict(ws=0x10010)):
        assert run(**bad) == 1, bad
    assert run(affinity_on=1, gate_up_proj_bias=F) == 2 and run(affinity_on=1, down_proj_bias=F) == 2
    assert run(nbytes=need - 1) == 3 and "workspace" in mx.last_error()
    assert run(T=0, hidden_states=None, topk_idx=None, ws=None) == 0
    assert L.moe_tokens_fwd_mxfp8(None, F, 1 << 60, None) == 1 and L.moe_tokens_fwd_mxfp8_workspace_size(None) == 0


def test_bindings_check_their_tensors():
    z = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        mx.mxfp8_quantize_transposed(torch.zeros(32, 4, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="32"):
        mx.mxfp8_quantize_transposed(z)
    with pytest.raises(ValueError, match="rows, cols"):
        mx.mxfp8_quantize_transposed(z[0])
    with pytest.raises(ValueError, match="device tensor"):
        mx.dropout_add(z, 0.1, None)
    with pytest.raises(TypeError):
        mx.dropout_add(z.half(), 0.1, None)
    w = torch.zeros(2, 2, 32, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="hidden_states"):
        mx.moe_fwd_mxfp8(z[0], None, w, None, None, None, None, None, 128)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="checkpoint"):
        mx.moe_fwd_mxfp8(z, None, w, None, None, None, None, i, 128, checkpoint="fp8")
    with pytest.raises(ValueError, match="device tensor"):
        mx.moe_fwd_mxfp8(z, None, w, None, None, None, None, i, 128)
    with pytest.raises(ValueError, match="topk_idx"):
        mx.moe_tokens_fwd_mxfp8(z, i, None, w, None, None, None)
    with pytest.raises(ValueError, match="device tensor"):
        mx.moe_tokens_fwd_mxfp8(z, i.view(1, 1), None, w, None, None, None)
