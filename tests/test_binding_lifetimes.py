"""What the bindings allocate lives until the library call has enqueued its work.

A tensor dropped before that goes back to the allocator, which may hand its
block to another thread, or unmap it, while the kernels that use it are not
even enqueued.  Without a GPU: the library call is replaced by a check."""
import weakref

import pytest
import torch

import mxfp8_grouped_gemm_amd as mx


def _router(z, idx):
    mx.moe_router_fwd(mx.ROUTER_SOFTMAX_OVER_TOPK, z, 2)


def _balance(z, idx):
    mx.moe_balance_loss(z, idx, 0.01, 0.001)


def _balance_bwd(z, idx):
    E = z.shape[1]
    mx.moe_balance_loss_bwd(z, torch.zeros(1, E, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 2, 0.01)


def _act(z, idx):
    mx.mxfp8_gated_act_fwd(torch.zeros(2, 2, 64, dtype=torch.bfloat16))


def _act_bwd(z, idx):
    mx.mxfp8_gated_act_bwd(torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.uint8),
                           torch.zeros(2, 2, 2, dtype=torch.uint8))


@pytest.mark.parametrize("call,made", [(_router, 3), (_balance, 4), (_balance_bwd, 1), (_act, 3), (_act_bwd, 1)])
def test_allocations_are_alive_at_the_library_call(monkeypatch, call, made):
    refs, alive = [], []

    def empty(*a, **kw):
        t = torch.empty(*a, **kw)
        refs.append(weakref.ref(t))
        return t

    monkeypatch.setattr(mx, "_empty", empty)
    monkeypatch.setattr(mx, "_dev", lambda t, dtype, name: None if t is None else t.data_ptr())
    monkeypatch.setattr(mx, "_call", lambda device, name, *a: alive.extend(r() is not None for r in refs))
    call(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
    assert alive == [True] * made
