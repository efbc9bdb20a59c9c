"""Seeded problems of the MoE forward for its tests: inputs on the host, the same on the device, and the 64-bit result."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from oracle import ffn

HALF = 2.0 ** -8        # half a bf16 step, relative


def bf16_values(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Problem:
    """T tokens of K selections among E experts, some dropped; weights quantised along the contraction."""

    def __init__(self, T, H, I, E, K, B=128, bias=False, geglu=False, on_i=False, residual=False, dropped=0.0, p=0.0,
                 seed=0, sigma=1.0, idx=None):
        self.T, self.H, self.I, self.E, self.K, self.B = T, H, I, E, K, B
        self.geglu, self.on_i, self.p = geglu, on_i, p
        r = np.random.default_rng(seed)

        def bf(*shape, s=1.0):
            return torch.from_numpy((r.standard_normal(shape) * s).astype(np.float32)).to(torch.bfloat16)

        self.x = bf(T, H, s=sigma)
        self.w_gate_up, self.w_down = bf(E, H, 2, I, s=H ** -0.5), bf(E, I, H, s=I ** -0.5)
        self.b1 = bf(E, 2, I, s=0.5) if bias else None
        self.b2 = bf(E, H, s=0.5) if bias else None
        self.residual = bf(T, H) if residual else None
        self.seed_offset = int(r.integers(0, 2 ** 62)), int(r.integers(0, 2 ** 40))
        if idx is None:
            idx = np.argsort(r.random((T, E)) + 0.3 * np.arange(E) / E, axis=1)[:, :K]
            idx = np.where(r.random((T, K)) < dropped, -1, idx)
        self.idx = np.asarray(idx, np.int32)
        self.scores = r.random((T, K)).astype(np.float32)
        live = self.idx >= 0
        self.aff = np.zeros((T, E), np.float32)
        t, k = np.nonzero(live)
        self.aff[t, self.idx[t, k]] = self.scores[t, k]
        # blocks: expert after expert, tokens ascending; one block at the end stays empty
        slots, owner = [], []
        self.pairs = {}
        for e in range(E):
            tok = np.nonzero((self.idx == e).any(1))[0]
            if tok.size:
                self.pairs[e] = (tok, self.aff[tok, e])
            for c in range(0, tok.size, B):
                part = np.full(B, -1, np.int32)
                part[:tok[c:c + B].size] = tok[c:c + B]
                slots.append(part)
                owner.append(e)
        slots.append(np.full(B, -1, np.int32))
        owner.append(E - 1)
        self.tpid, self.b2e = np.concatenate(slots), np.array(owner, np.int32)
        self.N = len(owner)
        wgu = self.w_gate_up.permute(0, 2, 3, 1).reshape(-1, H)
        wd = self.w_down.permute(0, 2, 1).reshape(-1, I)
        self.q = [a.reshape(s) for (a, s) in zip(
            [*oracle.quantize(_bits(wgu), 1, oracle.E4M3), *oracle.quantize(_bits(wd), 1, oracle.E4M3)],
            [(E, 2, I, H), (E, 2, I, H // 32), (E, H, I), (E, H, I // 32)])]

    def exact(self, blocks=True):
        """y, its bound and the gate/up values.  blocks: of the block form, which keeps the down projection's rows in scaled
        fp16 up to a contraction of 4096 (moe_fwd_down.hip)."""
        wgu, wd = ffn.mx_values(self.q[0], self.q[1]), ffn.mx_values(self.q[2], self.q[3])
        v = {k: None if t is None else bf16_values(t) for k, t in
             dict(b1=self.b1, b2=self.b2, residual=self.residual).items()}
        keep = ffn.dropout_keep(self.T * self.H, self.p, *self.seed_offset).reshape(self.T, self.H) if self.p else None
        return ffn.moe_fwd(bf16_values(self.x), self.pairs, wgu, wd, geglu=self.geglu, on_i=self.on_i, keep=keep,
                           scale=ffn.dropout_scale(self.p),
                           f16=blocks and (self.I < 4096 or self.I % 128 != 0), **v)

    def on(self, device="cuda"):
        """The arguments of moe_fwd_mxfp8 (positional, keywords) on a device."""
        d = lambda a: None if a is None else (a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))).to(device)   # noqa: E731
        pos = [d(a) for a in (self.x, self.aff.reshape(-1), *self.q, self.tpid, self.b2e)] + [self.B]
        kw = dict(gate_up_bias=d(self.b1), down_bias=d(self.b2), affinity_on=int(self.on_i), activation=int(self.geglu),
                  residual=d(self.residual), dropout_p=self.p,
                  dropout_rng=torch.tensor(self.seed_offset, dtype=torch.int64, device=device) if self.p else None)
        return pos, kw

    def tokens_on(self, device="cuda"):
        """The arguments of moe_tokens_fwd_mxfp8 on a device."""
        pos, kw = self.on(device)
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)   # noqa: E731
        for k in ("dropout_p", "dropout_rng"):
            kw.pop(k)
        return [pos[0], d(self.idx), d(self.scores), *pos[2:6]], kw


def _bits(t):
    return t.contiguous().view(torch.int16).numpy().view(np.uint16)


def check_rows(got, y, dy, what=""):
    """|got - y| within the bound and half a step of the output's type; says the worst element if not."""
    g = bf16_values(got)
    tol = dy + (np.abs(y) + dy) * HALF
    bad = ~(np.abs(g - y) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:5].tolist(), g[bad][:5], y[bad][:5], tol[bad][:5])
