"""The MoE backward's set-up regions against plain recomputation: slots, block
extents, expert lists (in one workgroup up to 1024 blocks and experts, in three
kernels past that), the inverse map, and d(affinity)'s zeros."""
import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_amd as mx
import synthetic as S
from moe_gpu_common import gpu_problem

pytestmark = pytest.mark.gpu


def _bound(gp, tpid, b2e, **kw):
    t, cfg = gp["t"], gp["cfg"]
    gu_c, gu_s, d_c, d_s = gp["wq"]
    E, H, I = cfg.E, cfg.H, cfg.I
    return mx.MoeBwd(t["hidden"], torch.from_numpy(gp["aff"]).cuda(), gu_c.view(E, H, 2, I), gu_s.view(E, H, 2, I // 32),
                     d_c.view(E, I, H), d_s.view(E, I, H // 32), tpid, b2e, t["dy"], cfg.B, t["ckpt"],
                     down_proj_bias=t["b2"], affinity_on=cfg.affinity_on, **kw)


def _check(cfg, op, tpid, b2e, N):
    L, ws, B, E, T = op.layout, op.workspace.cpu().numpy(), cfg.B, cfg.E, cfg.T
    i32 = lambda name, n: ws[L[name]:L[name] + 4 * n].view(np.int32)
    ok = (tpid >= 0) & (tpid < T) & (np.repeat(b2e, B) >= 0) & (np.repeat(b2e, B) < E)
    tok = np.where(ok, tpid, -1)
    assert np.array_equal(i32("slot_token", N * B), tok)
    aff = np.where(ok, op_aff(op, T, E)[np.maximum(tok, 0), np.clip(np.repeat(b2e, B), 0, E - 1)], 0)
    assert np.array_equal(ws[L["slot_affinity"]:L["slot_affinity"] + 4 * N * B].view(np.float32), aff.astype(np.float32))
    ext = np.array([(np.nonzero(row)[0][-1] + 1) if row.any() else 0 for row in ok.reshape(N, B)])
    assert np.array_equal(i32("block_flag", N), ext)
    lists = [[b for b in range(N) if b2e[b] == e and ext[b]] for e in range(E)]
    off = np.concatenate([[0], np.cumsum([len(x) for x in lists])])
    assert np.array_equal(i32("expert_block_offsets", E + 1), off)
    assert i32("expert_block_list", N)[:off[-1]].tolist() == [b for x in lists for b in x]
    inv = np.full((T, E), -1)
    s = np.nonzero(ok)[0]
    inv[tok[s], np.repeat(b2e, B)[s]] = s
    assert np.array_equal(i32("slot_of", T * E).reshape(T, E), inv)
    daff = op.out["daff"].float().cpu().numpy().reshape(T, E)
    assert not daff[inv < 0].any() and daff[inv >= 0].any()


def op_aff(op, T, E):
    return op.keep[1].cpu().numpy().reshape(T, E)


@pytest.mark.parametrize("T,E,N,order", [(256, 4, None, "sorted"), (300, 7, 40, "shuffled"), (64, 3, 1024, "shuffled"),
                                         (64, 3, 1025, "shuffled"), (200, 130, 190, "shuffled"),
                                         (31, 5, None, "sorted")])
def test_setup_regions(T, E, N, order):
    """Blocks in the builder's order and in any other, with empty blocks between,
    blocks of no expert, and odd T * E."""
    cfg = S.scaled(S.TINY, T=T, H=128, I=64, E=E, K=2, B=128)
    print("setup", T, E, N, order, flush=True)
    gp = gpu_problem(cfg, N=N)
    N = gp["N"]
    tpid, b2e = gp["tpid"].cpu().numpy().reshape(N, cfg.B), gp["b2e"].cpu().numpy().copy()
    if order == "shuffled":
        perm = np.random.default_rng(N).permutation(N)
        tpid, b2e = tpid[perm], b2e[perm]
        empty = np.nonzero((tpid < 0).all(1))[0]
        b2e[empty[::2]] = np.array([-1, E, 2 ** 30])[np.arange(len(empty[::2])) % 3]
        used = np.nonzero((tpid >= 0).any(1))[0]
        tpid[used[0]] = np.where(tpid[used[0]] >= 0, -5, T + 3)          # a block of ids out of range
        tpid[used[1], ::3] = -1                                          # holes inside a block
    tpid = np.ascontiguousarray(tpid.reshape(-1))
    op = _bound(gp, torch.from_numpy(tpid).cuda(), torch.from_numpy(np.ascontiguousarray(b2e)).cuda())
    op.out["daff"].fill_(3.0)
    op.run()
    torch.cuda.synchronize()
    _check(cfg, op, tpid, b2e, N)


def _ranges(ext, W, other, rr, B):
    """Tile starts, total and tile -> block map over the blocks' live slot tiles (round robin: whole blocks first)."""
    c = -(-ext // W) * other
    full = np.logical_and(rr, c == -(-B // W) * other)
    order = np.concatenate([np.nonzero(full)[0], np.nonzero(~full)[0]])
    start = np.zeros(len(ext) + 1, dtype=np.int64)
    start[order] = np.cumsum(c[order]) - c[order]
    start[-1] = c.sum()
    return np.concatenate([start, np.repeat(order, c[order])])


@pytest.mark.parametrize("H,I,B,E,N", [(128, 576, 128, 4, None), (256, 544, 512, 5, 30), (192, 96, 256, 3, 1024),
                                       (128, 576, 128, 3, 1025), (4096, 8192, 256, 2, None)])
def test_tile_ranges(H, I, B, E, N):
    """Phases 1 and 3 over short, partly filled and full blocks, in both tile orders
    (the last case: experts of 32 MiB and more, round robin)."""
    cfg = S.scaled(S.TINY, T=900, H=H, I=I, E=E, K=2, B=B)
    print("ranges", H, I, B, E, N, flush=True)
    gp = gpu_problem(cfg, N=N)
    op = _bound(gp, gp["tpid"], gp["b2e"])
    op.run()
    torch.cuda.synchronize()
    L, ws, N = op.layout, op.workspace.cpu().numpy(), gp["N"]
    i32 = lambda name, n: ws[L[name]:L[name] + 4 * n].view(np.int32)
    ext = i32("block_flag", N).astype(np.int64)
    m1, n1 = (128, 128) if H % 128 or H <= 2048 or I < 256 else (256, min(B, 256))
    if not (H % 128 == 0 and H <= 2048 and I <= 512):   # else Phase 1 takes every tile
        want = _ranges(ext, n1, -(-I // m1), I * H >= 2 ** 25, B)
        assert np.array_equal(i32("phase1_tiles", len(want)), want)
    wide = 2 * I % 128 == 0 and 2 * I >= 1024 and B >= 256 and H >= 256
    want = _ranges(ext, 256 if wide else 128, -(-H // 256), 2 * I * H >= 2 ** 25, B)
    assert np.array_equal(i32("phase3_tiles", len(want)), want)


@pytest.mark.parametrize("act8", [False, True])
@pytest.mark.parametrize("name", ["tiny", "fine_bias", "large_i", "geglu"])
def test_blocks_of_padding_change_nothing(name, act8):
    """A small layer takes Phase 1 and its epilogue apart, and Phases 3, 2 and 4 in one
    launch; with 300 blocks, all but the first few padding, it takes Phase 1 with its
    epilogue inside and the other phases apart.  The same bits.  db1 and db2 are atomic
    fp32 sums: their order moves a term's rounding (2^-19 of the largest), and each of two
    runs on each side may then round to the other bf16 neighbour, 4 * 2^-8 in all."""
    cfg = {"tiny": S.TINY, "fine_bias": S.scaled(S.FINE, T=512, H=256, I=128, E=16, K=4, B=128),
           "large_i": S.scaled(S.LARGE, T=256, H=384, I=160, E=4, K=2, B=256),
           "geglu": S.scaled(S.TINY, T=300, H=128, I=320, E=5, K=2, B=128)}[name]
    print("padding", name, act8, flush=True)
    gp = gpu_problem(cfg)
    n, N = gp["N"], 300
    assert n < N <= 1024
    t, E, H, I, B = gp["t"], cfg.E, cfg.H, cfg.I, cfg.B
    gu_c, gu_s, d_c, d_s = gp["wq"]
    act = mx.ACT_GEGLU if name == "geglu" else mx.ACT_SWIGLU

    def run(blocks, accumulate=False):
        pad = torch.full(((blocks - n) * B,), -1, dtype=torch.int32, device="cuda")
        tpid = torch.cat([gp["tpid"], pad])
        b2e = torch.cat([gp["b2e"], torch.arange(blocks - n, dtype=torch.int32, device="cuda") % E])
        ckpt = torch.cat([t["ckpt"], torch.full((blocks - n, 2, I, B), torch.nan, dtype=torch.bfloat16, device="cuda")])
        ck8 = mx.mxfp8_gated_act_fwd(ckpt, act, mx.E4M3, token_position_to_id=tpid, T=cfg.T)[1:] if act8 else None
        op = mx.MoeBwd(t["hidden"], torch.from_numpy(gp["aff"]).cuda(), gu_c.view(E, H, 2, I), gu_s.view(E, H, 2, I // 32),
                       d_c.view(E, I, H), d_s.view(E, I, H // 32), tpid, b2e, t["dy"], B, None if act8 else ckpt,
                       down_proj_bias=t["b2"], affinity_on=cfg.affinity_on, gate_up_checkpoint=ck8, activation=act,
                       accumulate=accumulate)
        for _ in range(2):
            op.run()
        torch.cuda.synchronize()
        return op.out

    for accumulate in (False, True):
        small, padded = run(n, accumulate), run(N, accumulate)
        for k in ("dx", "daff", "dwgu", "dwd"):
            assert torch.equal(small[k].view(torch.int16), padded[k].view(torch.int16)), k
        if cfg.has_bias:
            for k in ("db1", "db2"):
                a, b = small[k].float(), padded[k].float()
                assert ((a - b).abs() <= 2.0 ** -6 * b.abs() + 2.0 ** -19 * b.abs().max()).all(), k


@pytest.mark.parametrize("H,I,B,E,N,beside", [(128, 256, 128, 4, None, True), (256, 512, 512, 3, None, True),
                                              (2048, 256, 128, 5, 30, False), (128, 96, 1024, 2, 31, True),
                                              (128, 64, 128, 257, None, False)])
def test_tile_ranges_of_layers_too_small_to_fuse(H, I, B, E, N, beside):
    """H % 128 == 0, H <= 2048 and I <= 512 with fewer than 256 Phase-1 tiles: Phase 1 runs
    apart, on ranges made beside the gathers (up to 256 of their tiles, blocks and
    experts) or by the set-up's own kernel."""
    T = 300 if E > 256 else 900
    cfg = S.scaled(S.TINY, T=T, H=H, I=I, E=E, K=1 if E > 256 else 2, B=B)
    print("ranges", H, I, B, E, N, flush=True)
    gp = gpu_problem(cfg, N=N)
    N = gp["N"]
    tiles1 = -(-I // 128) * -(-B // 128) * N
    assert (H // 128 * N * B // 128 <= 256 and E <= 256) == beside and N <= 1024
    op = _bound(gp, gp["tpid"], gp["b2e"])
    L = op.layout
    if E <= 256:
        assert tiles1 < 256 and L["phase1_ds"] < L["phase1_tiles"] < L["phase3_tiles"]
    op.workspace.fill_(0x77)
    op.run()
    torch.cuda.synchronize()
    ws = op.workspace.cpu().numpy()
    i32 = lambda name, n: ws[L[name]:L[name] + 4 * n].view(np.int32)
    ext = i32("block_flag", N).astype(np.int64)
    if tiles1 < 256:
        want = _ranges(ext, 128, -(-I // 128), False, B)
        assert np.array_equal(i32("phase1_tiles", len(want)), want)
    wide = 2 * I % 128 == 0 and 2 * I >= 1024 and B >= 256 and H >= 256
    want = _ranges(ext, 256 if wide else 128, -(-H // 256), False, B)
    assert np.array_equal(i32("phase3_tiles", len(want)), want)
