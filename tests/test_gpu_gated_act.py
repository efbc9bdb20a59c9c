"""mxfp8_gated_act_fwd / _bwd on the GPU: codes and scales bit for bit against
the oracle's quantiser, inter and the gradient against fp64.

Rounding once to bf16 is off by at most 2^-8 of the value.  The fp32 evaluation
adds: sigmoid and the normal CDF with arguments rounded by 2^-24 |g| (|g| < 64
here; for the CDF's tail 2 g^2 2^-24), a few 2^-24 more: under 2^-15 of the
value; act'(g) crosses zero, where its terms of size (1 + |g|) round by 2^-23:
under 2^-18 |d u| in dGate.  Results under 2^-100 may be flushed on the way."""
import math

import numpy as np
import pytest
import torch

import mxfp8_grouped_gemm_amd as mx
import oracle
import synthetic as S

pytestmark = pytest.mark.gpu
REL, TINY = 2.0 ** -8 + 2.0 ** -15, 2.0 ** -100


def _act(g, geglu):
    from scipy.special import ndtr
    if geglu:
        return g * ndtr(g), ndtr(g) + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
    return g * s, s * (1 + g * (1 - s))


def _f64(t):
    return t.detach().double().cpu().numpy()


def _check_fwd(x, geglu, fmt, got):
    """x: the bf16 input [rows, 2, ...] with padding already zeroed."""
    inter, codes, scales = got
    n = x.shape[-1]
    bits = S.bf16_bits(x)
    rc, rs = oracle.quantize(bits.reshape(-1, n), 1, fmt)
    assert np.array_equal(codes.cpu().numpy().reshape(-1, n), rc)
    assert np.array_equal(scales.cpu().numpy().reshape(-1, n // 32), rs)
    v = _f64(x)
    ref = _act(v[:, 0], geglu)[0] * v[:, 1]
    assert np.all(np.abs(_f64(inter) - ref) <= REL * np.abs(ref) + TINY)


def _values(codes, scales, fmt):
    n = codes.shape[-1]
    v = oracle.dequantize(codes.cpu().numpy().reshape(-1, n), scales.cpu().numpy().reshape(-1, n // 32), 1, fmt)
    return np.asarray(v, dtype=np.float64).reshape(codes.shape)


def _check_bwd(d, codes, scales, geglu, fmt, got):
    v = _values(codes, scales, fmt)
    g, u, d = v[:, 0], v[:, 1], _f64(d)
    act, slope = _act(g, geglu)
    out = _f64(got)
    for k, ref in ((0, d * u * slope), (1, d * act)):
        assert np.all(np.abs(out[:, k] - ref) <= REL * np.abs(ref) + 2.0 ** -18 * np.abs(d * u) + TINY)


DENSE = [(1, 2, 32), (3, 2, 64), (77, 2, 352), (5, 2, 96), (33, 2, 4096), (257, 2, 2080)]
MOE = [(1, 2, 32, 128), (7, 2, 96, 128), (3, 2, 1408, 512), (5, 2, 64, 1024), (2, 2, 3, 96), (4, 2, 2, 32), (3, 2, 7, 2080)]


@pytest.mark.parametrize("geglu", [0, 1])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("shape", DENSE + MOE)
def test_matches_fp64_and_the_oracle(shape, fmt, geglu):
    print("gated act", shape, fmt, geglu, flush=True)
    x = S.normal_bf16(shape, 2.0, 3, 100 + shape[0], "cuda")
    _check_fwd(x, geglu, fmt, got := mx.mxfp8_gated_act_fwd(x, geglu, fmt))
    assert got[0].shape == shape[:1] + shape[2:] and got[1].shape == shape and got[2].shape[-1] == shape[-1] // 32
    d = S.normal_bf16(shape[:1] + shape[2:], 1.0, 4, 7, "cuda")
    dx = mx.mxfp8_gated_act_bwd(d, got[1], got[2], geglu, fmt)
    assert dx.shape == shape
    _check_bwd(d, got[1], got[2], geglu, fmt, dx)


@pytest.mark.parametrize("geglu", [0, 1])
@pytest.mark.parametrize("shape", MOE)
def test_padding_slots(shape, geglu):
    """Padding holds NaN, infinities and huge values: it reaches no scale, and its
    outputs are zero; the gradient ignores what the upstream holds there."""
    R, B = shape[0], shape[-1]
    rng = np.random.default_rng(R + B)
    T = R * B + 5
    ids = rng.integers(0, T, R * B).astype(np.int32)
    dead = rng.random(R * B) < 0.3
    dead[:B // 2] = True                      # whole groups without a token
    ids[dead] = rng.choice([-1, -7, T, 2 ** 31 - 1], int(dead.sum()))
    tp = torch.from_numpy(ids).cuda()
    pad = torch.from_numpy(dead).cuda().view(R, *([1] * (len(shape) - 2)), B)
    clean = S.normal_bf16(shape, 1.5, 9, 1, "cuda").masked_fill(pad, 0)
    junk = torch.tensor([math.nan, math.inf, -math.inf, 3e38], dtype=torch.bfloat16, device="cuda")
    junk = junk[torch.randint(0, 4, shape, device="cuda")]
    x = torch.where(pad, junk, clean)
    got = mx.mxfp8_gated_act_fwd(x, geglu, token_position_to_id=tp, T=T)
    _check_fwd(clean, geglu, 0, got)
    p2 = pad.expand(shape)
    assert not got[0][p2[:, 0]].any() and not got[1][p2].any()
    d = S.normal_bf16(shape[:1] + shape[2:], 1.0, 4, 7, "cuda")
    junk_codes = torch.where(p2, torch.full_like(got[1], 0x7f), got[1])
    dx = mx.mxfp8_gated_act_bwd(torch.where(p2[:, 0], junk[:, 0], d), junk_codes, got[2], geglu, token_position_to_id=tp, T=T)
    assert not dx[p2].any()
    _check_bwd(d.masked_fill(p2[:, 0], 0), got[1], got[2], geglu, 0, dx)


@pytest.mark.parametrize("fmt", [0, 1])
def test_every_bf16_pattern_and_every_code(fmt):
    """All finite bf16 magnitudes up to 2^60 as gates and ups: the codes of the oracle; then all codes of
    the format at scales across the range, as the backward reads them."""
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    bits = bits[(bits & 0x7FFF) < ((127 + 60) << 7)]
    rng = np.random.default_rng(fmt)
    n = bits.size // 64 * 64
    g = bits[rng.permutation(bits.size)[:n]].reshape(-1, 1, 64)
    u = np.full_like(g, 0x3F80)               # up = 1: inter = act(g)
    x = S.from_bits(np.concatenate([g, u], 1), "cuda")
    inter, codes, scales = mx.mxfp8_gated_act_fwd(x, 0, fmt)
    rc, rs = oracle.quantize(S.bf16_bits(x).reshape(-1, 64), 1, fmt)
    assert np.array_equal(codes.cpu().numpy().reshape(-1, 64), rc) and np.array_equal(scales.cpu().numpy().reshape(-1, 2), rs)
    v = _f64(x)
    ref = _act(v[:, 0], 0)[0]
    # below -88 the fp32 sigmoid saturates to 0, where |silu| < 100 * 2^-126
    assert np.all(np.abs(_f64(inter) - ref) <= REL * np.abs(ref) + 100 * 2.0 ** -126)
    every = np.arange(256, dtype=np.uint8)
    nan = (every & 0x7F) == 0x7F if fmt == 0 else (every & 0x7C) == 0x7C
    every = np.resize(every[~nan], (256,))
    c = np.stack([np.tile(every, (5, 1)), np.tile(every[::-1], (5, 1))], 1)   # [5, 2, 256]
    s = np.repeat(np.array([[60], [110], [119], [124], [0]], dtype=np.uint8), 16, 1).reshape(5, 2, 8)
    d = torch.ones(5, 256, dtype=torch.bfloat16, device="cuda")
    cc, ss = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()
    _check_bwd(d, cc, ss, 0, fmt, mx.mxfp8_gated_act_bwd(d, cc, ss, 0, fmt))


def test_gradient_is_the_forward_difference():
    """The backward of a checkpoint against central differences of act(g) u in
    fp64 at the checkpoint's values (step 1e-4: off by 1e-8, under the bf16 rounding)."""
    x = S.normal_bf16((9, 2, 128), 2.0, 5, 5, "cuda")
    for geglu in (0, 1):
        _, codes, scales = mx.mxfp8_gated_act_fwd(x, geglu)
        d = S.normal_bf16((9, 128), 1.0, 6, 6, "cuda")
        got = _f64(mx.mxfp8_gated_act_bwd(d, codes, scales, geglu))
        v, dd, h = _values(codes, scales, 0), _f64(d), 1e-4
        f = lambda g, u: _act(g, geglu)[0] * u * dd
        for k, (dg, du) in enumerate(((h, 0), (0, h))):
            fd = (f(v[:, 0] + dg, v[:, 1] + du) - f(v[:, 0] - dg, v[:, 1] - du)) / (2 * h)
            assert np.all(np.abs(got[:, k] - fd) <= REL * np.abs(fd) + 2.0 ** -18 * np.abs(dd * v[:, 1]) + 1e-7)


def test_offsets_past_32_bits():
    """Over 2^32 bytes and 2^31 elements: the last rows equal a call on them alone."""
    R, C, tail = 33000, 65536, 3
    x = torch.zeros((R, 2, C), dtype=torch.bfloat16, device="cuda")
    x[-tail:] = S.normal_bf16((tail, 2, C), 2.0, 3, 3, "cuda")
    inter, codes, scales = mx.mxfp8_gated_act_fwd(x)
    small = mx.mxfp8_gated_act_fwd(x[-tail:].contiguous())
    assert all(torch.equal(a[-tail:], b) for a, b in zip((inter, codes, scales), small))
    assert not inter[:-tail].any() and not codes[:-tail].any()
    del x
    inter[-tail:] = S.normal_bf16((tail, C), 1.0, 4, 4, "cuda")
    d = mx.mxfp8_gated_act_bwd(inter, codes, scales)
    assert torch.equal(d[-tail:], mx.mxfp8_gated_act_bwd(inter[-tail:].contiguous(), small[1], small[2]))
    assert not d[:-tail].any()


def test_empty_stream_graph_and_guard_bytes():
    x = S.normal_bf16((10, 2, 160), 1.0, 1, 1, "cuda")
    assert mx.mxfp8_gated_act_fwd(x[:0])[1].shape == (0, 2, 160)
    assert mx.mxfp8_gated_act_bwd(x[:0, 0].contiguous(), torch.empty(0, 2, 160, dtype=torch.uint8, device="cuda"),
                                  torch.empty(0, 2, 5, dtype=torch.uint8, device="cuda")).shape == (0, 2, 160)
    n = x.numel()
    guard = torch.full((n + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    sguard = torch.full((n // 32 + 256,), 0xAB, dtype=torch.uint8, device="cuda")
    iguard = torch.full((n // 2 + 256,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = (iguard[:n // 2].view(10, 160), guard[:n].view(10, 2, 160), sguard[:n // 32].view(10, 2, 5))
    dx, d = torch.empty_like(x), S.normal_bf16((10, 160), 1.0, 2, 2, "cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()

    def step():
        mx.mxfp8_gated_act_fwd(x, out=out)
        mx.mxfp8_gated_act_bwd(d, out[1], out[2], out=dx)

    with torch.cuda.stream(s):
        step()
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.synchronize()
    for k in range(3):
        x.copy_(S.normal_bf16((10, 2, 160), 1.0 + k, k, 1, "cuda"))
        graph.replay()
        torch.cuda.synchronize()
        _check_fwd(x, 0, 0, out)
        _check_bwd(d, out[1], out[2], 0, 0, dx)
    assert guard[n:].eq(0xAB).all() and sguard[n // 32:].eq(0xAB).all() and iguard[n // 2:].eq(7).all()


def test_geglu_over_the_whole_range():
    """Every bf16 gate in (-16, 16) and some far outside, with ups and upstreams of 1:
    g Phi(g) and its slope, relatively also in the left tail, where both fall
    below 1e-38 at g = -13."""
    from scipy.special import ndtr
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    bits = bits[(bits & 0x7FFF) < 0x4180]
    bits = np.concatenate([bits, np.array([0x7F00, 0xFF00, 0x4300, 0xC300, 0x4200, 0xC200], dtype=np.uint16)])
    g = np.resize(bits, (-(-bits.size // 32) * 32,)).reshape(-1, 1, 32)
    x = S.from_bits(np.concatenate([g, np.full_like(g, 0x3F80)], 1), "cuda")
    inter, codes, scales = mx.mxfp8_gated_act_fwd(x, mx.ACT_GEGLU)
    v = _f64(x)[:, 0]
    with np.errstate(over="ignore"):
        ref = v * ndtr(v)
    assert np.all(np.abs(_f64(inter) - ref) <= REL * np.abs(ref) + 2.0 ** -120)
    # the backward on gates that the codes hold exactly: 4 significant bits, one scale a group
    c = np.resize(np.arange(256, dtype=np.uint8)[(np.arange(256) & 0x7F) != 0x7F], 256).reshape(1, 256)
    cc = torch.from_numpy(np.stack([c, np.full_like(c, 0x38)], 1)).cuda()      # ups: 1
    ss = torch.from_numpy(np.stack([np.full((1, 8), 122, np.uint8), np.full((1, 8), 127, np.uint8)], 1)).cuda()
    d = torch.ones(1, 256, dtype=torch.bfloat16, device="cuda")
    _check_bwd(d, cc, ss, 1, 0, mx.mxfp8_gated_act_bwd(d, cc, ss, mx.ACT_GEGLU))
