"""The 64-bit definitions that the MoE forward and dropout are held to, pinned by published vectors, hand-worked values
and the other oracle."""
import numpy as np
import pytest

import oracle
from oracle import ffn


def test_philox_known_answers():
    """The known-answer vectors that the generator's authors publish for philox4x32-10."""
    def words(c, k):
        return [int(w) for w in ffn.philox_words(np.array([c[0] | c[1] << 32], np.uint64), c[2] | c[3] << 32,
                                                 k[0] | k[1] << 32)[0]]
    f = 0xFFFFFFFF
    assert words((0, 0, 0, 0), (0, 0)) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert words((f, f, f, f), (f, f)) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert words((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == [
        0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout_mask(p):
    n = 80003
    keep = ffn.dropout_keep(n, p, seed=5, offset=9)
    q = ffn.dropout_threshold(p) / 65536
    assert abs(keep.mean() - (1 - q)) <= 5 * np.sqrt(max(q * (1 - q), 1e-12) / n)
    assert q == 1 or ffn.dropout_scale(p) * (1 - q) == pytest.approx(1)
    assert np.array_equal(keep[:1001], ffn.dropout_keep(1001, p, 5, 9))       # element by element, whatever the size
    if 0 < p < 1:
        other = ffn.dropout_keep(n, p, 5, 10)
        assert abs((keep == other).mean() - (q * q + (1 - q) ** 2)) < 0.01    # another offset: another mask


@pytest.mark.parametrize("fmt", [oracle.E4M3, oracle.E5M2])
def test_requantisation_is_the_other_oracles(fmt):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((64, 96)) * np.exp2(rng.integers(-20, 20, (64, 96)))).astype(np.float32)
    bits = (x.view(np.uint32) >> 16).astype(np.uint16)
    v = oracle.bf16_to_float(bits).astype(np.float64)
    codes, scales = oracle.quantize(bits, 1, fmt)
    got, X = ffn.mx_requant(v, fmt)
    assert np.array_equal(X + 127, scales)
    assert np.array_equal(got, ffn.mx_values(codes, scales, fmt))


def test_requantisation_bounds():
    v = np.zeros(32)
    v[0], v[1], v[2] = 256.0, 1.0 + 1 / 16, 100.0      # scale 1; 17/16 lies between the codes 1 and 9/8
    base, off = ffn.mx_requant_bounds(v, np.full(32, 1e-6))
    assert base[1] == 1.0 and off[1] == 0.125 and off[2] == 8.0     # 100 lies between 96 and 104
    v[0] = 256.0 - 1e-7                                 # the scale may be 1/2 or 1
    _, off = ffn.mx_requant_bounds(v, np.full(32, 1e-6))
    assert off[0] >= 30                                 # 224 (saturated at 448 / 2) or 256


def test_one_pair_by_hand():
    """One token, one expert, H = I = 32, identity weights: y = Q(silu(x) x) with a = 1/2."""
    H = I = 32
    x = np.zeros((1, H))
    x[0, 0], x[0, 1] = 2.0, -1.0
    eye = np.eye(32)
    y, dy, gus = ffn.moe_fwd(x, {0: ([0], [0.5])}, np.stack([eye, eye])[None], eye[None])
    s = np.array([2 * 2 / (1 + np.exp(-2.0)), 1 / (1 + np.exp(1.0))])          # 3.523, 0.269
    # scale 2^(1-8): steps of 1/4 at 3.5 and 1/32 at 0.27
    assert np.allclose(y[0, :2], [0.5 * round(s[0] * 4) / 4, 0.5 * round(s[1] * 32) / 32])
    assert not y[0, 2:].any() and gus[0][0].shape == (1, 2, 32)
    assert (dy[0, :2] < 0.01 * np.abs(y[0, :2])).all()
    keep = np.ones((1, H), bool)
    keep[0, 0] = False
    z, _, _ = ffn.moe_fwd(x, {0: ([0], [0.5])}, np.stack([eye, eye])[None], eye[None], keep=keep, scale=2.0,
                          residual=np.ones((1, H)))
    assert z[0, 0] == 1.0 and z[0, 1] == pytest.approx(1 + 2 * y[0, 1])


def test_product_rests_by_hand():
    """Products below 2^(E - 13) of their 8 are cut off whole, others to a multiple; other groups keep their own unit."""
    a, b = np.ones((1, 32)), np.zeros((2, 32))
    b[0, 0], b[0, 1], b[0, 2] = 1.0, 2.0 ** -14, -1.5 * 2.0 ** -13      # unit 2^-13
    b[0, 8] = 2.0 ** -14
    b[1, :2] = 1.75 * 2.0 ** -10, 1.25
    assert np.array_equal(ffn.product_rests(a, b), [[2.0 ** -14 + 0.5 * 2.0 ** -13, 0.0]])
