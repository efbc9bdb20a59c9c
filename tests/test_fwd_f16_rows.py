"""The stated accuracy of the MoE forward's rows in scaled fp16 (include/mxfp8_moe.h, csrc/moe_fwd_down.hip), by their
arithmetic in numpy, without a GPU."""
import numpy as np


def _through_f16(v):
    """64 fp32 values a row through fp16 times the power of two that puts the largest in [2^14, 2^15)."""
    top = np.abs(v).max(-1, keepdims=True).astype(np.float32)
    ex = np.maximum(top.view(np.int32) >> 23, 15)
    mul = np.ldexp(np.float32(1), 141 - ex).astype(np.float32)
    return np.ldexp((v * mul).astype(np.float16).astype(np.float64), ex - 141)


def _rows(n, seed):
    r = np.random.default_rng(seed)
    e = -r.integers(0, 45, (n, 64)) * (r.random((n, 64)) < 0.9)
    v = (1 + r.random((n, 64))) * np.exp2(e) * np.exp2(r.integers(-60, 60, (n, 1))) * r.choice([-1, 1], (n, 64))
    return v.astype(np.float32)


def test_the_stated_bound_holds_and_is_no_looser_than_it_has_to_be():
    v = _rows(20000, 1)
    off, size = np.abs(_through_f16(v) - v), np.abs(v).astype(np.float64)
    top = size.max(-1, keepdims=True)
    normal = size >= top * 2.0 ** -28
    assert (off[normal] <= size[normal] * 2.0 ** -11).all()
    assert (off <= np.maximum(size * 2.0 ** -11, top * 2.0 ** -39)).all()
    assert (off[normal] > size[normal] * 2.0 ** -12).any()          # half of it would not hold
    below = (size < top * 2.0 ** -28) & (size > top * 2.0 ** -30)
    assert (off[below] > size[below] * 2.0 ** -11).any()            # nor the relative one further down
