"""dropout_add and its backward on the GPU against the mask and the formula in 64 bits."""
import numpy as np
import pytest
import torch

from oracle import ffn

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
SIZES = [(1, 1), (1, 7), (3, 8), (5, 9), (2, 257), (64, 128), (33, 1000), (129, 1501), (7, 4096), (2000, 3)]


def _exact(x, p, seed, offset, residual=None):
    keep = ffn.dropout_keep(x.numel(), p, seed, offset).reshape(x.shape)
    y = np.where(keep, x.double().cpu().numpy() * ffn.dropout_scale(p), 0.0)
    return y if residual is None else y + residual.double().cpu().numpy(), keep


def _close(got, y, x, residual=None, p=0.0):
    # the scale's rounding, the product's and the sum's in fp32, then half a step of the output's type
    mag = np.abs(x.double().cpu().numpy()) * ffn.dropout_scale(p)
    if residual is not None:
        mag = mag + np.abs(residual.double().cpu().numpy())
    tol = mag * 3 * 2.0 ** -24 + np.abs(y) * torch.finfo(got.dtype).eps / 2
    assert (np.abs(got.double().cpu().numpy() - y) <= tol * (1 + 1e-9)).all()


def _rng(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("shape", SIZES)
def test_forward_and_backward(shape, dtype):
    import mxfp8_grouped_gemm_amd as mx
    g = torch.Generator("cuda").manual_seed(shape[0] * 7 + shape[1])
    x = torch.randn(shape, device="cuda", generator=g).to(DT[dtype])
    r = torch.randn(shape, device="cuda", generator=g).to(DT[dtype])
    for p, seed, off in ((0.1, 2 ** 61 + 5, 2 ** 40 + 1), (0.5, -3, -7), (0.0, 1, 2), (1.0, 1, 2)):
        rng = _rng(seed, off)
        s, o = seed % 2 ** 64, off % 2 ** 64
        y, keep = _exact(x, p, s, o, r)
        _close(mx.dropout_add(x, p, rng, residual=r), y, x, r, p)
        y, _ = _exact(x, p, s, o)
        plain = mx.dropout_add(x, p, rng)
        _close(plain, y, x, None, p)
        assert torch.equal(mx.dropout_add_bwd(x, p, rng), plain)      # the same mask, whatever came before
        if p == 1.0:
            assert not plain.any()
        if p == 0.0:
            assert torch.equal(mx.dropout_add(x, 0.0, None), x)


def test_gradient_by_differences():
    """dropout_add is linear in x: its differences are its derivative, and the backward's product with any direction."""
    import mxfp8_grouped_gemm_amd as mx
    g = torch.Generator("cuda").manual_seed(0)
    x, v, dy = (torch.randn(37, 65, device="cuda", generator=g) for _ in range(3))
    rng = _rng(11, 12)
    d = (mx.dropout_add(x + v, 0.3, rng).double() - mx.dropout_add(x, 0.3, rng).double())
    left, right = (d * dy.double()).sum(), (mx.dropout_add_bwd(dy, 0.3, rng).double() * v.double()).sum()
    # x + v and both results are rounded to fp32: 4 roundings of values below 16 over 2405 elements of |dy| below 5
    assert abs(left - right) <= 2405 * 4 * 16 * 2.0 ** -24 * 5


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("cols,ld", [(64, 80), (64, 68), (63, 70), (1, 9), (200, 201)])
def test_strides(cols, ld, dtype):
    """Rows at a stride: the mask is that of the contiguous tensor, and nothing between the rows is touched."""
    import mxfp8_grouped_gemm_amd as mx
    g = torch.Generator("cuda").manual_seed(cols)
    rows = 19
    base = [torch.randn(rows, ld, device="cuda", generator=g).to(DT[dtype]) for _ in range(3)]
    x, r, y = (b[:, :cols] for b in base)
    rest = base[2][:, cols:].clone()
    rng = _rng(3, 4)
    want = mx.dropout_add(x.contiguous(), 0.25, rng, residual=r.contiguous())
    mx.dropout_add(x, 0.25, rng, residual=r, out=y)
    assert torch.equal(y, want) and torch.equal(base[2][:, cols:], rest)
    assert torch.equal(mx.dropout_add(x, 0.25, rng, residual=r), want)
    mx.dropout_add(x, 0.25, rng, residual=r, out=x)      # in place
    assert torch.equal(x, want)


def test_dropped_values_do_not_matter():
    import mxfp8_grouped_gemm_amd as mx
    keep = torch.from_numpy(ffn.dropout_keep(4096, 0.4, 1, 2)).cuda()
    x = torch.ones(4096, device="cuda")
    x[~keep] = float("nan")
    x[5] = float("inf") if keep[5] else x[5]
    y = mx.dropout_add(x, 0.4, _rng(1, 2))
    assert not y[~keep].any() and not torch.isnan(y).any()


def test_past_32_bits():
    """Elements behind the 2^32nd byte and counters of a tensor of 2^31 elements."""
    import mxfp8_grouped_gemm_amd as mx
    rows, cols = 2 ** 15 + 1, 2 ** 16
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    y = mx.dropout_add(x, 0.5, _rng(8, 9))
    for i in (0, 2 ** 31 - 64, rows * cols - 64):
        w = ffn.philox_words(np.arange(i // 8, i // 8 + 8, dtype=np.uint64), 9, 8)
        keep = np.stack([w & 0xFFFF, w >> 16], -1).reshape(-1) >= 32768
        assert np.array_equal(y.view(-1)[i:i + 64].float().cpu().numpy(), keep * 2.0)


def test_graph_reads_the_generator_at_replay():
    import mxfp8_grouped_gemm_amd as mx
    x, rng = torch.randn(50, 72, device="cuda"), _rng(1, 0)
    out = mx.dropout_add(x, 0.5, rng)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        mx.dropout_add(x, 0.5, rng, out=out)
    for k in range(3):
        rng[1] = 100 + k
        want = mx.dropout_add(x, 0.5, rng)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
