"""mxfp8_quantize_transposed on the GPU: the oracle's codes and scales of the transposed matrix, bit for bit."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [oracle.E4M3, oracle.E5M2])
@pytest.mark.parametrize("G,R,C", [(1, 32, 1), (1, 32, 2), (3, 96, 77), (2, 128, 128), (1, 160, 129), (5, 64, 1000), (2, 608, 130), (3, 160, 255),
                                   (1, 4096, 34), (40, 32, 64), (1, 64, 385), (2, 32, 127)])
def test_codes_and_scales(G, R, C, fmt):
    import mxfp8_grouped_gemm_amd as mx
    r = np.random.default_rng(G * R + C)
    x = (r.standard_normal((G, R, C)) * np.exp2(r.integers(-30, 30, (G, R, C)))).astype(np.float32)
    x[0, :32, 0] = 0.0
    t = torch.from_numpy(x).to(torch.bfloat16)
    bits = t.transpose(1, 2).contiguous().view(torch.int16).numpy().view(np.uint16).reshape(G * C, R)
    codes, scales = oracle.quantize(bits, 1, fmt)
    c, s = mx.mxfp8_quantize_transposed(t.cuda(), fmt)
    assert c.shape == (G, C, R) and s.shape == (G, C, R // 32)
    assert np.array_equal(c.cpu().numpy().reshape(codes.shape), codes)
    assert np.array_equal(s.cpu().numpy().reshape(scales.shape), scales)
    out = torch.full_like(c, 9), torch.full_like(s, 9)
    assert mx.mxfp8_quantize_transposed(t.cuda(), fmt, out=out) is out
    assert torch.equal(out[0], c) and torch.equal(out[1], s)
    if G == 1:
        assert torch.equal(mx.mxfp8_quantize_transposed(t[0].cuda(), fmt)[0], c[0])


def test_past_32_bits():
    """A batch whose last matrix lies behind the 2^32nd byte."""
    import mxfp8_grouped_gemm_amd as mx
    x = torch.zeros(33, 8192, 8224, dtype=torch.bfloat16, device="cuda")
    x[-1, -32:, -1] = torch.arange(1, 33, device="cuda").to(torch.bfloat16)
    c, s = mx.mxfp8_quantize_transposed(x)
    one = mx.mxfp8_quantize_transposed(x[-1].contiguous())
    assert torch.equal(c[-1], one[0]) and torch.equal(s[-1], one[1])
    assert not c[-1, :-1].any() and not c[:-1].any() and int(s[-1, -1, -1]) == 127 + 5 - 8


@pytest.mark.parametrize("shift", [1, 2, 4])
def test_scales_of_any_alignment(shift):
    import mxfp8_grouped_gemm_amd as mx
    x = torch.randn(2, 256, 70, device="cuda").to(torch.bfloat16)
    want = mx.mxfp8_quantize_transposed(x)
    buf = torch.full((2 * 70 * 8 + 16,), 77, dtype=torch.uint8, device="cuda")
    s = buf[shift:shift + 2 * 70 * 8].view(2, 70, 8)
    c, _ = mx.mxfp8_quantize_transposed(x, out=(torch.empty_like(want[0]), s))
    assert torch.equal(c, want[0]) and torch.equal(s, want[1])
    assert (buf[:shift] == 77).all() and (buf[shift + 2 * 70 * 8:] == 77).all()
