"""moe_fp8_quantize_weights at the ends of its contract: blocks of the smallest
values, and rows of codes wider than their blocks."""
import pytest
import torch

from quantized_routed_expert_gemv_gb300 import moe
from quantized_routed_expert_gemv_gb300.device import Fp8Linear

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("most", [1, 2, 100, 223, 224, 225, 500, 1 << 20])
def test_blocks_of_the_smallest_values(most):
    """Largest magnitudes of `most` units of 2^-149: no code is NaN, and an
    output is 0 to within all that the weights can add to it."""
    n, k = 140, 200
    bits = torch.zeros(n, k, dtype=torch.int32, device=DEV)
    bits[::3, ::2] = most
    bits[1::3, 1::2] = -(1 << 31) + most // 2
    w = bits.view(torch.float32)
    assert w.abs().max().item() > 0
    lin = Fp8Linear.from_weights(w, 4)
    x = torch.ones(4, k, device=DEV)
    out = lin(x, out_type=torch.float32)
    torch.cuda.synchronize()
    assert not ((lin.codes[:, :k] & 127) == 127).any()
    assert (lin.scales > 0).all() and torch.isfinite(lin.scales).all()
    assert (out.abs() <= 2.0 * k * most * 2.0 ** -149).all()


@pytest.mark.parametrize("n,k,ld", [(3, 100, 112), (130, 100, 128), (130, 100, 144), (5, 128, 256), (300, 300, 1040),
                                    (129, 257, 4096), (1, 1, 16), (2, 384, 384)])
def test_bytes_past_k_are_zero(n, k, ld):
    """Whatever the width of a row of codes, and nothing after the last row."""
    g = torch.Generator(device=DEV).manual_seed(n)
    w = torch.randn(n, k, generator=g, device=DEV)
    buf = torch.full((n * ld + 64,), 0xAB, dtype=torch.uint8, device=DEV)
    scales = torch.empty(-(-n // 128), -(-k // 128), device=DEV)
    moe.moe_fp8_quantize_weights(w.data_ptr(), moe.MOE_F32, k, n, k, buf.data_ptr(), ld, scales.data_ptr())
    torch.cuda.synchronize()
    codes = buf[:n * ld].view(n, ld)
    assert (codes[:, k:] == 0).all()
    assert (buf[n * ld:] == 0xAB).all()
    assert torch.equal(codes[:, :k], Fp8Linear.from_weights(w, 1).codes[:, :k])
