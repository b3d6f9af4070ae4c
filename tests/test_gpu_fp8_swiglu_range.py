"""fp8_swiglu_quantize where a block has nothing but strongly negative gates, down to
where exp(-gate) overflows, and gates that are not finite: a scale is as near the exact
one there as in any other block."""
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def _e4m3(q):
    """Nearest E4M3 value of 64-bit numbers, ties to even."""
    mag = q.abs().clamp_max(448.0)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))) - 3)
    return torch.copysign(torch.round(mag / step) * step, q)


@pytest.mark.parametrize("dtype,lo,hi,size", [
    (dtype, lo, hi, 1.0) for dtype in (torch.bfloat16, torch.float16, torch.float32)
    for lo, hi in [(-1.0, 1.0), (-5.0, -1.0), (-20.0, -10.0), (-45.0, -30.0), (-65.0, -60.0), (20.0, 90.0)]] + [
    (torch.bfloat16, -88.5, -87.5, 1e30), (torch.float32, -88.7, -87.3, 1e30), (torch.float32, -88.0, -80.0, 1e37)])
def test_scales_and_codes(dtype, lo, hi, size):
    """In steps of 2^-24: the exponential 4, its argument's correction 2, the product
    with it, the sum and the two products of silu 1 each, the reciprocal 2: 12; the
    scale's quotient 1, a code's factor and product 2: below 2^-20, 16 of them."""
    M, I = 64, 1024
    g = torch.Generator().manual_seed(int(abs(lo) * 8))
    gate = torch.rand(M, I, generator=g) * (hi - lo) + lo
    gu = torch.cat([gate, torch.randn(M, I, generator=g) * size], 1).to(dtype)
    codes, sf = B.fp8_swiglu_quantize(gu.to(DEV))
    x, u = gu.double().chunk(2, 1)
    h = (x / (1 + torch.exp(-x)) * u).view(M, -1, 128)
    amax = h.abs().amax(-1, keepdim=True)
    assert (amax >= 2.0 ** -99).all()
    d = 2.0 ** -20
    far = ((sf.cpu().double() - amax[..., 0] / 448).abs() / (amax[..., 0] / 448)).max()
    assert far <= d, float(torch.log2(far))
    q = (h * (448.0 / amax)).abs()
    got = codes.view(F8).cpu().double().view(M, -1, 128).abs()
    assert ((got >= _e4m3(q * (1 - d))) & (got <= _e4m3(q * (1 + d)))).all()


def test_gates_that_overflow_or_are_not_finite():
    inf, nan = float("inf"), float("nan")
    gate = torch.tensor([-89.0, -1000.0, -3e38, 3e38, inf, inf, -inf, nan, 1.0, 1.0])
    up = torch.tensor([1e20, 1e20, 1e20, 1e-30, 1.0, 0.0, 1.0, 1.0, inf, nan])
    gu = torch.zeros(10, 32)
    gu[:, 0], gu[:, 16] = gate, up
    codes, sf = B.fp8_swiglu_quantize(gu.to(DEV))
    sf = sf[:, 0].cpu()
    assert (sf[:3] == 0).all() and (codes[:3].cpu() & 0x7F == 0).all()
    assert abs(float(sf[3]) / (3e8 / 448) - 1) <= 2.0 ** -20
    assert sf[4] == inf and sf[8] == inf and torch.isnan(sf[[5, 6, 7, 9]]).all()
