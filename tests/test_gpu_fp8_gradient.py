"""The gradient of an 8-bit product with respect to A is a product with W's codes and
scales transposed: against the formula in 64 bits."""
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _values(codes, sf, each):
    v = codes.view(torch.float8_e4m3fn).double()
    s = sf.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]
    if each > 1:
        s = s.repeat_interleave(each, -2)[..., :codes.shape[-2], :]
    return v * s


def _close(got, dc, w):
    """f32 sums of N products, each within a step of the summed magnitudes, and the
    scales' product and its use."""
    N = dc.shape[1]
    want, size = dc @ w, dc.abs() @ w.abs()
    assert ((got.double() - want).abs() <= (N + -(-N // 128) + 2) * 2.0 ** -23 * size).all()


@pytest.mark.parametrize("M,N,K", [(1, 4096, 512), (40, 272, 400), (300, 640, 1040), (2000, 512, 300)])
def test_linear(M, N, K):
    g = torch.Generator().manual_seed(M)
    w, sw = B.fp8_quantize_weight(torch.randn(N, -(-K // 16) * 16, generator=g).to(DEV))
    w = w[:, :K]
    dc, sdc = B.fp8_quantize(torch.randn(M, N, generator=g).to(DEV))
    da = B.fp8_linear(dc, sdc, w.t().contiguous(), sw.t().contiguous(), out_dtype=torch.float32)
    _close(da, _values(dc, sdc, 1), _values(w, sw, 128))


def test_grouped():
    counts, N, K = [0, 30, 1, 200, 17], 400, 272
    E, M = len(counts), sum(counts)
    g = torch.Generator().manual_seed(9)
    w, sw = B.fp8_quantize_weight(torch.randn(E, N, K, generator=g).to(DEV))
    dc, sdc = B.fp8_quantize(torch.randn(M, N, generator=g).to(DEV))
    bounds = [sum(counts[:e]) for e in range(E + 1)]
    off = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    da = B.fp8_grouped_gemm(dc, sdc, w.transpose(1, 2).contiguous(), sw.transpose(1, 2).contiguous(), off,
                            out_dtype=torch.float32)
    vc, vw = _values(dc, sdc, 1), _values(w, sw, 128)
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        _close(da[lo:hi], vc[lo:hi], vw[e])
    assert B.nvfp4moe_last_device_status() == 0
