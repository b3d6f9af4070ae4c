"""The abort path of the 8-bit products: whichever role gives up, the call is
reported, a tile whose sums are not complete is not stored, and the next call is
right."""
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _codes(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    return B.fp8_quantize(torch.randn(M, K, generator=g).to(DEV))


# few rows: blocks of K that a cluster shares, all issued before the abort; one CTA
# a tile; 128-row tiles shared by a cluster; one CTA a tile
@pytest.mark.parametrize("stall", [1, 2])
@pytest.mark.parametrize("M,N,K", [(3, 512, 1024), (40, 512, 1024), (16, 24000, 256), (128, 4096, 7168),
                                   (700, 512, 128), (2500, 1000, 384)])
def test_nothing_is_stored_of_a_tile_that_is_not_complete(M, N, K, stall):
    a, sa = _codes(M, K, 1)
    g = torch.Generator().manual_seed(2)
    w, sw = B.fp8_quantize_weight(torch.randn(N, K, generator=g).to(DEV))
    good = B.fp8_linear(a, sa, w, sw)
    assert B.nvfp4moe_last_device_status() == 0
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    try:
        B.nvfp4moe_set_wait_limit_ns(20_000_000)
        B.nvfp4moe_set_test_stall(stall)
        B.fp8_linear(a, sa, w, sw, out=out)
        assert B.nvfp4moe_last_device_status() == -5
    finally:
        B.nvfp4moe_set_test_stall(0)
        B.nvfp4moe_set_wait_limit_ns(4_000_000_000)
    assert (out == 7).all()
    B.fp8_linear(a, sa, w, sw, out=out)
    assert torch.equal(out, good) and B.nvfp4moe_last_device_status() == 0


@pytest.mark.parametrize("stall", [1, 2])
def test_groups(stall):
    E, N, K = 40, 384, 512
    counts = [i % 5 for i in range(E)]
    bounds = [sum(counts[:e]) for e in range(E + 1)]
    a, sa = _codes(bounds[-1], K, 3)
    g = torch.Generator().manual_seed(4)
    w, sw = B.fp8_quantize_weight(torch.randn(E, N, K, generator=g).to(DEV))
    off = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    good = B.fp8_grouped_gemm(a, sa, w, sw, off)
    out = torch.full_like(good, 7.0)
    try:
        B.nvfp4moe_set_wait_limit_ns(20_000_000)
        B.nvfp4moe_set_test_stall(stall)
        B.fp8_grouped_gemm(a, sa, w, sw, off, out=out)
        assert B.nvfp4moe_last_device_status() == -5
    finally:
        B.nvfp4moe_set_test_stall(0)
        B.nvfp4moe_set_wait_limit_ns(4_000_000_000)
    assert (out == 7).all()
    assert torch.equal(B.fp8_grouped_gemm(a, sa, w, sw, off), good) and B.nvfp4moe_last_device_status() == 0
