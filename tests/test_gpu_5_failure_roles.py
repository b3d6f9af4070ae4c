"""An abort of the NVFP4 products that comes from the epilogue, when the producer and the
MMA issuer have issued all of their work (short products), or not: reported, and the
next call is right."""
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _operands(E, K, N, per):
    g = torch.Generator().manual_seed(K + N)
    M = E * per
    offsets = torch.arange(0, M + 1, per, dtype=torch.int32).to(DEV)
    rows = B.nvfp4moe_padded_rows(M, E)
    a_codes = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, generator=g).to(DEV)
    a_sf = torch.full((B.nvfp4_sf_bytes(rows, K, B.NVFP4_SF_TILED_ROWS),), 0x38, dtype=torch.uint8, device=DEV)
    b_codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, generator=g).to(DEV)
    b_sf = torch.full((E * B.nvfp4_sf_bytes(N, K),), 0x38, dtype=torch.uint8, device=DEV)
    return a_codes, a_sf, torch.ones(1, device=DEV), b_codes, b_sf, torch.ones(E, device=DEV), offsets


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("stall", [1, 2])
@pytest.mark.parametrize("E,K,N,per", [(2, 256, 256, 100), (4, 1024, 256, 200), (8, 2048, 4096, 300), (3, 512, 384, 20)])
def test_whichever_role_gives_up(E, K, N, per, stall, mode):
    ops = _operands(E, K, N, per)
    B.nvfp4moe_set_gemm_mode(mode)
    try:
        good = B.nvfp4_grouped_gemm(*ops).clone()
        assert B.nvfp4moe_last_device_status() == 0
        try:
            B.nvfp4moe_set_wait_limit_ns(20_000_000)
            B.nvfp4moe_set_test_stall(stall)
            B.nvfp4_grouped_gemm(*ops)
            status = B.nvfp4moe_last_device_status()
        finally:
            B.nvfp4moe_set_test_stall(0)
            B.nvfp4moe_set_wait_limit_ns(4_000_000_000)
        assert status == -5
        assert torch.equal(B.nvfp4_grouped_gemm(*ops), good)
        assert B.nvfp4moe_last_device_status() == 0
    finally:
        B.nvfp4moe_set_gemm_mode(0)
