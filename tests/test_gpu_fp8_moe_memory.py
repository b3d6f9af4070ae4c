"""fp8_moe_forward takes its workspace and weights from device memory only, and a
workspace of any type by its bytes."""
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_memory():
    T, K, I, E, k = 20, 256, 128, 8, 2
    g = torch.Generator().manual_seed(1)
    x, logits = torch.randn(T, K, generator=g).bfloat16().to(DEV), torch.randn(T, E, generator=g).to(DEV)
    weights = B.prepare_fp8_moe_weights(torch.randn(E, 2 * I, K, generator=g).to(DEV),
                                        torch.randn(E, K, I, generator=g).to(DEV))
    n = B.fp8_moe_forward_workspace_size(T, K, I, E, k)
    want = B.fp8_moe_forward(x, logits, weights, k)
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(n, dtype=torch.uint8, pin_memory=True),
                torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2]):
        with pytest.raises(B.NVFP4Error):
            B.fp8_moe_forward(x, logits, weights, k, ws=bad)
    for name in ("w1_codes", "w1_sf", "w2_codes", "w2_sf"):
        with pytest.raises(B.NVFP4Error):
            B.fp8_moe_forward(x, logits, dict(weights, **{name: weights[name].cpu()}), k)
    ws = torch.empty(-(-n // 4), dtype=torch.float32, device=DEV)
    assert torch.equal(B.fp8_moe_forward(x, logits, weights, k, ws=ws), want)
    assert B.nvfp4moe_last_device_status() == 0
