"""Sorted tokens and quantized rows of a rank that holds none of them, and rows
without columns."""
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,K", [(5, 2, 24), (700, 8, 1001), (2500, 4, 8)])
def test_no_rows(T, k, K, dtype):
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    rows = torch.empty((0, K), dtype=dtype, device=DEV)
    f2p = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
    w = torch.ones((T, k), device=DEV)
    assert B.moe_sort_tokens(x, f2p, k, topk_w=w, n_rows=0).shape == (0, K)
    d_rows, d_w = B.moe_unsort_tokens_backward(x, f2p, k, topk_w=w, rows=rows)
    assert d_rows.shape == (0, K) and d_w.shape == (T, k) and (d_w == 0).all()
    dx, d_w = B.moe_sort_tokens_backward(rows, f2p, k, topk_w=w, x=x)
    assert (dx == 0).all() and (d_w == 0).all()
    assert (B.moe_unsort_tokens(rows, f2p, k, topk_w=w) == 0).all()
    assert B.nvfp4moe_last_device_status() == 0
    # a slot that names a row all the same is reported
    f2p[3] = 0
    assert (B.moe_unsort_tokens_backward(x, f2p, k, topk_w=w, rows=rows)[1] == 0).all()
    assert B.nvfp4moe_last_device_status() == -1


@pytest.mark.parametrize("T,k", [(6, 3), (3000, 2)])
def test_no_columns(T, k):
    x, rows = torch.empty((T, 0), device=DEV), torch.empty((T * k, 0), device=DEV)
    f2p = torch.arange(T * k, dtype=torch.int32, device=DEV)
    w = torch.ones((T, k), device=DEV)
    assert B.moe_sort_tokens(x, f2p, k, topk_w=w).shape == (T * k, 0)
    assert B.moe_unsort_tokens(rows, f2p, k, topk_w=w).shape == (T, 0)
    for got, d_w in (B.moe_unsort_tokens_backward(x, f2p, k, topk_w=w, rows=rows),
                     B.moe_sort_tokens_backward(rows, f2p, k, topk_w=w, x=x)):
        assert got.numel() == 0 and d_w.shape == (T, k) and (d_w == 0).all()
    assert B.nvfp4moe_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_quantized_to_no_output_rows(dtype):
    x = torch.ones((7, 528), dtype=dtype, device=DEV)
    f2p = torch.full((14,), -1, dtype=torch.int32, device=DEV)
    codes, sf = B.fp8_quantize(x, flat_to_perm=f2p, k=2, out_rows=0)
    assert codes.shape == (0, 528) and sf.shape == (0, 5) and B.nvfp4moe_last_device_status() == 0
    f2p[5] = 0
    B.fp8_quantize(x, flat_to_perm=f2p, k=2, out_rows=0)
    assert B.nvfp4moe_last_device_status() == -1
