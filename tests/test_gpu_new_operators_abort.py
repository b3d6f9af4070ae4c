"""The abort paths of the norms of many rows, the products with an epilogue and the expert
layer for a few tokens: a wait that runs out is reported, nothing that is not complete is
stored as a result, and the next call is right."""
import contextlib

import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


@contextlib.contextmanager
def _stalled(stall=1):
    try:
        B.nvfp4moe_set_wait_limit_ns(20_000_000)
        B.nvfp4moe_set_test_stall(stall)
        yield
        assert B.nvfp4moe_last_device_status() == -5
    finally:
        B.nvfp4moe_set_test_stall(0)
        B.nvfp4moe_set_wait_limit_ns(4_000_000_000)


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV)


@pytest.mark.parametrize("rows,K", [(1300, 6144), (2000, 7168)])
def test_norms(rows, K):
    x, r, dy = (_randn(s, rows, K).bfloat16() for s in (1, 2, 3))
    gamma = 1 + 0.1 * _randn(4, K)
    y, h = B.rms_norm(x, gamma, 1e-6, residual=r)
    want = B.rms_norm_backward(dy, h, gamma, 1e-6, dh=r)
    a, b, c = (torch.full_like(x, 7.0) for _ in range(3))
    with _stalled():
        B.rms_norm(x, gamma, 1e-6, residual=r, y=a, h=b)
    with _stalled():
        B.rms_norm_backward(dy, h, gamma, 1e-6, dh=r, dx=c)
    assert all((t == 7).all() for t in (a, b, c))
    B.rms_norm(x, gamma, 1e-6, residual=r, y=a, h=b)
    got = B.rms_norm_backward(dy, h, gamma, 1e-6, dh=r, dx=c)
    assert torch.equal(a, y) and torch.equal(b, h) and all(torch.equal(s, t) for s, t in zip(got, want))
    assert B.nvfp4moe_last_device_status() == 0


@pytest.mark.parametrize("stall", [1, 2])
@pytest.mark.parametrize("M,N,K", [(3, 512, 1024), (128, 4096, 7168), (2500, 1000, 384)])
def test_products(M, N, K, stall):
    a, sa = B.fp8_quantize(_randn(1, M, K))
    w, sw = B.fp8_quantize_weight(_randn(2, N, K))
    bias, res = _randn(3, N), _randn(4, M, N)
    for act in ("none", "silu"):
        good = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, residual=res, out_dtype=torch.float32)
        out = torch.full_like(good, 7.0)
        with _stalled(stall):
            B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, residual=res, out=out)
        assert (out == 7).all()
        B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, residual=res, out=out)
        assert torch.equal(out, good) and B.nvfp4moe_last_device_status() == 0


# h of all slots in shared memory; a counter for 32 columns; activations in pieces
@pytest.mark.parametrize("T,K,I,E,k", [(1, 512, 256, 8, 2), (8, 256, 2048, 16, 6), (32, 4096, 512, 4, 4)])
def test_few_tokens(T, K, I, E, k):
    x, logits = _randn(1, T, K).bfloat16(), _randn(2, T, E)
    weights = B.prepare_fp8_moe_weights(_randn(3, E, 2 * I, K) * K ** -0.5, _randn(4, E, K, I) * I ** -0.5)
    good = B.fp8_moe_few_tokens(x, logits, weights, k)
    y = torch.full_like(good, 7.0)
    with _stalled():
        B.fp8_moe_few_tokens(x, logits, weights, k, y=y)
    assert (y == 7).all()
    B.fp8_moe_few_tokens(x, logits, weights, k, y=y)
    assert torch.equal(y, good) and B.nvfp4moe_last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
@pytest.mark.parametrize("T,K,I,E,k", [(8, 256, 2048, 16, 6), (32, 512, 1024, 4, 4), (20, 1040, 2064, 3, 2)])
def test_few_tokens_joined_by_a_counter(T, K, I, E, k, dtype):
    """Warps that end beside others that gave up, in the form whose last unit joins the columns."""
    x, logits = _randn(1, T, K).to(dtype), _randn(2, T, E)
    weights = B.prepare_fp8_moe_weights(_randn(3, E, 2 * I, K) * K ** -0.5, _randn(4, E, K, I) * I ** -0.5)
    good = B.fp8_moe_few_tokens(x, logits, weights, k)
    y = torch.full_like(good, 7.0)
    for _ in range(3):
        with _stalled():
            B.fp8_moe_few_tokens(x, logits, weights, k, y=y)
        assert (y == 7).all()
    B.fp8_moe_few_tokens(x, logits, weights, k, y=y)
    assert torch.equal(y, good) and B.nvfp4moe_last_device_status() == 0
