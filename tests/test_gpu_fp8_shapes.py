"""Shapes of scales, weights and slots: a transposed one has as many elements, and is
refused; one without its dimensions of 1, or flat, is the same memory and is taken."""
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _operands(M=6, E=3, N=300, K=512):
    a, sa = B.fp8_quantize(torch.randn(M, K, generator=torch.Generator().manual_seed(1)).to(DEV))
    w, sw = B.fp8_quantize_weight(torch.randn(E, N, K, generator=torch.Generator().manual_seed(2)).to(DEV))
    return a, sa, w, sw, torch.tensor([0, 2, 3, 6], dtype=torch.int32, device=DEV)


def _refused(call):
    with pytest.raises(B.NVFP4Error):
        call()


def test_products():
    a, sa, w, sw, off = _operands()
    want, grouped = B.fp8_linear(a, sa, w[0], sw[0]), B.fp8_grouped_gemm(a, sa, w, sw, off)
    for bad in (sa.t().contiguous(), sa.view(3, 8), sa.view(2, 3, 4)):
        _refused(lambda: B.fp8_linear(a, bad, w[0], sw[0]))
        _refused(lambda: B.fp8_grouped_gemm(a, bad, w, sw, off))
    _refused(lambda: B.fp8_linear(a, sa, w[0], sw[0].t().contiguous()))
    for bad in (sw.transpose(1, 2).contiguous(), sw.view(9, 4)):
        _refused(lambda: B.fp8_grouped_gemm(a, sa, w, bad, off))
    _refused(lambda: B.fp8_grouped_gemm(a, sa, w, sw, off.view(2, 2)))
    for same in (sa.view(1, 6, 4), sa.view(-1)):
        assert torch.equal(B.fp8_linear(a, same, w[0], sw[:1]), want)
        assert torch.equal(B.fp8_grouped_gemm(a, same, w, sw.view(-1), off.view(1, 4)), grouped)
    one = B.fp8_linear(a[:1], sa[:1], w[0], sw[0])
    for same in (sa[0], sa[:1].t().contiguous(), sa[:1]):
        assert torch.equal(B.fp8_linear(a[:1], same, w[0], sw[0]), one)


def test_outputs_of_the_quantizers():
    x = torch.randn(6, 512, generator=torch.Generator().manual_seed(3)).to(DEV)
    codes, sf = torch.empty((6, 512), dtype=torch.uint8, device=DEV), torch.empty((6, 4), device=DEV)
    _refused(lambda: B.fp8_quantize(x, codes=codes.view(512, 6), sf=sf))
    _refused(lambda: B.fp8_quantize(x, codes=codes, sf=sf.view(4, 6)))
    _refused(lambda: B.fp8_swiglu_quantize(torch.cat([x, x], 1), codes=codes, sf=sf.view(4, 6)))
    want = B.fp8_quantize(x)
    B.fp8_quantize(x, codes=codes.view(-1), sf=sf.view(1, 6, 4))
    assert torch.equal(codes, want[0]) and torch.equal(sf, want[1])


def test_slots_and_weights():
    T, k, K = 4, 2, 24
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(4)).to(DEV)
    f2p = torch.randperm(T * k, generator=torch.Generator().manual_seed(5)).int().to(DEV)
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(6)).to(DEV)
    rows = B.moe_sort_tokens(x, f2p, k, topk_w=w)
    _refused(lambda: B.moe_sort_tokens(x, f2p.view(k, T), k, topk_w=w))
    _refused(lambda: B.moe_sort_tokens(x, f2p, k, topk_w=w.t().contiguous()))
    _refused(lambda: B.moe_unsort_tokens(rows, f2p, k, topk_w=w.t().contiguous()))
    _refused(lambda: B.moe_unsort_tokens_backward(x, f2p.view(k, T), k, topk_w=w, rows=rows))
    assert torch.equal(B.moe_sort_tokens(x, f2p.view(T, k), k, topk_w=w.view(-1)), rows)


def test_the_stride_of_a_single_row_does_not_matter():
    """One row of a wider matrix, whose stride no second row has to keep to."""
    wide = torch.randn(3, 512 + 5, generator=torch.Generator().manual_seed(7)).to(DEV)
    x = wide[:1, :512]
    codes, sf = B.fp8_quantize(x)
    want = B.fp8_quantize(x.contiguous())
    assert torch.equal(codes, want[0]) and torch.equal(sf, want[1])
    for got, want in zip(B.fp8_swiglu_quantize(x), B.fp8_swiglu_quantize(x.contiguous())):
        assert torch.equal(got, want)
    _, _, w, sw, _ = _operands()
    a = torch.zeros((2, 512 + 7), dtype=torch.uint8, device=DEV)[:1, :512]
    a.copy_(codes)
    one = B.fp8_linear(codes, sf, w[0], sw[0])
    assert torch.equal(B.fp8_linear(a, sf, w[0], sw[0]), one)
    row = torch.zeros((2, 512 + 9), dtype=torch.uint8, device=DEV)[:1, :512]
    row.copy_(w[0, :1])
    assert torch.equal(B.fp8_linear(codes, sf, row, sw[0, :1]), B.fp8_linear(codes, sf, w[0, :1], sw[0, :1]))
    out = torch.zeros((2, 301), dtype=torch.bfloat16, device=DEV)[:1, :300]
    assert torch.equal(B.fp8_linear(codes, sf, w[0], sw[0], out=out), one)
    f2p = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    assert torch.equal(B.moe_sort_tokens(x, f2p, 2), x.expand(2, 512))
