"""The 8-bit expert forward: its stages' own results bit for bit, the layer against
64 bits, graph capture, and the example that trains through the token sort."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT
from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _layer(T, K, I, E, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g).bfloat16().to(DEV)
    logits = torch.randn(T, E, generator=g).to(DEV)
    w1 = (torch.randn(E, 2 * I, K, generator=g) * K ** -0.5).bfloat16().to(DEV)
    w2 = (torch.randn(E, K, I, generator=g) * I ** -0.5).bfloat16().to(DEV)
    return x, logits, w1, w2


def _values(codes, sf, each):
    v = codes.view(torch.float8_e4m3fn).double()
    s = sf.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]
    if each > 1:
        s = s.repeat_interleave(each, -2)[..., :codes.shape[-2], :]
    return v * s


@pytest.mark.parametrize("T,K,I,E,k", [(1, 128, 64, 4, 1), (5, 272, 144, 8, 3), (64, 512, 256, 8, 2),
                                       (300, 1040, 400, 33, 6), (700, 2048, 512, 16, 8)])
def test_forward(T, K, I, E, k):
    x, logits, w1, w2 = _layer(T, K, I, E, T + E)
    weights = B.prepare_fp8_moe_weights(w1, w2)
    y = B.fp8_moe_forward(x, logits, weights, k)
    # the stages one by one give the same bits
    ids, w = B.moe_route_topk(logits, k)
    off, p2f, f2p = B.moe_permute(ids, E)
    a, sa = B.fp8_quantize(x, flat_to_perm=f2p, k=k)
    gu = B.fp8_grouped_gemm(a, sa, weights["w1_codes"], weights["w1_sf"], off)
    h, sh = B.fp8_swiglu_quantize(gu)
    out = B.fp8_grouped_gemm(h, sh, weights["w2_codes"], weights["w2_sf"], off)
    assert torch.equal(y, B.moe_unsort_tokens(out, f2p, k, topk_w=w))
    assert B.nvfp4moe_last_device_status() == 0
    # and lie near the layer of the same quantized operands in 64 bits: each
    # stage rounds to BF16 (2^-8) and h to E4M3 (2^-4, which an operand a
    # rounding away can turn the other way: another 2^-4), all relative to a
    # value whose errors add up in quadrature over the sums
    want = torch.zeros(T * k, K, dtype=torch.float64, device=DEV)
    bounds = off.tolist()
    va = _values(a, sa, 1)
    v1, v2 = _values(weights["w1_codes"], weights["w1_sf"], 128), _values(weights["w2_codes"], weights["w2_sf"], 128)
    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        gate, up = (va[lo:hi] @ v1[e].t()).chunk(2, 1)
        want[lo:hi] = (gate * torch.sigmoid(gate) * up) @ v2[e].t()
    ref = (want[f2p.long()].view(T, k, K) * w.double()[..., None]).sum(1)
    far = float((y.double() - ref).norm() / ref.norm())
    assert far <= 2 ** -4 + 2 ** -4 + 4 * 2 ** -8, far


def test_forward_in_a_graph_and_with_the_callers_memory():
    T, K, I, E, k = 40, 512, 128, 8, 2
    x, logits, w1, w2 = _layer(T, K, I, E, 3)
    weights = B.prepare_fp8_moe_weights(w1, w2)
    want = B.fp8_moe_forward(x, logits, weights, k)
    n = B.fp8_moe_forward_workspace_size(T, K, I, E, k)
    guard = torch.full((n + 512,), 0x5A, dtype=torch.uint8, device=DEV)
    ws, y = guard[256:256 + n], torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.fp8_moe_forward(x, logits, weights, k, ws=ws, y=y)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)
    assert (guard[:256] == 0x5A).all() and (guard[256 + n:] == 0x5A).all()
    with pytest.raises(B.NVFP4Error):
        B.fp8_moe_forward(x, logits, weights, k, ws=ws[:n - 1])
    with pytest.raises(B.NVFP4Error):
        B.fp8_moe_forward(x[:, :256].contiguous(), logits, weights, k)
    assert B.fp8_moe_forward(x[:0], logits[:0], weights, k).shape == (0, K)


def test_example():
    spec = importlib.util.spec_from_file_location("fp8_experts", os.path.join(ROOT, "examples", "fp8_experts.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    far, far_x, far_w = example.main()
    # activations, weights and h in E4M3, each off by at most 2^-4, rms 2^-4 / sqrt(3):
    # three of them in quadrature 2^-4, the products' one for gate and up twice
    assert far <= 2 * 2 ** -4
    # BF16 rows, products and gradients: a handful of roundings of 2^-8
    assert far_x <= 8 * 2 ** -8 and far_w <= 8 * 2 ** -8
