"""A call that writes into a tensor of the caller's counts as an in-place operation on it: what
autograd saved of its old contents is not used unnoticed."""
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
EPS = 1e-5
T, K, I, E, k = 8, 256, 128, 4, 2


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV)


@pytest.fixture(scope="module")
def operands():
    o = {"x": _randn(1, T, K).bfloat16(), "res": _randn(2, T, K).bfloat16(), "gamma": 1 + 0.1 * _randn(3, K),
         "logits": _randn(4, T, E), "w": B.prepare_fp8_moe_weights(_randn(5, E, 2 * I, K) / 16, _randn(6, E, K, I) / 12),
         "w4": B.prepare_moe_weights((_randn(5, E, 2 * I, K) / 16).bfloat16(), (_randn(6, E, K, I) / 12).bfloat16()),
         "gs": torch.ones(1, device=DEV)}
    o["a"], o["sa"] = B.fp8_quantize(o["x"])
    o["dense"], o["sd"] = B.fp8_quantize_weight(_randn(7, K, K) / 16)
    o["ids"], o["topk_w"] = B.moe_route_topk(o["logits"], k)
    o["offsets"], _, o["f2p"] = B.moe_permute(o["ids"], E)
    o["rows"] = B.moe_sort_tokens(o["x"], o["f2p"], k)
    o["ra"], o["rs"] = B.fp8_quantize(o["rows"])
    o["x4"], o["sx4"], o["gs4"] = B.nvfp4_quantize(o["x"])
    o["d4"], o["sd4"], o["gd4"] = B.nvfp4_quantize((_randn(7, K, K) / 16).bfloat16())
    return o


# a call with `to` (T, K) of BF16 as its result
INTO = {
    "rms_norm y": lambda o, to: B.rms_norm(o["x"], o["gamma"], EPS, y=to),
    "rms_norm h": lambda o, to: B.rms_norm(o["x"], o["gamma"], EPS, residual=to, h=to),
    "rms_norm_backward dx": lambda o, to: B.rms_norm_backward(o["x"], o["res"], o["gamma"], EPS, dx=to),
    "fp8_rms_norm_quantize y": lambda o, to: B.fp8_rms_norm_quantize(o["x"], o["gamma"], EPS, y=to),
    "fp8_rms_norm_quantize h": lambda o, to: B.fp8_rms_norm_quantize(o["x"], o["gamma"], EPS, residual=to, h=to),
    "fp8_linear": lambda o, to: B.fp8_linear(o["a"], o["sa"], o["dense"], o["sd"], out=to),
    "fp8_linear_epilogue": lambda o, to: B.fp8_linear_epilogue(o["a"], o["sa"], o["dense"], o["sd"], residual=to, out=to),
    "fp8_moe_few_tokens": lambda o, to: B.fp8_moe_few_tokens(o["x"], o["logits"], o["w"], k, residual=to, y=to),
    "fp8_moe_forward": lambda o, to: B.fp8_moe_forward(o["x"], o["logits"], o["w"], k, y=to),
    "moe_forward": lambda o, to: B.moe_forward(o["x"], o["logits"], o["w4"], k, o["gs"], y=to),
    "moe_forward_static": lambda o, to: B.moe_forward_static(o["x"], o["logits"], o["w4"], k, o["gs"], o["gs"], y=to),
    "moe_unsort_tokens": lambda o, to: B.moe_unsort_tokens(o["rows"], o["f2p"], k, topk_w=o["topk_w"], y=to),
    "moe_sort_tokens_backward": lambda o, to: B.moe_sort_tokens_backward(o["rows"], o["f2p"], k, dx=to),
    "moe_combine": lambda o, to: B.moe_combine(o["rows"], o["topk_w"], o["f2p"].view(-1), y=to),
    "nvfp4_linear": lambda o, to: B.nvfp4_linear(torch.zeros(128, K // 2, dtype=torch.uint8, device=DEV),
                                                 torch.zeros(B.nvfp4_sf_bytes(128, K, B.NVFP4_SF_TILED_ROWS),
                                                             dtype=torch.uint8, device=DEV),
                                                 o["gs4"], T, o["d4"], o["sd4"], o["gd4"], out=to),
    "moe_forward_stages": lambda o, to: B.moe_forward_stages(o["x"], o["logits"], o["w4"], k, o["gs"], _ws4(), to),
    "moe_forward_static_stages": lambda o, to: B.moe_forward_static_stages(o["x"], o["logits"], o["w4"], k, o["gs"],
                                                                           o["gs"], _ws4(), to),
}


def _ws4():
    return torch.empty(B.moe_forward_workspace_size(T, K, I, E, k), dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("name", INTO)
def test_a_saved_tensor_is_overwritten(operands, name):
    """A norm saved h for its backward pass; a call puts its result there."""
    x = operands["x"].clone().requires_grad_()
    y, h = B.rms_norm(x, operands["gamma"], EPS, residual=operands["res"])
    with torch.no_grad():
        INTO[name](operands, h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


# further tensors of the caller's: (shape, type), call
def _codes(rows=T, cols=K):
    return torch.empty(rows, cols, dtype=torch.uint8, device=DEV)


OTHERS = {
    "moe_sort_tokens rows": lambda o: (torch.empty(T * k, K, dtype=BF16, device=DEV),
                                       lambda t: B.moe_sort_tokens(o["x"], o["f2p"], k, rows=t)),
    "moe_unsort_tokens_backward d_rows": lambda o: (torch.empty(T * k, K, dtype=BF16, device=DEV),
                                                    lambda t: B.moe_unsort_tokens_backward(o["x"], o["f2p"], k, d_rows=t)),
    "fp8_quantize codes": lambda o: (_codes(), lambda t: B.fp8_quantize(o["x"], codes=t)),
    "fp8_quantize sf": lambda o: (torch.empty(T, K // 128, device=DEV), lambda t: B.fp8_quantize(o["x"], sf=t)),
    "fp8_swiglu_quantize codes": lambda o: (_codes(T, K // 2), lambda t: B.fp8_swiglu_quantize(o["x"], codes=t)),
    "fp8_swiglu_quantize sf": lambda o: (torch.empty(T, K // 256, device=DEV), lambda t: B.fp8_swiglu_quantize(o["x"], sf=t)),
    "fp8_rms_norm_quantize codes": lambda o: (_codes(), lambda t: B.fp8_rms_norm_quantize(o["x"], o["gamma"], EPS, codes=t)),
    "fp8_rms_norm_quantize sf": lambda o: (torch.empty(T, K // 128, device=DEV),
                                           lambda t: B.fp8_rms_norm_quantize(o["x"], o["gamma"], EPS, sf=t)),
    "fp8_grouped_gemm out": lambda o: (torch.empty(T * k, 2 * I, dtype=BF16, device=DEV),
                                       lambda t: B.fp8_grouped_gemm(o["ra"], o["rs"], o["w"]["w1_codes"], o["w"]["w1_sf"],
                                                                    o["offsets"], out=t)),
    "fp8_moe_few_tokens ws": lambda o: (
        torch.empty(B.fp8_moe_few_tokens_workspace_size(T, K, I, E, k), dtype=torch.uint8, device=DEV),
        lambda t: B.fp8_moe_few_tokens(o["x"], o["logits"], o["w"], k, ws=t)),
    "fp8_moe_forward ws": lambda o: (
        torch.empty(B.fp8_moe_forward_workspace_size(T, K, I, E, k), dtype=torch.uint8, device=DEV),
        lambda t: B.fp8_moe_forward(o["x"], o["logits"], o["w"], k, ws=t)),
    "moe_forward ws": lambda o: (_ws4(), lambda t: B.moe_forward(o["x"], o["logits"], o["w4"], k, o["gs"], ws=t)),
    "moe_forward_static ws": lambda o: (
        _ws4(), lambda t: B.moe_forward_static(o["x"], o["logits"], o["w4"], k, o["gs"], o["gs"], ws=t)),
    "nvfp4_quantize codes": lambda o: (_codes(T, K // 2), lambda t: B.nvfp4_quantize(o["x"], codes=t)),
    "nvfp4_quantize sf": lambda o: (torch.empty_like(o["sx4"]), lambda t: B.nvfp4_quantize(o["x"], sf=t)),
    "nvfp4_quantize gs_out": lambda o: (torch.empty(1, device=DEV), lambda t: B.nvfp4_quantize(o["x"], gs_out=t)),
    "nvfp4_rmsnorm_rope_quantize y_out": lambda o: (
        torch.empty(T, K, device=DEV),
        lambda t: B.nvfp4_rmsnorm_rope_quantize(o["x"], o["gamma"], EPS, 0, None, None, None, o["gs"], y_out=t)),
    "nvfp4_sf_from_tiled out": lambda o: (_codes(T, K // 16), lambda t: B.nvfp4_sf_from_tiled(o["sx4"], 1, T, K, out=t)),
    "nvfp4_sf_to_tiled out": lambda o: (torch.empty_like(o["sx4"]),
                                        lambda t: B.nvfp4_sf_to_tiled(_codes(T, K // 16).zero_(), T, K, out=t)),
}


@pytest.mark.parametrize("name", OTHERS)
def test_a_result_counts(operands, name):
    t, call = OTHERS[name](operands)
    before = t._version
    call(t)
    assert t._version > before
    with torch.inference_mode():      # whose tensors have no count
        t, call = OTHERS[name](operands)
        call(t)
    torch.cuda.synchronize()


def test_a_refused_call_does_not_count(operands):
    o = operands
    to = torch.empty(T, K, dtype=BF16, device=DEV)
    for call in (lambda: B.rms_norm(o["x"], o["gamma"], -1.0, y=to), lambda: B.rms_norm(o["x"][:4], o["gamma"], EPS, y=to),
                 lambda: B.fp8_moe_few_tokens(o["x"], o["logits"], o["w"], 17, y=to),
                 lambda: B.fp8_linear_epilogue(o["a"], o["sa"], o["dense"], o["sd"], activation="tanh", out=to)):
        with pytest.raises(B.NVFP4Error):
            call()
    assert to._version == 0
    B.rms_norm_backward(o["x"], o["res"], o["gamma"], EPS)
    assert all(o[name]._version == 0 for name in ("x", "logits", "topk_w"))


def test_recorded_calls_in_place(operands):
    """A recorded call's own result in the caller's tensor can be differentiated, and an earlier
    norm that saved the tensor cannot any more."""
    o = operands
    x = o["x"].float().requires_grad_()
    stream = o["res"].float()
    y1, h1 = B.rms_norm(x, o["gamma"], EPS, residual=stream, h=stream)
    y1.sum().backward()                       # its own h is intact
    assert torch.isfinite(x.grad).all()
    stream = o["res"].float()
    y1, h1 = B.rms_norm(x, o["gamma"], EPS, residual=stream)
    with torch.no_grad():
        y2, h2 = B.rms_norm(o["x"].float(), o["gamma"], EPS, residual=h1, h=h1)
    assert h2.data_ptr() == h1.data_ptr()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y1.sum().backward()
