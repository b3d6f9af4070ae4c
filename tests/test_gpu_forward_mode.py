"""Forward-mode derivatives, which no call has: the calls that are differentiable, or that refuse to
lose a gradient, refuse an operand with a tangent and do not take it as a constant."""
import pytest
import torch
import torch.autograd.forward_ad as fwAD

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5
T, K, I, E, k = 4, 256, 128, 4, 2


def _randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DEV)


def _operands():
    o = {"x": _randn(1, T, K), "r": _randn(2, T, K), "gamma": _randn(3, K), "logits": _randn(4, T, E), "out": _randn(5, T, K),
         "rows": _randn(6, T * k, K)}
    o["ids"], o["w"] = B.moe_route_topk(o["logits"], k)
    return o


def _calls():
    a, sa = B.fp8_quantize(_randn(7, T, K))
    d, sd = B.fp8_quantize_weight(_randn(8, K, K))
    experts = B.prepare_fp8_moe_weights(_randn(9, E, 2 * I, K), _randn(10, E, K, I))
    _, _, f2p = B.moe_permute(_operands()["ids"], E)
    return {
        "rms_norm": (("x", "r", "gamma", "out"), lambda o: B.rms_norm(o["x"], o["gamma"], EPS, residual=o["r"], y=o["out"])),
        "rms_norm h": (("out",), lambda o: B.rms_norm(o["x"], o["gamma"], EPS, residual=o["r"], h=o["out"])),
        "rms_norm_backward": (("x", "r", "gamma", "rows4", "out"),
                              lambda o: B.rms_norm_backward(o["x"], o["r"], o["gamma"], EPS, dh=o["rows4"], dx=o["out"])),
        "fp8_rms_norm_quantize": (("x", "r", "gamma", "out"), lambda o: B.fp8_rms_norm_quantize(
            o["x"], o["gamma"], EPS, residual=o["r"], y=o["out"])),
        "fp8_linear_epilogue": (("bias", "r", "out"), lambda o: B.fp8_linear_epilogue(
            a, sa, d, sd, bias=o["bias"], residual=o["r"], out=o["out"])),
        "fp8_moe_few_tokens": (("x", "logits", "r", "out"), lambda o: B.fp8_moe_few_tokens(
            o["x"], o["logits"], experts, k, residual=o["r"], y=o["out"])),
        "moe_sort_tokens": (("x", "w", "rows"), lambda o: B.moe_sort_tokens(o["x"], f2p, k, topk_w=o["w"], rows=o["rows"])),
        "moe_unsort_tokens": (("rows", "w", "out"), lambda o: B.moe_unsort_tokens(o["rows"], f2p, k, topk_w=o["w"], y=o["out"])),
        "moe_sort_tokens_backward": (("rows", "w", "x", "out"), lambda o: B.moe_sort_tokens_backward(
            o["rows"], f2p, k, topk_w=o["w"], x=o["x"], dx=o["out"])),
        "moe_unsort_tokens_backward": (("x", "w", "rows", "rows2"), lambda o: B.moe_unsort_tokens_backward(
            o["x"], f2p, k, topk_w=o["w"], rows=o["rows"], d_rows=o["rows2"])),
    }


NAMES = ["rms_norm", "rms_norm h", "rms_norm_backward", "fp8_rms_norm_quantize", "fp8_linear_epilogue", "fp8_moe_few_tokens",
         "moe_sort_tokens", "moe_unsort_tokens", "moe_sort_tokens_backward", "moe_unsort_tokens_backward"]


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_tangents_are_refused(name, grad):
    operands, call = _calls()[name]
    o = _operands()
    o.update(rows4=_randn(11, T, K), rows2=_randn(12, T * k, K), bias=_randn(13, K))
    call(o)
    with torch.set_grad_enabled(grad), fwAD.dual_level():
        for dual in operands:
            p = dict(o)
            p[dual] = fwAD.make_dual(o[dual], torch.ones_like(o[dual]))
            with pytest.raises(B.NVFP4Error, match="forward"):
                call(p)
    call(o)                      # out of the level there is none


def test_tangents_with_reverse_mode():
    """Also where the call would be recorded."""
    o = _operands()
    with fwAD.dual_level():
        x = fwAD.make_dual(o["x"].requires_grad_(), torch.ones_like(o["x"]))
        with pytest.raises(B.NVFP4Error, match="forward"):
            B.rms_norm(x, o["gamma"], EPS)
        with pytest.raises(B.NVFP4Error, match="forward"):
            B.fp8_rms_norm_quantize(x, o["gamma"], EPS, residual=o["r"])
