"""An expert layer in 8-bit block-scaled form, and a gradient step through the
token sort of a BF16 one.

    python examples/fp8_experts.py

Part 1 quantizes the experts' weights once (fp8_quantize_weight), runs the
forward (fp8_moe_forward: route, quantize into expert order, grouped products,
SwiGLU, weighted sum) and compares it with the same layer in f32.
Part 2 trains one step: tokens to expert order (moe_sort_tokens), any expert
function of the rows, the weighted sum back (moe_unsort_tokens), and the
gradients of both, down to the tokens and the routing weights.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from nvfp4_block_scaled_05_gb300 import binding as B  # noqa: E402


def experts(rows, offsets, w1, w2):
    """silu(gate) * up and the down projection, expert by expert."""
    bounds = offsets.tolist()
    out = []
    for e in range(w1.shape[0]):
        gate, up = (rows[bounds[e]:bounds[e + 1]] @ w1[e].t()).chunk(2, 1)
        out.append((torch.nn.functional.silu(gate) * up) @ w2[e].t())
    return torch.cat(out)


def main():
    dev = torch.device("cuda")
    T, K, I, E, k = 256, 1024, 512, 16, 4
    g = torch.Generator(device=dev).manual_seed(0)
    x = torch.randn(T, K, device=dev, generator=g).bfloat16()
    logits = torch.randn(T, E, device=dev, generator=g)
    w1 = (torch.randn(E, 2 * I, K, device=dev, generator=g) * K ** -0.5).bfloat16()
    w2 = (torch.randn(E, K, I, device=dev, generator=g) * I ** -0.5).bfloat16()

    # 1. the 8-bit forward
    weights = B.prepare_fp8_moe_weights(w1, w2)
    y = B.fp8_moe_forward(x, logits, weights, k)
    ids, w = B.moe_route_topk(logits, k)
    offsets, perm_to_flat, flat_to_perm = B.moe_permute(ids, E)
    rows = experts(x.float()[perm_to_flat.long() // k], offsets, w1.float(), w2.float())
    want = (rows[flat_to_perm.long()].view(T, k, K) * w[..., None]).sum(1)
    far = float((y.float() - want).norm() / want.norm())
    print("8-bit forward: %.4f from f32 (2-norm)" % far)

    # 2. a gradient step through the sort
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    w1g, w2g = w1.clone().requires_grad_(), w2.clone().requires_grad_()
    target = torch.randn(T, K, device=dev, generator=g).bfloat16()
    rows = experts(B.moe_sort_tokens(xg, flat_to_perm, k), offsets, w1g, w2g)
    y = B.moe_unsort_tokens(rows, flat_to_perm, k, topk_w=wg)
    loss = (y.float() - target.float()).square().mean()
    loss.backward()
    xr, wr = x.float().requires_grad_(), w.clone().requires_grad_()
    rows = experts(xr[perm_to_flat.long() // k], offsets, w1.float(), w2.float())
    ref = (rows[flat_to_perm.long()].view(T, k, K) * wr[..., None]).sum(1)
    (ref - target.float()).square().mean().backward()
    far_x = float((xg.grad.float() - xr.grad).norm() / xr.grad.norm())
    far_w = float((wg.grad - wr.grad).norm() / wr.grad.norm())
    print("loss %.4f; gradients from f32 (2-norm): tokens %.4f, routing weights %.4f" % (loss.item(), far_x, far_w))
    assert B.nvfp4moe_last_device_status() == 0
    return far, far_x, far_w


if __name__ == "__main__":
    main()
