"""Group bounds of the 8-bit grouped product that are not in order, or not inside the
operands: a group starts at the largest bound so far, so that groups never share a
row, and the rows of no group are not written."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _random(seed, E, M):
    return np.random.default_rng(seed).integers(-M // 4, M + M // 4, E + 1).tolist()


@pytest.mark.parametrize("M,N,K,bounds", [
    (40, 130, 144, [0, 10, 2 ** 31 - 1, 5, 40]),
    (40, 130, 144, [-7, 3, 3, 2 ** 30, 60]),
    (40, 130, 144, [50, 60, 70, 80, 90]),
    (40, 130, 144, [0, 10, 40, 5, 40]),
    (40, 130, 1040, [0, 30, 10, 35, -2 ** 31, 38]),
    (60, 200, 144, [0, 20, 60, 0, 60, 0, 60, 0, 60, 0, 60]),        # would be three times the rows
    (3000, 600, 272, [0, 2000, 500, 2600, 100, 3000, 2900]),
    (3000, 600, 272, [0, 3000, 0, 3000, 0, 3000, 0, 3000, 0, 3000]),
    (100, 256, 128, _random(1, 70, 100)),
    (2000, 256, 128, _random(2, 33, 2000)),
    (2000, 300, 128, sorted(_random(3, 100, 2000))),
])
def test_every_group(M, N, K, bounds):
    E = len(bounds) - 1
    g = torch.Generator().manual_seed(E)
    a, sa = B.fp8_quantize(torch.randn(M, K, generator=g).to(DEV))
    w, sw = B.fp8_quantize_weight(torch.randn(E, N, K, generator=g).to(DEV))
    off = torch.tensor(bounds, dtype=torch.int32, device=DEV)
    guard = torch.full((M + 400, N), 3.0, device=DEV)
    got = B.fp8_grouped_gemm(a, sa, w, sw, off, out=guard[200:200 + M])
    assert B.nvfp4moe_last_device_status() == 0
    assert (guard[:200] == 3).all() and (guard[200 + M:] == 3).all()
    at = np.maximum.accumulate(np.clip(bounds, 0, M))
    # f32 sums: at most K + KB additions a block's order apart, each a step of f32 of the summed magnitudes
    va = (a.view(torch.float8_e4m3fn).double() * sa.double().repeat_interleave(128, 1)[:, :K])
    for e in range(E):
        lo, hi = int(at[e]), int(at[e + 1])
        vw = w[e].view(torch.float8_e4m3fn).double() * \
            sw[e].double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
        want, size = va[lo:hi] @ vw.t(), va[lo:hi].abs() @ vw.abs().t()
        lim = (K + -(-K // 128) + 3) * 2.0 ** -23 * size
        assert ((got[lo:hi].double() - want).abs() <= lim).all(), e
    assert (got[:int(at[0])] == 3).all() and (got[int(at[-1]):] == 3).all()
