"""Sizes that one of the 8-bit expert forward's stages refuses have no workspace size, and
the forward refuses them before its first stage runs (no GPU needed)."""
import ctypes

import pytest

vp = ctypes.c_void_p
P = vp(1 << 20)
UNSUPPORTED = -2


@pytest.mark.parametrize("T,K,I,E,k", [
    (16, 16, 1 << 20, 1024, 1),            # 2^31 rows of gate and up weights
    (16, 1 << 21, 16, 1024, 1),            # 2^31 rows of the down weights
    ((1 << 27) - 200, (1 << 24) - 16, 16, 1, 1),      # 2^36 tiles of the down product
    ((1 << 30) - 200, 16, 4096 * 8, 16, 2),           # 2^24 x 2^8 tiles of the first, blocks of h
])
def test_refused(T, K, I, E, k):
    from nvfp4_block_scaled_05_gb300 import binding
    lib = binding.lib()
    assert lib.fp8_moe_forward_workspace_size(T, K, I, E, k) == 0
    got = lib.fp8_moe_forward(P, P, T, K, I, E, k, P, P, P, P, P, P, ctypes.c_size_t((1 << 62)), None)
    assert got == UNSUPPORTED


@pytest.mark.parametrize("T,K,I,E,k", [(8192, 7168, 2048, 256, 8), (1, 16, 16, 1, 1), (1 << 20, 7168, 2048, 256, 8),
                                       (65536, 16384, 16384, 1024, 16)])
def test_taken(T, K, I, E, k):
    from nvfp4_block_scaled_05_gb300 import binding
    assert binding.lib().fp8_moe_forward_workspace_size(T, K, I, E, k) > T * k * (K + 2 * I)
