"""Calls of a rank that holds no rows, or whose rows have no columns: what their host
checks refuse and let through (no GPU needed: a call that is let through ends at the
missing device)."""
import ctypes

import pytest

INVALID, LAUNCH = -1, -4
vp = ctypes.c_void_p
P = vp(1 << 20)


@pytest.fixture(scope="module")
def lib():
    import torch
    from nvfp4_block_scaled_05_gb300 import binding
    if torch.cuda.is_available():
        pytest.skip("the pointers are not the device's")
    return binding.lib()


def test_the_token_rows_are_read_whatever_the_slots_hold(lib):
    def sort(x, K, n):
        return lib.moe_sort_tokens(x, 0, 4, K, 16, P, 2, None, None, n, 16, None)
    assert sort(None, 10, 0) == INVALID
    assert lib.moe_unsort_tokens_backward(None, 0, 4, 10, 16, P, 2, P, P, 16, None, 0, 16, P, None) == INVALID
    assert sort(P, 10, 0) == LAUNCH
    assert sort(None, 0, 8) == 0 and sort(None, 0, 0) == 0
