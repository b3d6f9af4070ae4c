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


def test_weights_gradients_of_no_rows_and_of_no_columns(lib):
    """d_w asks for the dot products; their operand may be null where it is empty."""
    def unsort_back(rows, n, K, dw=P, w=P, d_rows=None):
        return lib.moe_unsort_tokens_backward(P, 0, 4, K, 16, P, 2, w, rows, 16, d_rows, n, 16, dw, None)

    def sort_back(x, K, d=P, n=8, dx=P, w=P, dw=P):
        return lib.moe_sort_tokens_backward(d, 0, n, K, 16, P, 4, 2, w, x, 16, dx, 16, dw, None)
    assert unsort_back(None, 0, 10) == LAUNCH and unsort_back(None, 8, 0) == LAUNCH
    assert unsort_back(None, 8, 10, d_rows=P) == INVALID
    assert unsort_back(None, 0, 10, w=None) == INVALID
    assert unsort_back(P, 8, 10, dw=None, d_rows=P) == INVALID        # an operand without its gradient
    assert sort_back(None, 0, dx=None) == LAUNCH and sort_back(P, 10, d=None, n=0) == LAUNCH
    assert sort_back(None, 10) == INVALID and sort_back(None, 10, d=None, n=0) == INVALID
    assert sort_back(None, 0, w=None) == INVALID


def test_rows_quantized_to_no_output_rows(lib):
    def q(codes, sf, out, f2p=P):
        return lib.fp8_quantize(P, 0, 4, 64, 64, f2p, 1, out, codes, sf, None)
    assert q(None, None, 0) == LAUNCH
    assert q(None, P, 4) == INVALID and q(P, None, 4) == INVALID
    assert q(None, None, 0, f2p=None) == -2                           # fewer output rows than rows
