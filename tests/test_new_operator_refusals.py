"""What the norms, the product with an epilogue and the expert layer for a few tokens refuse on the
host, before anything is launched (no GPU needed)."""
import ctypes

import pytest

from nvfp4_block_scaled_05_gb300 import binding as B

P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 2)
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def test_constants_match_the_header():
    import os
    import re
    from conftest import ROOT
    with open(os.path.join(ROOT, "include", "nvfp4moe.h")) as f:
        defs = dict(re.findall(r"#define (NVFP4\w+) (\d+)", f.read()))
    assert int(defs["NVFP4MOE_FEW_TOKENS_MAX"]) == B.FEW_TOKENS_MAX


def _norm(lib, quantize=True, type=0, rows=4, K=64, ldx=64, r=P, ldr=64, gamma=P, eps=1e-5, h=P, ldh=64, y=P, ldy=64,
          codes=P, sf=P, x=P):
    if quantize:
        return lib.fp8_rms_norm_quantize(x, type, rows, K, ldx, r, ldr, gamma, eps, h, ldh, y, ldy, codes, sf, None)
    return lib.rms_norm(x, type, rows, K, ldx, r, ldr, gamma, eps, h, ldh, y, ldy, None)


@pytest.mark.parametrize("quantize", [False, True])
def test_norm(lib, quantize):
    for kw, status in (({"type": 3}, UNSUPPORTED), ({"rows": -1}, UNSUPPORTED), ({"K": -1}, UNSUPPORTED),
                       ({"K": 16400, "ldx": 16400}, UNSUPPORTED), ({"eps": -1.0}, UNSUPPORTED),
                       ({"eps": float("nan")}, UNSUPPORTED), ({"x": None}, INVALID), ({"gamma": None}, INVALID),
                       ({"ldx": 63}, INVALID), ({"ldr": 63}, INVALID), ({"h": None}, INVALID), ({"ldh": 63}, INVALID),
                       ({"ldy": 63}, INVALID), ({"x": ODD, "type": 2}, INVALID), ({"rows": 0}, OK), ({"K": 0}, OK)):
        assert _norm(lib, quantize, **kw) == status, kw
    if quantize:
        for kw, status in (({"K": 40}, UNSUPPORTED), ({"codes": None}, INVALID), ({"sf": None}, INVALID),
                           ({"x": ODD}, INVALID), ({"ldx": 65}, INVALID), ({"gamma": ctypes.c_void_p((1 << 20) + 4)}, INVALID)):
            assert _norm(lib, **kw) == status, kw
    else:
        assert _norm(lib, False, y=None) == INVALID


def test_norm_backward(lib):
    size = lib.rms_norm_backward_workspace_size
    assert size(-1, 64) == size(4, 16385) == size(0, 64) == 0
    assert size(1, 7168) == 7168 * 4 and size(10 ** 6, 7168) == 1216 * 7168 * 4
    need = size(4, 64)
    good = [P, 0, 4, 64, 64, P, 64, P, 1e-5, P, 64, P, 64, P, P, need, None]
    for at, value, status in ((1, 5, UNSUPPORTED), (2, -1, UNSUPPORTED), (8, -1.0, UNSUPPORTED), (0, None, INVALID),
                              (4, 60, INVALID), (5, None, INVALID), (7, None, INVALID), (10, 60, INVALID),
                              (11, None, INVALID), (12, 60, INVALID), (13, None, INVALID), (14, None, WORKSPACE),
                              (15, need - 1, WORKSPACE), (14, ODD, WORKSPACE), (3, 0, OK)):
        args = list(good)
        args[at] = value
        assert lib.rms_norm_backward(*args) == status, (at, value)


def test_linear_epilogue(lib):
    good = [P, P, 4, 128, P, P, 64, 128, 128, P, 4, P, 64, P, 0, 64, None]
    for at, value, status in ((0, None, INVALID), (3, 100, INVALID), (7, 0, UNSUPPORTED), (14, 3, UNSUPPORTED),
                              (9, ctypes.c_void_p((1 << 20) + 4), INVALID), (10, 5, UNSUPPORTED), (10, -1, UNSUPPORTED),
                              (12, 63, INVALID), (11, ctypes.c_void_p((1 << 20) + 1), INVALID), (15, 63, INVALID),
                              (2, 0, OK)):
        args = list(good)
        args[at] = value
        assert lib.fp8_linear_epilogue(*args) == status, (at, value)


def test_few_tokens(lib):
    size = lib.fp8_moe_few_tokens_workspace_size
    for args in ((33, 128, 64, 8, 2), (1, 100, 64, 8, 2), (1, 128, 60, 8, 2), (1, 128, 64, 8, 9), (1, 128, 64, 8, 0),
                 (1, 128, 64, 1025, 2), (1, 128, 64, 32, 17), (-1, 128, 64, 8, 2), (1, 1 << 20, 64, 8, 2)):
        assert size(*args) == 0, args
    need = size(4, 128, 64, 8, 2)
    assert need >= 4 * 2 * (64 + 128) * 4
    good = [P, 0, 4, 128, 128, P, 64, 8, 2, P, P, P, P, P, 128, P, 128, P, need, None]
    for at, value, status in ((0, None, INVALID), (0, ODD, INVALID), (1, 3, UNSUPPORTED), (2, 33, UNSUPPORTED),
                              (3, 120, UNSUPPORTED), (4, 127, INVALID), (4, 132, INVALID), (5, None, INVALID),
                              (6, 40, UNSUPPORTED), (7, 1, UNSUPPORTED), (8, 17, UNSUPPORTED), (9, None, INVALID),
                              (9, ODD, INVALID), (10, None, INVALID), (11, None, INVALID), (12, None, INVALID),
                              (13, ctypes.c_void_p((1 << 20) + 1), INVALID), (14, 100, INVALID), (15, None, INVALID),
                              (16, 100, INVALID), (17, None, WORKSPACE), (17, ODD, WORKSPACE), (18, need - 1, WORKSPACE),
                              (2, 0, OK)):
        args = list(good)
        args[at] = value
        assert lib.fp8_moe_few_tokens(*args) == status, (at, value)


@pytest.mark.parametrize("quantize", [False, True])
def test_norm_h_without_a_residual(lib, quantize):
    """h is the sum with the residual: given alone it would be left unwritten."""
    assert _norm(lib, quantize, r=None, ldr=0) == INVALID
    assert _norm(lib, quantize, r=None, ldr=0, type=1) == INVALID
    assert _norm(lib, quantize, r=None, rows=0) == OK
