"""The 8-bit operators' and the sorted-token operators' host checks: what they refuse
comes back as a status before anything is launched, and an empty call is fine (no GPU
needed)."""
import ctypes

import pytest

INVALID, UNSUPPORTED = -1, -2
vp, i64 = ctypes.c_void_p, ctypes.c_int64
P = vp(1 << 20)


@pytest.fixture(scope="module")
def lib():
    from nvfp4_block_scaled_05_gb300 import binding
    return binding.lib()


def test_quantizers(lib):
    def q(x=P, type=0, rows=4, K=64, ld=64, f2p=None, k=1, out=4, codes=P, sf=P):
        return lib.fp8_quantize(x, type, rows, K, ld, f2p, k, out, codes, sf, None)
    assert q(rows=0) == 0 and q(K=0) == 0
    assert q(type=3) == UNSUPPORTED and q(K=72) == UNSUPPORTED and q(rows=-1) == UNSUPPORTED
    assert q(f2p=P, k=17) == UNSUPPORTED and q(f2p=P, k=0) == UNSUPPORTED and q(out=3) == UNSUPPORTED
    assert q(x=None) == INVALID and q(codes=None) == INVALID and q(sf=None) == INVALID
    assert q(ld=48) == INVALID and q(ld=68) == INVALID and q(x=vp((1 << 20) + 8)) == INVALID
    assert q(codes=vp((1 << 20) + 8)) == INVALID and q(sf=vp((1 << 20) + 2)) == INVALID
    assert lib.fp8_swiglu_quantize(P, 0, 4, 64, 64, P, P, None) == INVALID       # rows of 2 * 64
    assert lib.fp8_swiglu_quantize(P, 0, 4, 40, 128, P, P, None) == UNSUPPORTED
    assert lib.fp8_quantize_weight(P, 0, 1, 16, 24, 32, P, P, None) == UNSUPPORTED
    assert lib.fp8_quantize_weight(P, 0, 65536, 16, 32, 32, P, P, None) == UNSUPPORTED
    assert lib.fp8_quantize_weight(P, 0, 1, 16, 32, 16, P, P, None) == INVALID
    assert lib.fp8_quantize_weight(None, 0, 1, 16, 32, 32, P, P, None) == INVALID
    assert lib.fp8_quantize_weight(None, 0, 0, 16, 32, 32, None, None, None) == 0


def test_products(lib):
    def g(a=P, M=4, lda=64, w=P, off=P, E=2, N=32, K=64, ldw=64, c=P, type=0, ldc=32, sa=P, sw=P):
        return lib.fp8_grouped_gemm(a, sa, M, lda, w, sw, off, E, N, K, ldw, c, type, ldc, None)
    assert g(M=0) == 0 and g(N=0) == 0 and g(M=0, off=None) == 0
    assert g(off=None) == INVALID
    assert g(E=0) == UNSUPPORTED and g(E=1025) == UNSUPPORTED and g(K=0) == UNSUPPORTED and g(M=-1) == UNSUPPORTED
    assert g(E=1024, N=1 << 21) == UNSUPPORTED and g(M=1 << 31) == UNSUPPORTED and g(type=5) == UNSUPPORTED
    assert g(M=(1 << 31) - 200, N=1 << 19, ldc=1 << 19) == UNSUPPORTED
    for name in ("a", "w", "c", "sa", "sw"):
        assert g(**{name: None}) == INVALID
    assert g(lda=72) == INVALID and g(ldw=48) == INVALID and g(ldc=31) == INVALID
    assert g(a=vp((1 << 20) + 8)) == INVALID and g(c=vp((1 << 20) + 1)) == INVALID
    assert lib.fp8_linear(P, P, 4, 60, P, P, 32, 64, 64, P, 0, 32, None) == INVALID
    assert lib.fp8_linear(None, None, 0, 64, None, None, 32, 64, 64, None, 0, 32, None) == 0


def test_sorted_tokens(lib):
    def sort(x=P, type=0, T=4, K=10, ldx=10, f2p=P, k=2, w=None, rows=P, n=8, ldr=10):
        return lib.moe_sort_tokens(x, type, T, K, ldx, f2p, k, w, rows, n, ldr, None)
    assert sort(T=0) == 0 and sort(K=0) == 0
    assert sort(type=-1) == UNSUPPORTED and sort(k=0) == UNSUPPORTED and sort(k=17) == UNSUPPORTED
    assert sort(T=1 << 30) == UNSUPPORTED and sort(n=-1) == UNSUPPORTED
    assert sort(x=None) == INVALID and sort(f2p=None) == INVALID and sort(rows=None) == INVALID
    assert sort(ldx=9) == INVALID and sort(ldr=9) == INVALID and sort(x=vp((1 << 20) + 1)) == INVALID

    def back(d=P, n=8, K=10, ldr=10, T=4, k=2, w=P, x=P, ldx=10, dx=P, lddx=10, dw=P):
        return lib.moe_sort_tokens_backward(d, 2, n, K, ldr, P, T, k, w, x, ldx, dx, lddx, dw, None)
    assert back(T=0) == 0
    assert back(dx=None) == INVALID and back(d=None) == INVALID and back(w=None) == INVALID
    assert back(dw=None) == INVALID and back(x=None) == INVALID and back(ldx=9) == INVALID
    assert back(dx=vp((1 << 20) + 2)) == INVALID
    assert lib.moe_unsort_tokens(P, 0, 8, 10, 9, P, 4, 2, None, P, 10, None) == INVALID
    assert lib.moe_unsort_tokens_backward(P, 0, 4, 10, 10, P, 2, None, P, 10, P, 8, 10, P, None) == INVALID


def test_expert_forward(lib):
    sz = ctypes.c_size_t
    T, K, I, E, k = 16, 256, 128, 8, 2
    need = lib.fp8_moe_forward_workspace_size(T, K, I, E, k)
    assert need > 0
    for bad in [(T, 200, I, E, k), (T, K, 100, E, k), (T, K, I, 1, 2), (T, K, I, 1025, k), (T, K, I, E, 17), (-1, K, I, E, k)]:
        assert lib.fp8_moe_forward_workspace_size(*bad) == 0

    def run(x=P, T=T, K=K, w2=P, y=P, ws=P, n=need):
        return lib.fp8_moe_forward(x, P, T, K, I, E, k, P, P, w2, P, y, ws, sz(n), None)
    assert run(T=0) == 0
    assert run(K=200) == UNSUPPORTED
    assert run(x=None) == INVALID and run(w2=None) == INVALID and run(y=vp((1 << 20) + 8)) == INVALID
    assert run(n=need - 1) == -3 and run(ws=None) == -3 and run(ws=vp((1 << 20) + 16)) == -3
