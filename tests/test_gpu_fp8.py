"""The 8-bit block-scaled operators: codes and scales bit for bit against the rule,
products against 64 bits (exactly where every partial sum is representable), over
ragged sizes, empty groups, strides, bad offsets, and the failure path."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
U32 = 2.0 ** -24
TINY = 2.0 ** -100


def _blocks(n):
    return -(-n // 128)


def _rand(shape, seed, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def _pad(x, dim):
    n = -x.shape[dim] % 128
    shape = list(x.shape)
    shape[dim] = n
    return torch.cat([x, x.new_zeros(shape)], dim) if n else x


def _rule(x, dims):
    """Codes (as values) and scales of f32 blocks that span `dims`, one f32 operation a step."""
    x = x.numpy()
    bits = (x.view(np.uint32) & np.uint32(0x7FFFFFFF)).max(axis=dims, keepdims=True)
    amax = bits.view(np.float32)
    with np.errstate(all="ignore"):
        live = ~(amax < np.float32(TINY))
        inv = np.where(live, np.float32(448) / amax, np.float32(0)).astype(np.float32)
        sf = np.where(live, amax / np.float32(448), np.float32(0)).astype(np.float32)
        q = (x * inv).astype(np.float32)
    return torch.from_numpy(np.clip(q, -448, 448)).to(F8), torch.from_numpy(sf)


def _rule_rows(x):
    M, K = x.shape
    codes, sf = _rule(_pad(x.float(), 1).view(M, -1, 128).contiguous(), (2,))
    return codes.reshape(M, -1)[:, :K], sf[..., 0]


def _rule_weight(w):
    E, N, K = w.shape
    b = _pad(_pad(w.float(), 2), 1).view(E, _blocks(N), 128, _blocks(K), 128).contiguous()
    codes, sf = _rule(b, (2, 4))
    return codes.reshape(E, _blocks(N) * 128, -1)[:, :N, :K], sf[:, :, 0, :, 0]


def _same(codes, want):
    """Equal code bytes, NaN codes of either sign being the same."""
    a, b = codes.cpu(), want.contiguous().view(torch.uint8)
    nan = (b & 0x7F) == 0x7F
    return torch.equal(torch.where(nan, b & 0x7F, b), torch.where((a & 0x7F) == 0x7F, a & 0x7F, a))


def _same_scales(a, b):
    return torch.equal(a.cpu().nan_to_num(nan=-1.0, posinf=-2.0), b.nan_to_num(nan=-1.0, posinf=-2.0))


# ------------------------------------------------------------------ quantizers

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (7, 512), (5, 528), (33, 2000), (130, 7168)])
def test_rows_match_the_rule_bit_for_bit(M, K, dtype):
    x = _rand((M, K), M + K).to(dtype)
    codes, sf = B.fp8_quantize(x.to(DEV))
    want, want_sf = _rule_rows(x)
    assert codes.dtype == torch.uint8 and codes.shape == (M, K) and sf.shape == (M, _blocks(K))
    assert _same(codes, want) and _same_scales(sf, want_sf)


def test_special_blocks():
    """Zeros, signed zeros, blocks at and below 2^-100, the type's largest, infinities and NaN."""
    x = _rand((12, 384), 5)
    x[0] = 0.0
    x[1, :128] = -0.0
    x[2] *= TINY / 8
    x[3, 128:256] = 0.0
    x[3, 200] = TINY                                     # exactly the bound: a normal block
    x[4, 128:256] = 0.0
    x[4, 200] = float(np.nextafter(np.float32(TINY), np.float32(0)))
    x[5, 17] = torch.finfo(torch.float32).max
    x[6, 17] = float("inf")
    x[7, 300] = float("-inf")
    x[8, 5] = float("nan")
    x[9, :] = float("nan")
    x[10] *= 1e30
    x[11, 0] = 2.0 ** -149
    codes, sf = B.fp8_quantize(x.to(DEV))
    want, want_sf = _rule_rows(x)
    assert _same(codes, want) and _same_scales(sf, want_sf)
    back = codes.view(F8).float().cpu().view(12, 3, 128) * sf.cpu()[..., None]
    whole = torch.isnan(back).all(-1)
    assert whole.sum() == 6 and whole[6, 0] and whole[7, 2] and whole[8, 0] and whole[9].all()
    assert not torch.isnan(back[~whole]).any()


@pytest.mark.parametrize("T,k,K,extra,dropped", [(1, 1, 16, 0, 0), (9, 8, 640, 0, 0), (40, 6, 1040, 13, 0.3),
                                                 (64, 16, 128, 0, 0)])
def test_rows_written_in_expert_order(T, k, K, extra, dropped):
    rng = np.random.default_rng(T)
    R = T * k + extra
    p = rng.permutation(R)[:T * k].astype(np.int32)
    p[rng.random(T * k) < dropped] = -1
    x = _rand((T, K), 2, dtype=torch.bfloat16)
    codes = torch.full((R, K), 0x55, dtype=torch.uint8, device=DEV)
    sf = torch.full((R, _blocks(K)), -3.0, device=DEV)
    B.fp8_quantize(x.to(DEV), flat_to_perm=torch.from_numpy(p).to(DEV), k=k, out_rows=R, codes=codes, sf=sf)
    one, one_sf = B.fp8_quantize(x.to(DEV))
    want = torch.full((R, K), 0x55, dtype=torch.uint8)
    want_sf = torch.full((R, _blocks(K)), -3.0)
    for f, r in enumerate(p):
        if r >= 0:
            want[r], want_sf[r] = one[f // k].cpu(), one_sf[f // k].cpu()
    assert torch.equal(codes.cpu(), want) and torch.equal(sf.cpu(), want_sf)
    assert B.nvfp4moe_last_device_status() == 0


def test_a_row_out_of_range_is_reported_and_skipped():
    x = _rand((3, 64), 1).to(DEV)
    p = torch.tensor([0, 3, 1], dtype=torch.int32, device=DEV)
    guard = torch.full((9, 64), 0x11, dtype=torch.uint8, device=DEV)
    sf = torch.zeros((9, 1), device=DEV)
    B.fp8_quantize(x, flat_to_perm=p, k=1, out_rows=3, codes=guard[3:6], sf=sf[3:6])
    assert B.nvfp4moe_last_device_status() == -1
    assert (guard[:3] == 0x11).all() and (guard[5:] == 0x11).all() and (sf[5:] == 0).all()
    assert torch.equal(guard[3:5], B.fp8_quantize(x[[0, 2]])[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("E,N,K", [(1, 1, 16), (1, 128, 128), (2, 130, 272), (3, 300, 1040)])
def test_weight_blocks_match_the_rule_bit_for_bit(E, N, K, dtype):
    w = _rand((E, N, K), N, 0.02, dtype)
    w[0, :, :16] = 0
    if N > 128:
        w[-1, 128:] = 0
    codes, sf = B.fp8_quantize_weight(w.to(DEV))
    want, want_sf = _rule_weight(w)
    assert _same(codes, want) and _same_scales(sf, want_sf)
    if E == 1:
        c2, s2 = B.fp8_quantize_weight(w[0].to(DEV))
        assert torch.equal(c2, codes[0]) and torch.equal(s2, sf[0])


def _e4m3(q):
    """Nearest E4M3 value of 64-bit numbers, ties to even."""
    mag = q.abs().clamp_max(448.0)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))) - 3)
    return torch.copysign(torch.round(mag / step) * step, q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,I", [(1, 16), (5, 144), (40, 2048)])
def test_swiglu_codes_are_those_of_nearby_values(M, I, dtype):
    """The f32 h is within 2^-20 of the exact one (exponential and reciprocal 2 ulp
    each, the sum and the products half an ulp, the exponent's own rounding
    |g| 2^-24 with |g| below 10 wherever the code is not 0), so the scale is too
    and every code lies between the codes of x * inv * (1 -+ 2^-20)."""
    gu = _rand((M, 2 * I), 7, 2.0, dtype)
    gu[0, :4] = torch.tensor([-100.0, 100.0, 0.0, -20.0]).to(dtype)
    codes, sf = B.fp8_swiglu_quantize(gu.to(DEV))
    g, u = gu.double().chunk(2, 1)
    h = _pad(g * torch.sigmoid(g) * u, 1).view(M, -1, 128)
    amax = h.abs().amax(-1, keepdim=True)
    d = 2.0 ** -20
    assert ((sf.cpu().double() - amax[..., 0] / 448).abs() <= d * amax[..., 0] / 448).all()
    q = h * (448.0 / amax.clamp_min(TINY))
    got = _pad(codes.view(F8).cpu().double(), 1).view(M, -1, 128).abs()
    q = q.abs()
    # the f32 exponential overflows to infinity below -88: such a value is 0
    assert ((got >= _e4m3(q * (1 - d)) - 0.0) & (got <= _e4m3(q * (1 + d)))).all()
    assert (torch.signbit(_pad(codes.view(F8).cpu().float(), 1).view(M, -1, 128)) == torch.signbit(h))[got > 0].all()


# ------------------------------------------------------------------ products

def _operands(M, E, N, K, seed):
    a, sa = B.fp8_quantize(_rand((max(M, 1), K), seed).to(DEV))
    w, sw = B.fp8_quantize_weight(_rand((E, N, K), seed + 1, 0.05).to(DEV))
    return a[:M], sa[:M], w, sw


def _values(codes, sf, each):
    v = codes.view(F8).double()
    s = sf.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]
    if each > 1:
        s = s.repeat_interleave(each, -2)[..., :codes.shape[-2], :]
    return v * s


def _check(got, a, sa, w, sw, out, what):
    """f32 sums of K products in 128-element blocks: at most K + KB additions, each
    within one step of f32 (the tensor core may truncate) of the summed magnitudes,
    two roundings of the scales' product and its use, and one rounding to the type."""
    va, vw = _values(a, sa, 1), _values(w, sw, 128)
    want, size = va @ vw.t(), va.abs() @ vw.abs().t()
    K = a.shape[1]
    lim = (K + _blocks(K) + 2) * 2 * U32 * size
    lim = lim + torch.finfo(out).eps / 2 * (want.abs() + lim) + torch.finfo(out).smallest_normal
    assert got.dtype == out
    bad = (got.double() - want).abs() > lim
    assert not bad.any(), "%s: %d of %d" % (what, int(bad.sum()), bad.numel())


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 4096, 7168), (2, 128, 128), (17, 100, 144), (128, 256, 512),
                                   (129, 257, 528), (333, 1111, 2000), (64, 640, 16), (700, 384, 1040),
                                   (24, 384, 640), (40, 333, 400), (16, 130, 7168), (32, 129, 2064)])
def test_linear(M, N, K, out):
    a, sa, w, sw = _operands(M, 1, N, K, M + N + K)
    got = B.fp8_linear(a, sa, w[0], sw[0], out_dtype=out)
    _check(got, a, sa, w[0], sw[0], out, "linear")
    assert B.nvfp4moe_last_device_status() == 0
    assert torch.equal(B.fp8_linear(a.view(F8), sa, w[0].view(F8), sw[0], out_dtype=out), got)   # and again


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1200, 2304, 1040), (1300, 2303, 528), (1150, 2306, 144), (1290, 2308, 256),
                                   (128, 4096, 7168), (100, 4100, 7168), (65, 8200, 1024), (4100, 300, 400)])
def test_linear_of_many_tiles(M, N, K, out):
    """More tiles than SMs, or tiles whose blocks of K a cluster shares; rows of C
    that are whole sectors, whole 16, 8, 4 bytes, or none of them."""
    a, sa, w, sw = _operands(M, 1, N, K, M + N + K)
    got = B.fp8_linear(a, sa, w[0], sw[0], out_dtype=out)
    _check(got, a, sa, w[0], sw[0], out, "linear")
    assert B.nvfp4moe_last_device_status() == 0


@pytest.mark.parametrize("counts,N,K", [([1], 128, 128), ([0, 0, 5], 200, 272), ([3, 0, 128, 129, 0, 1], 257, 400),
                                        ([0, 300, 16, 17, 32, 33, 64, 65], 512, 1024),
                                        ([2] * 70, 384, 256), ([1000, 0, 0, 1], 300, 2000),
                                        ([900, 0, 700, 1, 300, 129], 2050, 400), ([1500, 127, 0, 600], 2304, 528),
                                        ([1] * 600, 520, 128)])
def test_grouped(counts, N, K):
    E, M = len(counts), sum(counts)
    a, sa, w, sw = _operands(M, E, N, K, M + N)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    for out in (torch.bfloat16, torch.float32):
        got = B.fp8_grouped_gemm(a, sa, w, sw, off, out_dtype=out)
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            _check(got[lo:hi], a[lo:hi], sa[lo:hi], w[e], sw[e], out, "expert %d" % e)
    assert B.nvfp4moe_last_device_status() == 0


@pytest.mark.parametrize("M,N,K", [(5, 130, 640), (200, 512, 2048), (1, 256, 7168)])
def test_exact_where_every_partial_sum_is(M, N, K):
    """Codes of 0, +-1, +-2 and +-4 and scales that are powers of two of a narrow
    range: every partial sum is a multiple of 2^-4 below 2^20, exact in f32 in
    any order, so the f32 result has no rounding at all."""
    rng = np.random.default_rng(K)
    vals = torch.tensor([0.0, 1.0, -1.0, 2.0, -2.0, 4.0, -4.0])
    a = vals[torch.from_numpy(rng.integers(0, 7, (M, K)))].to(F8)
    w = vals[torch.from_numpy(rng.integers(0, 7, (N, K)))].to(F8)
    sa = torch.exp2(torch.from_numpy(rng.integers(-2, 2, (M, _blocks(K)))).float())
    sw = torch.exp2(torch.from_numpy(rng.integers(-2, 2, (_blocks(N), _blocks(K)))).float())
    got = B.fp8_linear(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), out_dtype=torch.float32)
    want = _values(a.view(torch.uint8), sa, 1) @ _values(w.view(torch.uint8), sw, 128).t()
    assert torch.equal(got.double().cpu(), want)


def test_strides_and_unaligned_outputs():
    M, N, K = 150, 200, 272
    a, sa, w, sw = _operands(M, 1, N, K, 3)
    want = B.fp8_linear(a, sa, w[0], sw[0])
    wide_a = torch.full((M, K + 48), 0x7F, dtype=torch.uint8, device=DEV)
    wide_w = torch.full((N, K + 16), 0x7F, dtype=torch.uint8, device=DEV)
    wide_a[:, 32:32 + K], wide_w[:, :K] = a, w[0]
    for pad, shift in [(0, 0), (1, 0), (24, 8), (16, 3)]:
        c = torch.full((M, N + pad + shift), 9.0, dtype=torch.bfloat16, device=DEV)
        got = B.fp8_linear(wide_a[:, 32:32 + K], sa, wide_w[:, :K], sw[0], out=c[:, shift:shift + N])
        assert torch.equal(got, want)
        assert (c[:, :shift] == 9).all() and (c[:, shift + N:] == 9).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N", [3, 131, 256, 300])
def test_rows_of_c_that_start_anywhere(N, dtype):
    """Enough rows for the form with 128-row tiles: the values of rows at every
    alignment are those of rows alone, and nothing beside them is written."""
    M, K = 80000 if N < 128 else 20100, 144
    a, sa, w, sw = _operands(M, 1, N, K, 5)
    want = B.fp8_linear(a, sa, w[0], sw[0], out_dtype=dtype)
    _check(want[:300], a[:300], sa[:300], w[0], sw[0], dtype, "linear")
    _check(want[-300:], a[-300:], sa[-300:], w[0], sw[0], dtype, "linear")
    for pad, shift in [(0, 0), (1, 0), (0, 1), (2, 5), (16, 16), (5, 8), (3, 15), (12, 4), (8, 7), (6, 2)]:
        ld = N + pad + shift
        c = torch.full((M, ld), 9.0, dtype=dtype, device=DEV)
        got = B.fp8_linear(a, sa, w[0], sw[0], out=c[:, shift:shift + N])
        assert torch.equal(got, want), (pad, shift)
        assert (c[:, :shift] == 9).all() and (c[:, shift + N:] == 9).all(), (pad, shift)
    assert B.nvfp4moe_last_device_status() == 0


def test_bad_values_stay_in_their_row_and_column():
    M, N, K = 70, 300, 256
    a, sa, w, sw = _operands(M, 1, N, K, 4)
    want = B.fp8_linear(a, sa, w[0], sw[0], out_dtype=torch.float32)
    a2, sa2, w2 = a.clone(), sa.clone(), w.clone()
    a2[3, 200] = 0x7F                                    # a NaN code
    sa2[40, 0] = float("inf")
    w2[0, 299, 0] = 0xFF
    got = B.fp8_linear(a2, sa2, w2[0], sw[0], out_dtype=torch.float32)
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[40]).any() and torch.isnan(got[:, 299]).all()
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[[3, 40]] = False
    assert torch.equal(got[keep][:, :299], want[keep][:, :299])


def test_bad_offsets_write_nothing_outside():
    """Bounds past the operands, negative or descending are clamped."""
    M, N, K, E = 40, 130, 144, 4
    a, sa, w, sw = _operands(M, E, N, K, 6)
    for bounds in ([0, 10, 2 ** 31 - 1, 5, 40], [-7, 3, 3, 2 ** 30, 60], [50, 60, 70, 80, 90]):
        off = torch.tensor(bounds, dtype=torch.int32, device=DEV)
        guard = torch.full((M + 300, N), 3.0, device=DEV)
        got = B.fp8_grouped_gemm(a, sa, w, sw, off, out=guard[150:150 + M])
        assert (guard[:150] == 3).all() and (guard[150 + M:] == 3).all()
        assert B.nvfp4moe_last_device_status() == 0
        for e in range(E):
            lo = min(max(bounds[e], 0), M)
            hi = min(max(bounds[e + 1], lo), M)
            if bounds == [-7, 3, 3, 2 ** 30, 60] and hi > lo and e != 3:
                _check(got[lo:hi], a[lo:hi], sa[lo:hi], w[e], sw[e], torch.float32, "expert %d" % e)


def test_empty_products():
    a, sa, w, sw = _operands(0, 3, 64, 128, 2)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    assert B.fp8_grouped_gemm(a, sa, w, sw, off).shape == (0, 64)
    assert B.fp8_linear(a, sa, w[0], sw[0]).shape == (0, 64)
    a, sa, _, _ = _operands(5, 1, 64, 128, 2)
    out = torch.full((5, 64), 2.0, dtype=torch.bfloat16, device=DEV)
    B.fp8_grouped_gemm(a, sa, w, sw, off, out=out)       # no group has a row
    assert (out == 2).all()


@pytest.mark.parametrize("M,N", [(3, 512), (700, 512), (2500, 4096), (128, 4096)])
def test_a_wait_that_runs_out_is_reported(M, N):
    a, sa, w, sw = _operands(M, 1, N, 1024, 8)
    good = B.fp8_linear(a, sa, w[0], sw[0])
    assert B.nvfp4moe_last_device_status() == 0
    try:
        B.nvfp4moe_set_wait_limit_ns(20_000_000)
        B.nvfp4moe_set_test_stall(True)
        B.fp8_linear(a, sa, w[0], sw[0])
        assert B.nvfp4moe_last_device_status() == -5
    finally:
        B.nvfp4moe_set_test_stall(False)
        B.nvfp4moe_set_wait_limit_ns(4_000_000_000)
    assert torch.equal(B.fp8_linear(a, sa, w[0], sw[0]), good)
    assert B.nvfp4moe_last_device_status() == 0


def test_graph_capture():
    a, sa, w, sw = _operands(100, 1, 384, 512, 9)
    want = B.fp8_linear(a, sa, w[0], sw[0])
    x = _rand((100, 512), 9).to(DEV)
    out = torch.zeros_like(want)
    codes, sf = torch.empty_like(a), torch.empty_like(sa)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.fp8_quantize(x, codes=codes, sf=sf)
        B.fp8_linear(codes, sf, w[0], sw[0], out=out)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals():
    a, sa, w, sw = _operands(8, 2, 64, 128, 2)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    x = torch.zeros((8, 128), device=DEV)
    for bad in [lambda: B.fp8_quantize(x.double()), lambda: B.fp8_quantize(x[:, :120]),
                lambda: B.fp8_quantize(x[:, 1:113]), lambda: B.fp8_quantize(x.t()),
                lambda: B.fp8_quantize(x, flat_to_perm=off, k=2), lambda: B.fp8_quantize(x, out_rows=7),
                lambda: B.fp8_quantize_weight(x[:, :120]), lambda: B.fp8_quantize_weight(x[0]),
                lambda: B.fp8_swiglu_quantize(x[:, :31]), lambda: B.fp8_swiglu_quantize(x[:, :24]),
                lambda: B.fp8_linear(a, sa, w[0][:, :64], sw[0]), lambda: B.fp8_linear(a, sa[:7], w[0], sw[0]),
                lambda: B.fp8_linear(a, sa, w[0], sw), lambda: B.fp8_linear(a.float(), sa, w[0], sw[0]),
                lambda: B.fp8_linear(a, sa.half(), w[0], sw[0]),
                lambda: B.fp8_linear(a, sa, w[0], sw[0], out_dtype=torch.float64),
                lambda: B.fp8_linear(a, sa, w[0], sw[0], out=torch.zeros((8, 63), device=DEV)),
                lambda: B.fp8_linear(a[:, 8:72], sa, w[0][:, :64].contiguous(), sw[0]),
                lambda: B.fp8_grouped_gemm(a, sa, w, sw, off[:2]), lambda: B.fp8_grouped_gemm(a, sa, w[0], sw, off),
                lambda: B.fp8_grouped_gemm(a, sa, w, sw, off.long()), lambda: B.fp8_linear(a.cpu(), sa, w[0], sw[0])]:
        with pytest.raises(B.NVFP4Error):
            bad()
