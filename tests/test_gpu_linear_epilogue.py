"""fp8_linear_epilogue: act(A W^T + bias) + residual, against fp8_linear and 64 bits."""
import math

import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _operands(M, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    up = -(-K // 16) * 16
    a, sa = B.fp8_quantize(torch.randn(M, up, generator=g).to(DEV))
    w, sw = B.fp8_quantize_weight((torch.randn(N, up, generator=g) * (4.0 / math.sqrt(K))).to(DEV))
    return a[:, :K], sa, w[:, :K], sw, torch.randn(N, generator=g).to(DEV), torch.randn(M, N, generator=g).to(DEV)


def _values(codes, sf, each):
    v = codes.contiguous().view(torch.float8_e4m3fn).double()
    s = sf.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]
    if each > 1:
        s = s.repeat_interleave(each, -2)[..., :codes.shape[-2], :]
    return v * s


def _act(v, act):
    if act == "relu":
        return v.clamp_min(0.0)
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v / math.sqrt(2.0))
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return v * torch.sigmoid(v) if act == "silu" else v


# one row and few (columns as lanes), clusters that share K, whole tiles, several tiles a
# CTA, and widths whose rows start on no sector
SIZES = [(1, 4096, 512), (1, 130, 64), (17, 257, 400), (64, 8191, 128), (100, 512, 2048), (128, 96, 48), (333, 1111, 272),
         (600, 512, 496), (1300, 4096, 256), (2100, 2050, 128)]


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_parts(M, N, K, dtype):
    """Without an activation the parts are f32 additions to fp8_linear's sums, before or after
    them: each of the blocks' additions rounds by 2^-24 of the bias and residual more."""
    a, sa, w, sw, bias, res = _operands(M, N, K, M + N)
    res = res.to(dtype)
    sums = B.fp8_linear(a, sa, w, sw, out_dtype=F32)
    size = _values(a, sa, 1).abs() @ _values(w, sw, 128).abs().t()
    for b, r in ((None, None), (bias, None), (None, res), (bias, res)):
        for act in ("none", "relu"):
            want = sums if b is None else sums + b
            want = want.clamp_min(0.0) if act == "relu" else want
            want = want if r is None else want + r.float()
            got = B.fp8_linear_epilogue(a, sa, w, sw, bias=b, activation=act, residual=r, out_dtype=dtype)
            if b is None and r is None:
                assert got.dtype == dtype and torch.equal(got, want.to(dtype)), (act, b is None, r is None)
                continue
            more = size + (0 if b is None else b.double().abs()) + (0 if r is None else r.double().abs())
            off = 2 * (K // 128 + 4) * 2.0 ** -24 * more
            off = off + torch.finfo(dtype).eps / 2 * (want.double().abs() + off)
            assert got.dtype == dtype and ((got.double() - want.double()).abs() <= off).all(), (act, b is None, r is None)
    assert B.nvfp4moe_last_device_status() == 0


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", SIZES)
def test_activations(M, N, K, act):
    a, sa, w, sw, bias, res = _operands(M, N, K, M + N + 1)
    va, vw = _values(a, sa, 1), _values(w, sw, 128)
    pre, size = va @ vw.t() + bias.double(), va.abs() @ vw.abs().t() + bias.double().abs()
    for dtype in (F32, BF16):
        r = res.to(dtype)
        want = _act(pre, act) + r.double()
        got = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, residual=r, out_dtype=dtype).double()
        # a step of 2^-23 for each of the K products and the blocks' and bias' sums, through a slope of at
        # most 1.13; the activation itself within 2^-20 of its argument; the residual's sum; the result's half step
        off = 1.13 * (K + K // 128 + 3) * 2.0 ** -23 * size + 2.0 ** -20 * pre.abs()
        off = off + (torch.finfo(dtype).eps / 2 + 2.0 ** -24) * (want.abs() + off)
        assert ((got - want).abs() <= off).all(), float(((got - want).abs() / off).max())


@pytest.mark.parametrize("act", ACTS)
def test_far_values(act):
    """Arguments over the whole f32 range, infinities and NaN, through the bias."""
    a = torch.zeros(3, 128, dtype=torch.uint8, device=DEV)
    w = torch.zeros(64, 128, dtype=torch.uint8, device=DEV)
    sa, sw = torch.ones(3, 1, device=DEV), torch.ones(1, 1, device=DEV)
    v = torch.tensor([0.0, 1e-30, 1e-6, 0.5, 3.0, 10.0, 20.0, 80.0, 90.0, 1e4, 1e30, 3e38, math.inf], device=DEV)
    bias = torch.zeros(64, device=DEV)
    bias[:13], bias[13:26], bias[26] = v, -v, math.nan
    got = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, out_dtype=F32)
    want = _act(bias.double(), act)
    want[25] = {"none": -math.inf}.get(act, 0.0)          # the limit at minus infinity
    want[12] = math.inf
    assert torch.isnan(got[:, 26]).all()
    ok = ~torch.isnan(bias)
    g, t = got[:, ok].double(), want[ok]
    # four roundings of 2^-24 on an exponent that is below 2^4 where the result counts
    near = (g - t).abs() <= 2.0 ** -18 * t.abs()
    assert ((g == t) | near | ((t.abs() < 1e-6) & (g.abs() < 1e-6))).all()


@pytest.mark.parametrize("M,N", [(1, 300), (40, 512), (300, 640), (300, 333), (2000, 4096)])
def test_in_place_and_strides(M, N):
    """The residual's place taken by the result; rows apart by more than their width."""
    a, sa, w, sw, bias, res = _operands(M, N, 384, 5)
    want = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation="silu", residual=res, out_dtype=F32)
    own = res.clone()
    got = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation="silu", residual=own, out=own)
    assert got.data_ptr() == own.data_ptr() and torch.equal(own, want)
    for pad, shift in ((8, 0), (3, 1), (0, 5)):
        buf = torch.full((M, N + pad + shift), 9.0, device=DEV)
        out = buf[:, shift:shift + N]
        out.copy_(res)
        B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation="silu", residual=out, out=out)
        assert torch.equal(out, want)
        other = torch.zeros(M, N + 7, device=DEV)[:, 2:N + 2]
        other.copy_(res)
        assert torch.equal(B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation="silu", residual=other,
                                                 out_dtype=F32), want)
        out.fill_(9.0)
        assert (buf == 9.0).all()


def test_no_rows_and_graph():
    a, sa, w, sw, bias, res = _operands(200, 384, 256, 6)
    assert B.fp8_linear_epilogue(a[:0], sa[:0], w, sw, bias=bias, residual=res[:0], out_dtype=F32).shape == (0, 384)
    want = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation="gelu", residual=res, out_dtype=F32)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation="gelu", residual=res, out_dtype=F32)
    for _ in range(2):
        got.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_refusals():
    a, sa, w, sw, bias, res = _operands(20, 64, 128, 7)
    call = B.fp8_linear_epilogue
    grown = torch.cat([bias[:1], bias])[1:]     # off 16-byte boundaries
    for kw in ({"bias": bias[:32]}, {"bias": bias.bfloat16()}, {"bias": grown}, {"activation": "tanh"}, {"activation": 1},
               {"residual": res}, {"residual": res[:10], "out_dtype": F32}, {"residual": res.t(), "out_dtype": F32},
               {"out": torch.empty(20, 63, device=DEV)}, {"bias": bias.clone().requires_grad_()},
               {"residual": res.clone().requires_grad_(), "out_dtype": F32}):
        with pytest.raises(B.NVFP4Error):
            call(a, sa, w, sw, **kw)
    with torch.no_grad():
        call(a, sa, w, sw, bias=bias.clone().requires_grad_())


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("M,N,K", SIZES + [(4096, 640, 7168), (4100, 520, 1040)])
def test_f32_parts_are_single_additions(M, N, K, act):
    """An F32 result is fp8_linear's sums, the bias and the residual in one addition each, whatever their size."""
    a, sa, w, sw, bias, res = _operands(M, N, K, M + N)
    sums = B.fp8_linear(a, sa, w, sw, out_dtype=F32)
    far = torch.where(torch.arange(N, device=DEV) % 3 == 0, 2.0 ** 20, 1.0)
    for b, r in ((bias, None), (None, res), (bias, res), (bias * far, None), (None, res * far), (bias * far, -res * far)):
        want = sums if b is None else sums + b
        want = want.clamp_min(0.0) if act == "relu" else want
        want = want if r is None else want + r
        got = B.fp8_linear_epilogue(a, sa, w, sw, bias=b, activation=act, residual=r, out_dtype=F32)
        assert torch.equal(got, want), (b is None, r is None)


@pytest.mark.parametrize("M", [3, 300, 2500])
def test_products_far_below_the_residual(M):
    """56 blocks of 0.05 beside a residual, or a bias, of 2^20: an F32 result keeps their sum."""
    N, K = 272, 7168
    a = torch.zeros(M, K, device=DEV)
    a[:, ::128] = 0.05
    w = torch.zeros(N, K, device=DEV)
    w[:, ::128] = 1.0
    (a, sa), (w, sw) = B.fp8_quantize(a), B.fp8_quantize_weight(w)
    sums = (_values(a, sa, 1) @ _values(w, sw, 128).t())
    for act in ("none", "relu"):
        res = torch.full((M, N), 2.0 ** 20, device=DEV)
        got = B.fp8_linear_epilogue(a, sa, w, sw, activation=act, residual=res, out_dtype=F32).double()
        # half a step of 2^20's f32, and the 56 sums' own roundings
        assert ((got - 2.0 ** 20 - sums).abs() <= 2.0 ** -4 + 64 * 2.0 ** -24 * sums).all()
        got = B.fp8_linear_epilogue(a, sa, w, sw, bias=res[0], activation=act, out_dtype=F32).double()
        assert ((got - 2.0 ** 20 - sums).abs() <= 2.0 ** -4 + 64 * 2.0 ** -24 * sums).all()
        for dtype in (BF16, F16):        # 2^15 is in F16's range: its step is larger than the products' sum
            res16 = torch.full((M, N), 2.0 ** 15, dtype=dtype, device=DEV)
            got = B.fp8_linear_epilogue(a, sa, w, sw, activation=act, residual=res16, out_dtype=dtype).double()
            want = 2.0 ** 15 + sums
            assert ((got - want).abs() <= (torch.finfo(dtype).eps / 2 + 64 * 2.0 ** -24) * want).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 300, 2500])
def test_infinite_residuals(M, act, dtype):
    """An infinity or NaN of the residual is the result's, and stays in its place."""
    N, K = 264, 384
    a, sa, w, sw, bias, res = _operands(M, N, K, 8)
    res = res.to(dtype)
    want = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, residual=res, out_dtype=dtype)
    places = [(0, 0, math.inf), (M - 1, N - 1, -math.inf), (M // 2, 129, math.nan), (M // 2, 7, math.inf)]
    for i, j, v in places:
        res[i, j] = v
    got = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, residual=res, out_dtype=dtype)
    for i, j, v in places:
        assert torch.isnan(got[i, j]) if math.isnan(v) else got[i, j] == v
        got[i, j] = want[i, j]
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [3, 2500])
@pytest.mark.parametrize("act", ACTS)
def test_small_and_far_arguments(act, M):
    """Every argument's own bits, down to the smallest, through the bias: no absolute allowance
    but where the exponential leaves f32's range."""
    a = torch.zeros(M, 128, dtype=torch.uint8, device=DEV)
    w = torch.zeros(64, 128, dtype=torch.uint8, device=DEV)
    sa, sw = torch.ones(M, 1, device=DEV), torch.ones(1, 1, device=DEV)
    v = torch.tensor([1e-35, 1e-30, 1e-20, 1e-10, 1e-6, 1e-3, 0.03, 0.5, 1.0, 2.0, 3.0, 4.0, 5.5, 7.0, 9.0, 12.0, 15.0, 20.0,
                      40.0, 80.0, 86.0, 1e3, 1e10, 3e38], device=DEV)
    bias = torch.zeros(64, device=DEV)
    bias[:24], bias[24:48] = v, -v
    got = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, out_dtype=F32).double()
    if act in ("none", "relu"):
        assert torch.equal(got, _act(bias.double(), act).expand(M, 64))
        return
    b = bias.double()
    want = _act(b, act)
    if act == "gelu_tanh":                       # 1 + tanh(u) = 2 sigmoid(2u), without the cancellation
        want = b * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (b + 0.044715 * b ** 3))
    # the exponent, whose factors' and products' roundings (at most 8 of 2^-24) the exponential carries over
    exponent = {"silu": b.abs(), "gelu": b * b / 2, "gelu_tanh": 1.6 * b.abs() * (1 + 0.045 * b * b)}[act].clamp_max(90.0)
    # gelu: ten steps of its polynomial, whose coefficients add up to 1.73 of its value; below 2^-126 results are 0
    off = (2.0 ** -19 + 2.0 ** -21 * exponent) * want.abs() + 87 * 2.0 ** -126
    assert ((got - want).abs() <= off).all(), float(((got - want).abs() / off).max())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("M,N", [(3, 264), (300, 640), (300, 333), (2000, 4096), (2500, 1031)])
def test_residuals_in_place(M, N, act, dtype):
    """A result in its residual's place, wherever the residual is added, again and again the same."""
    a, sa, w, sw, bias, res = _operands(M, N, 640, 9)
    res = res.to(dtype)
    want = B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, residual=res, out_dtype=dtype)
    for _ in range(5):
        own = res.clone()
        B.fp8_linear_epilogue(a, sa, w, sw, bias=bias, activation=act, residual=own, out=own)
        assert torch.equal(own, want)
