"""moe_sort_tokens, moe_unsort_tokens and their gradients against the formulas in
64 bits, at odd widths, strides, dropped slots and rows that nothing names."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32 = 2.0 ** -24                       # half a step of f32, relative


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _least(dtype):
    """Half a step among the subnormal numbers of a type, absolute."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def _place(T, k, n_rows, dropped, seed):
    """Distinct rows for the T * k slots, some of them dropped."""
    rng = np.random.default_rng(seed)
    p = rng.permutation(n_rows)[:T * k].astype(np.int32)
    p[rng.random(T * k) < dropped] = -1
    return torch.from_numpy(p)


def _tensor(shape, dtype, seed, ld=None, shift=0):
    """Random rows with a leading dimension and an element offset of their own."""
    g = torch.Generator().manual_seed(seed)
    ld = shape[1] if ld is None else ld
    base = torch.randn(shift + shape[0] * ld + 8, generator=g).to(dtype).to(DEV)
    return base[shift:shift + shape[0] * ld].view(shape[0], ld)[:, :shape[1]] if shape[0] else \
        torch.empty(shape, dtype=dtype, device=DEV)


def _weights(T, k, seed):
    return torch.softmax(torch.randn(T, k, generator=torch.Generator().manual_seed(seed)), 1)


def _close(got, want, size, dtype, steps, what):
    """|got - want| within `steps` f32 roundings of the summed magnitudes `size`
    and one rounding to dtype."""
    got, want = got.double().cpu(), want.double()
    lim = steps * U32 * size + _half_step(dtype) * (want.abs() + steps * U32 * size) + _least(dtype)
    bad = (got - want).abs() > lim
    assert not bad.any(), "%s: %d of %d out of tolerance" % (what, int(bad.sum()), bad.numel())


CASES = [
    # T, k, K, extra rows, dropped, leading dimension - K, element offset
    (1, 1, 1, 0, 0.0, 0, 0),
    (1, 16, 7, 0, 0.0, 0, 0),
    (5, 2, 8, 3, 0.3, 0, 0),
    (33, 8, 1001, 0, 0.0, 0, 0),
    (33, 6, 1001, 40, 0.2, 7, 1),
    (64, 4, 2056, 0, 0.0, 8, 8),
    (130, 8, 7168, 0, 0.0, 0, 0),
    (17, 9, 515, 5, 0.5, 0, 3),
    (3, 3, 40, 0, 1.0, 0, 0),           # every slot dropped
    (700, 8, 401, 9, 0.1, 0, 0),        # many tokens, short rows
    (700, 2, 72, 0, 0.0, 8, 0),
    (650, 16, 500, 0, 0.1, 1, 1),
    (700, 3, 1790, 0, 0.0, 2, 0),
    (2501, 8, 64, 5, 0.1, 0, 0),        # more tokens still, a warp each
    (2434, 2, 101, 0, 0.1, 1, 1),
    (3001, 1, 1, 0, 0.5, 0, 0),
    (2435, 16, 24, 0, 0.0, 8, 8),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,k,K,extra,dropped,pad,shift", CASES)
def test_against_the_formulas(T, k, K, extra, dropped, pad, shift, weighted, dtype):
    R = T * k + extra
    f2p = _place(T, k, R, dropped, T + K)
    live = f2p >= 0
    w = _weights(T, k, 3) if weighted else None
    wd = w.double() if weighted else torch.ones(T, k, dtype=torch.float64)
    x = _tensor((T, K), dtype, 1, K + pad, shift)
    rows = _tensor((R, K), dtype, 2, K + pad, shift)
    xd, rd = x.double().cpu(), rows.double().cpu()
    dev_f2p, dev_w = f2p.to(DEV), w.to(DEV) if weighted else None
    # token rows out to the slots' rows
    scaled = (xd[:, None, :] * wd[..., None]).reshape(-1, K)
    for call, what in [(lambda o: B.moe_sort_tokens(x, dev_f2p, k, topk_w=dev_w, rows=o), "sort"),
                       (lambda o: B.moe_unsort_tokens_backward(x, dev_f2p, k, topk_w=dev_w,
                                                               rows=rows if weighted else None, d_rows=o),
                        "unsort backward")]:
        out = torch.full((R, K + pad), 7.0, dtype=dtype, device=DEV)[:, :K]
        got = call(out)
        d_w = None
        if isinstance(got, tuple):
            got, d_w = got
        assert got.data_ptr() == out.data_ptr()
        at = f2p[live].long()
        _close(got.cpu()[at], scaled[live], scaled[live].abs(), dtype, 1, what)
        rest = torch.ones(R, dtype=torch.bool)
        rest[at] = False
        assert torch.equal(got.cpu()[rest], torch.full((int(rest.sum()), K), 7.0, dtype=dtype)), what
        if d_w is not None:
            _dots(d_w, rd, xd, f2p, T, k, K, what)
    # slots' rows back to the tokens
    taken = torch.where(live[:, None], rd[f2p.long().clamp_min(0)], 0.0).view(T, k, K)
    want = (taken * wd[..., None]).sum(1)
    size = (taken.abs() * wd[..., None]).sum(1)
    y = B.moe_unsort_tokens(rows, dev_f2p, k, topk_w=dev_w)
    _close(y, want, size, dtype, k, "unsort")
    dx, d_w = B.moe_sort_tokens_backward(rows, dev_f2p, k, topk_w=dev_w, x=x if weighted else None)
    _close(dx, want, size, dtype, k, "sort backward")
    if weighted:
        _dots(d_w, rd, xd, f2p, T, k, K, "sort backward")
    else:
        assert d_w is None
    assert B.nvfp4moe_last_device_status() == 0


def _dots(d_w, rd, xd, f2p, T, k, K, what):
    live = (f2p >= 0).view(T, k)
    prod = rd[f2p.long().clamp_min(0)].view(T, k, K) * xd[:, None, :]
    want = torch.where(live, prod.sum(-1), 0.0)
    size = torch.where(live, prod.abs().sum(-1), 0.0)
    assert d_w.dtype == torch.float32
    _close(d_w, want, size, torch.float32, K, what)


def test_gradients_against_differences():
    """The sums are linear in rows, tokens and weights alike: a central difference
    of a forward call's inner product is its gradient up to rounding. f32; every
    term of the inner products is below 8 in magnitude, there are T*k*K of them,
    and the step is 1/4."""
    T, k, K, h = 6, 3, 20, 0.25
    f2p = _place(T, k, T * k, 0.0, 4)
    d2p, w = f2p.to(DEV), _weights(T, k, 5).to(DEV)
    x, g = _tensor((T, K), torch.float32, 6), _tensor((T * k, K), torch.float32, 7)
    dx, d_w = B.moe_sort_tokens_backward(g, d2p, k, topk_w=w, x=x)
    lim = T * k * K * 64 * U32 / h

    def sort_loss(x, w):
        return float((B.moe_sort_tokens(x, d2p, k, topk_w=w).double() * g.double()).sum())

    def unsort_loss(rows, w):
        return float((B.moe_unsort_tokens(rows, d2p, k, topk_w=w).double() * x.double()).sum())

    d_rows, d_w2 = B.moe_unsort_tokens_backward(x, d2p, k, topk_w=w, rows=g)
    for loss, a, grads in [(sort_loss, x, (dx, d_w)), (unsort_loss, g, (d_rows, d_w2))]:
        for i, j in [(0, 0), (3, 7), (5, 19)]:
            up, down = a.clone(), a.clone()
            up[i, j] += h
            down[i, j] -= h
            assert abs((loss(up, w) - loss(down, w)) / (2 * h) - float(grads[0][i, j])) <= lim
        for i, j in [(0, 0), (2, 1), (5, 2)]:
            up, down = w.clone(), w.clone()
            up[i, j] += h
            down[i, j] -= h
            assert abs((loss(a, up) - loss(a, down)) / (2 * h) - float(grads[1][i, j])) <= lim


@pytest.mark.parametrize("K", [8, 33])
def test_rows_out_of_range_are_reported_and_skipped(K):
    T, k = 4, 2
    f2p = torch.tensor([0, 1, 2, 9, 4, 5, 6, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    x, rows = _tensor((T, K), torch.float32, 1), _tensor((8, K), torch.float32, 2)
    w = torch.ones(T, k, device=DEV)
    guard = torch.full((24, K), 5.0, device=DEV)
    for call in [lambda: B.moe_sort_tokens(x, f2p, k, rows=guard[8:16]),
                 lambda: B.moe_unsort_tokens_backward(x, f2p, k, topk_w=w, rows=rows, d_rows=guard[8:16])]:
        guard.fill_(5.0)
        out = call()
        assert B.nvfp4moe_last_device_status() == -1
        assert torch.equal(guard[9], x[0]) and torch.equal(guard[14], x[3])
        assert (guard[:8] == 5).all() and (guard[16:] == 5).all()
        assert (guard[11] == 5).all() and (guard[15] == 5).all()
        if isinstance(out, tuple):
            assert out[1][1, 1] == 0 and out[1][3, 1] == 0
    y = B.moe_unsort_tokens(rows, f2p, k)
    assert B.nvfp4moe_last_device_status() == -1
    assert torch.equal(y[1], rows[2]) and torch.equal(y[3], rows[6])
    assert B.nvfp4moe_last_device_status() == 0


def test_sorted_rows_follow_the_permutation():
    """With moe_permute's arrays, row r holds the token of slot perm_to_flat[r],
    and the sum over the experts undoes the sort."""
    T, k, E, K = 300, 4, 16, 264
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, generator=torch.Generator().manual_seed(1)).to(DEV)
    off, p2f, f2p = B.moe_permute(ids, E)
    x = _tensor((T, K), torch.bfloat16, 3)
    rows = B.moe_sort_tokens(x, f2p, k)
    assert torch.equal(rows, x[p2f.long() // k])
    quarter = torch.full((T, k), 0.25, device=DEV)
    assert torch.equal(B.moe_unsort_tokens(rows, f2p, k, topk_w=quarter), x)


def test_moe_combine_gives_the_same_bits():
    """The BF16 weighted sum is the one that moe_forward's last stage computes."""
    T, k, K = 200, 8, 1024
    f2p = _place(T, k, T * k, 0.0, 8).to(DEV)
    rows, w = _tensor((T * k, K), torch.bfloat16, 9), _weights(T, k, 10).to(DEV)
    assert torch.equal(B.moe_unsort_tokens(rows, f2p, k, topk_w=w), B.moe_combine(rows, w, f2p))


def test_empty_batches_and_infinities():
    x = torch.empty((0, 16), dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    assert B.moe_sort_tokens(x, none, 2).shape == (0, 16)
    assert B.moe_unsort_tokens(x, none, 2).shape == (0, 16)
    # a row that a dropped slot does not name does not reach the sum
    rows = torch.full((2, 16), float("nan"), device=DEV)
    rows[1] = 2.0
    f2p = torch.tensor([-1, 1], dtype=torch.int32, device=DEV)
    w = torch.tensor([[float("inf"), 0.5]], device=DEV)
    assert (B.moe_unsort_tokens(rows, f2p, 2, topk_w=w) == 1.0).all()
    d_rows, d_w = B.moe_unsort_tokens_backward(torch.ones((1, 16), device=DEV), f2p, 2, topk_w=w, rows=rows)
    assert d_w.tolist() == [[0.0, 32.0]] and (d_rows[1] == 0.5).all()


def test_graph_capture_and_another_stream():
    T, k, K = 50, 4, 520
    f2p = _place(T, k, T * k, 0.0, 11).to(DEV)
    w, x = _weights(T, k, 12).to(DEV), _tensor((T, K), torch.float16, 13)
    want = B.moe_sort_tokens(x, f2p, k, topk_w=w)
    back, d_w = B.moe_sort_tokens_backward(want, f2p, k, topk_w=w, x=x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(B.moe_sort_tokens(x, f2p, k, topk_w=w), want)
    side.synchronize()
    rows, out = torch.zeros_like(want), torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_sort_tokens(x, f2p, k, topk_w=w, rows=rows)
        _, d_g = B.moe_sort_tokens_backward(rows, f2p, k, topk_w=w, x=x, dx=out)
    for _ in range(2):
        rows.zero_()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(rows, want) and torch.equal(out, back) and torch.equal(d_g, d_w)


def test_refusals():
    x = torch.zeros((4, 16), device=DEV)
    f2p = torch.arange(8, dtype=torch.int32, device=DEV)
    w = torch.ones((4, 2), device=DEV)
    for bad in [lambda: B.moe_sort_tokens(x.cpu(), f2p, 2), lambda: B.moe_sort_tokens(x.double(), f2p, 2),
                lambda: B.moe_sort_tokens(x, f2p.long(), 2), lambda: B.moe_sort_tokens(x, f2p, 3),
                lambda: B.moe_sort_tokens(x.t(), f2p, 2), lambda: B.moe_sort_tokens(x, f2p, 2, topk_w=w.half()),
                lambda: B.moe_sort_tokens(x, f2p, 2, topk_w=w[:3]), lambda: B.moe_sort_tokens(x[0], f2p, 2),
                lambda: B.moe_sort_tokens(x, f2p, 2, rows=torch.zeros((8, 15), device=DEV)),
                lambda: B.moe_sort_tokens(x.expand(4, 16)[:1].expand(4, 16), f2p, 2),
                lambda: B.moe_sort_tokens_backward(torch.zeros((8, 16), device=DEV), f2p, 2, x=x),
                lambda: B.moe_unsort_tokens_backward(x, f2p, 2, topk_w=w, rows=torch.zeros((8, 15), device=DEV)),
                lambda: B.moe_unsort_tokens(x, torch.arange(34, dtype=torch.int32, device=DEV), 17)]:
        with pytest.raises(B.NVFP4Error):
            bad()
