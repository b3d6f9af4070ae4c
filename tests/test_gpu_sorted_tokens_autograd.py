"""moe_sort_tokens and moe_unsort_tokens of tensors that require gradients."""
import pytest
import torch

from nvfp4_block_scaled_05_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
U32 = 2.0 ** -24


def _case(T, k, K, extra, dropped, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    place = torch.randperm(T * k + extra, generator=g)[:T * k].int()
    place[torch.rand(T * k, generator=g) < dropped] = -1
    x = torch.randn(T, K, generator=g).to(dtype).to(DEV)
    rows = torch.randn(T * k + extra, K, generator=g).to(dtype).to(DEV)
    w = torch.rand(T, k, generator=g).to(DEV)
    return x, rows, w, place.to(DEV)


def _near(got, want, size, dtype, steps):
    """Within `steps` f32 roundings of the summed magnitudes and one to the type."""
    lim = steps * U32 * size + torch.finfo(dtype).eps / 2 * (want.abs() + steps * U32 * size) + 2.0 ** -24
    assert got.dtype == dtype and ((got.double() - want).abs() <= lim).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,K,extra,dropped", [(1, 1, 8, 0, 0.0), (33, 4, 101, 0, 0.0), (40, 3, 64, 17, 0.3),
                                                 (5, 2, 16, 0, 1.0)])
def test_gradients(T, k, K, extra, dropped, dtype):
    x, rows, w, f2p = _case(T, k, K, extra, dropped, dtype)
    live = (f2p >= 0)
    at = f2p.long()[live]
    token = torch.arange(T * k, device=DEV)[live] // k

    # rows[at] = w x[token]; a loss that reads the named rows only
    xs, ws = x.clone().requires_grad_(), w.clone().requires_grad_()
    out = B.moe_sort_tokens(xs, f2p, k, topk_w=ws, n_rows=T * k + extra)
    assert out.requires_grad
    (out[at].float() * rows[at].float()).sum().backward()
    xd, wd, rd = x.double(), w.double().view(-1)[live, None], rows.double()[at]
    dx = torch.zeros_like(xd).index_add_(0, token, wd * rd)
    size = torch.zeros_like(xd).index_add_(0, token, (wd * rd).abs())
    dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    dw[live] = (rd * xd[token]).sum(1)
    dsize = torch.zeros_like(dw)
    dsize[live] = (rd * xd[token]).abs().sum(1)
    _near(xs.grad, dx, size, dtype, k)
    assert ws.grad.shape == (T, k)
    _near(ws.grad.view(-1), dw, dsize, torch.float32, K)

    # y[token] += w rows[at]; the gradient of rows that no slot names is zero
    rs, ws = rows.clone().requires_grad_(), w.clone().requires_grad_()
    y = B.moe_unsort_tokens(rs, f2p, k, topk_w=ws)
    (y.float() * x.float()).sum().backward()
    d_rows = torch.zeros_like(rows, dtype=torch.float64)
    d_rows[at] = wd * xd[token]
    _near(rs.grad, d_rows, d_rows.abs(), dtype, 1)
    _near(ws.grad.view(-1), dw, dsize, torch.float32, K)
    assert B.nvfp4moe_last_device_status() == 0


def test_one_of_the_inputs_and_no_weights():
    T, k, K = 20, 2, 24
    x, rows, w, f2p = _case(T, k, K, 0, 0.0, torch.float32)
    xs = x.clone().requires_grad_()
    B.moe_sort_tokens(xs, f2p, k).sum().backward()           # an expanded gradient
    assert (xs.grad == k).all()
    rs = rows.clone().requires_grad_()
    B.moe_unsort_tokens(rs, f2p, k).sum().backward()
    assert (rs.grad == 1).all()
    ws = w.view(-1).clone().requires_grad_()                 # flat weights, flat gradient
    B.moe_sort_tokens(x, f2p, k, topk_w=ws).sum().backward()
    assert ws.grad.shape == (T * k,)
    lim = K * U32 * x.abs().sum(1).double() + 2.0 ** -24
    assert ((ws.grad.view(T, k).double() - x.double().sum(1, keepdim=True)).abs() <= 2 * lim[:, None]).all()
    ws = w.clone().requires_grad_()
    B.moe_unsort_tokens(rows, f2p, k, topk_w=ws).sum().backward()
    want, size = rows.double()[f2p.long()].view(T, k, K).sum(-1), rows.double().abs()[f2p.long()].view(T, k, K).sum(-1)
    assert ((ws.grad.double() - want).abs() <= 2 * K * U32 * size).all()


def test_values_are_those_without_gradients():
    T, k, K = 64, 4, 256
    x, rows, w, f2p = _case(T, k, K, 0, 0.0, torch.bfloat16)
    want, y = B.moe_sort_tokens(x, f2p, k, topk_w=w), B.moe_unsort_tokens(rows, f2p, k, topk_w=w)
    assert not want.requires_grad
    xs, rs = x.clone().requires_grad_(), rows.clone().requires_grad_()
    assert torch.equal(B.moe_sort_tokens(xs, f2p, k, topk_w=w), want)
    assert torch.equal(B.moe_unsort_tokens(rs, f2p, k, topk_w=w), y)
    with torch.no_grad():
        out = B.moe_sort_tokens(xs, f2p, k, topk_w=w)
    assert torch.equal(out, want) and not out.requires_grad


def test_given_outputs():
    T, k, K = 6, 2, 16
    x, rows, w, f2p = _case(T, k, K, 0, 0.0, torch.float32)
    xs, buf = x.clone().requires_grad_(), torch.zeros_like(rows)
    out = B.moe_sort_tokens(xs, f2p, k, rows=buf)
    assert out.data_ptr() == buf.data_ptr() and buf.requires_grad
    (buf * rows).sum().backward()
    want = rows.double()[f2p.long()].view(T, k, K).sum(1)
    assert ((xs.grad.double() - want).abs() <= k * 2 * U32 * rows.abs().max() * k).all()
    rs, y = rows.clone().requires_grad_(), torch.zeros_like(x)
    B.moe_unsort_tokens(rs, f2p, k, y=y)
    y.sum().backward()
    assert (rs.grad == 1).all()
    with pytest.raises(B.NVFP4Error):                        # an output that has gradients of its own
        B.moe_sort_tokens(xs, f2p, k, rows=torch.zeros_like(rows).requires_grad_() * 1)


def test_double_backward_is_refused():
    x, rows, w, f2p = _case(4, 2, 8, 0, 0.0, torch.float32)
    xs = x.clone().requires_grad_()
    (g,) = torch.autograd.grad((B.moe_sort_tokens(xs, f2p, 2) ** 2).sum(), xs, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_another_stream():
    x, rows, w, f2p = _case(300, 4, 512, 0, 0.0, torch.bfloat16)
    xs = x.clone().requires_grad_()
    B.moe_sort_tokens(xs, f2p, 4, topk_w=w).backward(rows)
    want, xs.grad = xs.grad, None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out = B.moe_sort_tokens(xs, f2p, 4, topk_w=w)
    torch.cuda.current_stream().wait_stream(side)
    out.backward(rows)
    torch.cuda.synchronize()
    assert torch.equal(xs.grad, want)


def test_forward_and_backward_in_a_graph():
    T, k, K = 50, 4, 128
    x, rows, w, f2p = _case(T, k, K, 10, 0.1, torch.bfloat16)
    xs, ws = x.clone().requires_grad_(), w.clone().requires_grad_()

    def step():
        out = B.moe_unsort_tokens(B.moe_sort_tokens(xs, f2p, k, topk_w=ws, n_rows=T * k + 10), f2p, k, topk_w=ws)
        return torch.autograd.grad(out, (xs, ws), x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert B.nvfp4moe_last_device_status() == 0
