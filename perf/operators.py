"""Measured cases of the 8-bit expert operators and of the sorted-token operators.

Operators (entry points of nvfp4_block_scaled_05_gb300.binding):

* block quantization to E4M3: fp8_quantize (rows, one scale per 128 elements,
  optionally written straight into expert order), fp8_quantize_weight (one
  scale per 128 x 128 block) and fp8_swiglu_quantize (silu(gate) * up);
* the matrix product of such operands: fp8_linear (one group) and
  fp8_grouped_gemm (one group per expert);
* tokens sorted by expert and back: moe_sort_tokens, moe_unsort_tokens and
  their gradients.

Block rule: s = amax / 448, code = E4M3(x * (448 / amax)), every step one f32
operation; a block whose amax is below 2^-100 has scale 0 and codes 0.
"""
import math

import torch

own = False

BLOCK = 128
TINY = 2.0 ** -100
F8 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the activations of a prefill step, quantized once and written to the k experts of each token
        {"name": "quantize_sorted_prefill", "op": "quantize", "T": 8192, "K": 7168, "k": 8, "E": 256, "dtype": "bf16"},
        # a checkpoint's expert weights (gate and up rows of eight experts), quantized when they are loaded
        {"name": "quantize_weights", "op": "weight", "E": 8, "N": 4096, "K": 7168, "dtype": "bf16"},
        # the gate and up products of a prefill step of 2048 tokens, on their way to the down projection
        {"name": "swiglu_prefill", "op": "swiglu", "M": 16384, "I": 2048, "dtype": "bf16"},
        # a projection for one new token: the weights are read once, latency counts
        {"name": "linear_one_token", "op": "linear", "M": 1, "N": 4096, "K": 7168, "out": "bf16"},
        # sizes that fit no tile, with an f32 result (a router's or an output head's logits)
        {"name": "linear_ragged", "op": "linear", "M": 333, "N": 1111, "K": 2000, "out": "f32"},
        # the shared expert's product over a prefill step
        {"name": "linear_prefill", "op": "linear", "M": 4096, "N": 4096, "K": 7168, "out": "bf16"},
        # the gate and up product of a decode step: a few rows for each of 256 experts
        {"name": "grouped_decode", "op": "grouped", "T": 128, "k": 8, "E": 256, "N": 4096, "K": 7168,
         "routing": "uniform", "out": "bf16"},
        # the down product of a prefill step whose experts are unequally popular, some of them without a row
        {"name": "grouped_skewed", "op": "grouped", "T": 8192, "k": 8, "E": 32, "N": 7168, "K": 2048,
         "routing": "zipf", "out": "bf16"},
        # a training step's dispatch: rows in expert order, and the gradient back to the tokens
        {"name": "sort_prefill", "op": "sort", "T": 8192, "K": 7168, "k": 8, "E": 256, "dtype": "bf16",
         "weighted": False},
        # a small batch of a narrow f32 layer with the weights applied before the experts, odd width
        {"name": "sort_small", "op": "sort", "T": 77, "K": 1001, "k": 4, "E": 16, "dtype": "f32", "weighted": True},
        # a training step's weighted sum over the experts, and the gradients of rows and weights
        {"name": "unsort_prefill", "op": "unsort", "T": 8192, "K": 7168, "k": 8, "E": 256, "dtype": "bf16",
         "weighted": True},
        # the same for a decode-sized batch in f16
        {"name": "unsort_decode", "op": "unsort", "T": 32, "K": 7168, "k": 8, "E": 256, "dtype": "f16",
         "weighted": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "weight", "swiglu", "linear", "linear", "grouped", "grouped", "sort", "unsort"])
    k = rng.choice([1, 2, 4, 6, 8])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "quantize":
        return {"op": op, "T": _log(rng, 1, 8192), "K": 16 * _log(rng, 8, 448), "k": k, "E": rng.randint(8, 256),
                "dtype": dtype}
    if op == "weight":
        return {"op": op, "E": rng.randint(1, 8), "N": _log(rng, 64, 4096), "K": 16 * _log(rng, 8, 448),
                "dtype": dtype}
    if op == "swiglu":
        return {"op": op, "M": _log(rng, 1, 16384), "I": 16 * _log(rng, 8, 128), "dtype": dtype}
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 64, 4096), "K": 16 * _log(rng, 8, 448),
                "out": rng.choice(["bf16", "bf16", "f32"])}
    if op == "grouped":
        routing = rng.choice(["uniform", "zipf"])
        return {"op": op, "T": _log(rng, 1, 8192 if routing == "uniform" else 4096), "k": k,
                "E": rng.randint(8, 64 if routing == "uniform" else 32), "N": _log(rng, 128, 4096),
                "K": 16 * _log(rng, 8, 256), "routing": routing, "out": rng.choice(["bf16", "bf16", "f32"])}
    return {"op": op, "T": _log(rng, 1, 8192), "K": _log(rng, 64, 7168 if dtype != "f32" else 3500), "k": k,
            "E": rng.randint(8, 256), "dtype": dtype, "weighted": rng.random() < 0.5}


def work(c):
    op = c["op"]
    if op == "quantize":
        T, K, k = c["T"], c["K"], c["k"]
        out = T * k * (K + 4 * _blocks(K))
        return {"bytes": T * K * SIZE[c["dtype"]] + T * k * 4 + out, "flops": 3 * T * K}
    if op == "weight":
        E, N, K = c["E"], c["N"], c["K"]
        return {"bytes": E * N * K * (SIZE[c["dtype"]] + 1) + 4 * E * _blocks(N) * _blocks(K), "flops": 3 * E * N * K}
    if op == "swiglu":
        M, I = c["M"], c["I"]
        return {"bytes": 2 * M * I * SIZE[c["dtype"]] + M * (I + 4 * _blocks(I)), "flops": 8 * M * I}
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        sf = 4 * _blocks(K) * (M + _blocks(N))
        return {"bytes": (M + N) * K + sf + M * N * SIZE[c["out"]], "flops": 2 * M * N * K}
    if op == "grouped":
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        M = T * k
        # experts with at least one row (all but the dead ones where popularity is skewed)
        live = E * (1.0 - (1.0 - k / E) ** T) if c["routing"] == "uniform" else min(M, E - _dead(E))
        sf = 4 * _blocks(K) * (M + live * _blocks(N))
        return {"bytes": M * K + live * N * K + sf + M * N * SIZE[c["out"]], "flops": 2 * M * N * K}
    # sort: read x, write rows; then read d_rows (and x again for the weights' gradient), write dx
    # unsort: read rows, write y; then read dy (and rows again for the weights' gradient), write d_rows
    T, K, k, s = c["T"], c["K"], c["k"], SIZE[c["dtype"]]
    once, full = T * K * s, T * k * K * s
    if op == "sort":
        n = once + full + full + once + (once if c["weighted"] else 0)
    else:
        n = full + once + once + full + (full if c["weighted"] else 0)
    return {"bytes": n + 2 * 4 * T * k + (3 * 4 * T * k if c["weighted"] else 0),
            "flops": (6 if c["weighted"] else 2) * T * k * K}


# ------------------------------------------------------------------ inputs

def _blocks(n):
    return -(-n // BLOCK)


def _dead(E):
    return E // 16


def _gen(seed, part):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 7919 * part + 17)
    return g


def _randn(shape, seed, part, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=_gen(seed, part), device="cuda") * scale).to(dtype)


def _activations(shape, seed, part, dtype):
    """N(0, 1) with a few columns far larger than the others and a few blocks of zeros."""
    x = torch.randn(shape, generator=_gen(seed, part), device="cuda")
    K = shape[-1]
    wide = torch.randint(0, K, (max(1, K // 500),), generator=_gen(seed, part + 1), device="cuda")
    x[..., wide] *= 30.0
    full = K // BLOCK
    if full:
        zero = torch.rand(x.shape[0], full, generator=_gen(seed, part + 2), device="cuda") < 0.01
        x[:, :full * BLOCK].view(x.shape[0], full, BLOCK).masked_fill_(zero[..., None], 0.0)
    return x.to(dtype)


def _routing(T, k, E, seed, routing):
    """Experts and weights of each token, and the expert order of the T * k slots."""
    logits = torch.randn((T, E), generator=_gen(seed, 40), device="cuda")
    if routing == "zipf":
        rank = torch.randperm(E, generator=_gen(seed, 41), device="cuda")
        p = 1.0 / (1.0 + rank.double()) ** 1.2
        u = torch.rand((T, E), generator=_gen(seed, 42), device="cuda", dtype=torch.float64).clamp(1e-12, 1 - 1e-12)
        logits = (p.log() - torch.log(-torch.log(u))).float()
        logits[:, rank < _dead(E)] = -math.inf
    k = min(k, E)
    top = torch.topk(logits, k, dim=1)
    w = torch.softmax(top.values, dim=1)
    ids = top.indices.to(torch.int32)
    order = torch.sort(ids.reshape(-1), stable=True).indices
    f2p = torch.empty_like(order)
    f2p[order] = torch.arange(order.numel(), device="cuda")
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return {"w": w.contiguous(), "perm_to_flat": order.to(torch.int32), "flat_to_perm": f2p.to(torch.int32),
            "offsets": offsets, "most": int(counts.max())}


def _codes_of_rows(shape, seed, part):
    codes, sf = _quantize_rows(_activations(shape, seed, part, torch.bfloat16))
    return codes.contiguous(), sf.contiguous()


def _codes_of_weights(E, N, K, seed, part):
    codes = torch.empty((E, N, K), dtype=torch.uint8, device="cuda")
    sf = torch.empty((E, _blocks(N), _blocks(K)), device="cuda")
    for e in range(E):
        c, s = _quantize_blocks(_randn((1, N, K), seed * 521 + e, part, scale=0.02))
        codes[e], sf[e] = c[0], s[0]
    return codes, sf


def prepare(c, seed):
    op = c["op"]
    if op == "quantize":
        s = {"c": c, "x": _activations((c["T"], c["K"]), seed, 1, TYPES[c["dtype"]])}
        if c["k"] > 1:
            s.update(_routing(c["T"], c["k"], c["E"], seed, "uniform"))
        return s
    if op == "weight":
        return {"c": c, "w": _randn((c["E"], c["N"], c["K"]), seed, 2, TYPES[c["dtype"]], 0.02)}
    if op == "swiglu":
        return {"c": c, "gu": _randn((c["M"], 2 * c["I"]), seed, 3, TYPES[c["dtype"]], 1.7)}
    if op == "linear":
        a_codes, a_sf = _codes_of_rows((c["M"], c["K"]), seed, 4)
        w_codes, w_sf = _codes_of_weights(1, c["N"], c["K"], seed, 8)
        return {"c": c, "a_codes": a_codes, "a_sf": a_sf, "w_codes": w_codes[0], "w_sf": w_sf[0]}
    if op == "grouped":
        s = {"c": c}
        s.update(_routing(c["T"], c["k"], c["E"], seed, c["routing"]))
        s["a_codes"], s["a_sf"] = _codes_of_rows((s["flat_to_perm"].numel(), c["K"]), seed, 4)
        s["w_codes"], s["w_sf"] = _codes_of_weights(c["E"], c["N"], c["K"], seed, 8)
        return s
    s = {"c": c}
    s.update(_routing(c["T"], c["k"], c["E"], seed, "uniform"))
    T, K, R, t = c["T"], c["K"], s["flat_to_perm"].numel(), TYPES[c["dtype"]]
    if op == "sort":
        s["x"] = _activations((T, K), seed, 1, t)
        s["d_rows"] = _randn((R, K), seed, 5, t, 0.01)
    else:
        s["rows"] = _activations((R, K), seed, 1, t)
        s["dy"] = _randn((T, K), seed, 5, t, 0.01)
    return s


# ------------------------------------------------------------------ plain forms

def _padded(x, *sides):
    """Zeros after the last columns (and rows), up to whole blocks."""
    pad = []
    for d in sides:
        pad += [0, -x.shape[d] % BLOCK]
    return torch.nn.functional.pad(x, pad) if any(pad) else x


def _codes(x, amax):
    """x in blocks and each block's amax -> codes and scales."""
    live, top = amax >= TINY, amax.new_full((), 448.0)   # a tensor, so that the quotients are true divisions
    inv = torch.where(live, top / amax.clamp_min(TINY), 0.0)
    sf = torch.where(live, amax / top, 0.0)
    return (x * inv).clamp(-448.0, 448.0).to(F8).view(torch.uint8), sf


def _quantize_rows(x):
    M, K = x.shape
    b = _padded(x.float(), -1).view(M, -1, BLOCK)
    codes, sf = _codes(b, b.abs().amax(-1, keepdim=True))
    return codes.view(M, -1)[:, :K], sf[..., 0]


def _quantize_blocks(w):
    E, N, K = w.shape
    b = _padded(w.float(), -1, -2)
    b = b.view(E, _blocks(N), BLOCK, _blocks(K), BLOCK)
    codes, sf = _codes(b, b.abs().amax((2, 4), keepdim=True))
    return codes.view(E, _blocks(N) * BLOCK, -1)[:, :N, :K], sf[:, :, 0, :, 0]


def _values_of_rows(codes, sf, dtype=torch.float32):
    M, K = codes.shape
    v = _padded(codes, -1).view(F8).to(dtype).view(M, -1, BLOCK)
    return v.mul_(sf.to(dtype)[..., None]).view(M, -1)[:, :K]


def _values_of_weights(codes, sf, dtype=torch.float32):
    E, N, K = codes.shape
    v = _padded(codes, -1, -2).view(F8).to(dtype).view(E, _blocks(N), BLOCK, _blocks(K), BLOCK)
    return v.mul_(sf.to(dtype)[:, :, None, :, None]).view(E, _blocks(N) * BLOCK, -1)[:, :N, :K]


def _plain_grouped(s):
    """Groups padded to the largest, one batched product, the rows taken back."""
    off, most = s["offsets"].long(), s["most"]
    a = _values_of_rows(s["a_codes"], s["a_sf"])
    M = a.shape[0]
    at = (off[:-1, None] + torch.arange(most, device=a.device)).clamp_max(M - 1)
    w = _values_of_weights(s["w_codes"], s["w_sf"])
    out = torch.bmm(a[at], w.transpose(1, 2))
    r = torch.arange(M, device=a.device)
    e = torch.searchsorted(off[1:], r, right=True)
    return out[e, r - off[e]].to(TYPES[s["c"]["out"]])


def _plain_sort(s):
    c = s["c"]
    T, K, k = c["T"], c["K"], s["w"].shape[1]
    slot, place, t = s["perm_to_flat"].long(), s["flat_to_perm"].long(), TYPES[c["dtype"]]
    x, d = s["x"].float(), s["d_rows"].float()
    rows, back = x[slot // k], d[place].view(T, k, K)
    if not c["weighted"]:
        return {"rows": rows.to(t), "dx": back.sum(1).to(t)}
    return {"rows": (rows * s["w"].view(-1)[slot, None]).to(t), "dx": (back * s["w"][..., None]).sum(1).to(t),
            "d_w": (back * x[:, None, :]).sum(-1)}


def _plain_unsort(s):
    c = s["c"]
    T, K, k = c["T"], c["K"], s["w"].shape[1]
    slot, place, t = s["perm_to_flat"].long(), s["flat_to_perm"].long(), TYPES[c["dtype"]]
    dy, rows = s["dy"].float(), s["rows"].float()
    per, d = rows[place].view(T, k, K), dy[slot // k]
    if not c["weighted"]:
        return {"y": per.sum(1).to(t), "d_rows": d.to(t)}
    return {"y": (per * s["w"][..., None]).sum(1).to(t), "d_rows": (d * s["w"].view(-1)[slot, None]).to(t),
            "d_w": (per * dy[:, None, :]).sum(-1)}


def _plain(s):
    c = s["c"]
    op = c["op"]
    if op == "quantize":
        codes, sf = _quantize_rows(s["x"])
        if c["k"] > 1:
            token = s["perm_to_flat"].long() // s["w"].shape[1]
            codes, sf = codes[token], sf[token]
        return codes.contiguous().view(F8), sf
    if op == "weight":
        codes, sf = _quantize_blocks(s["w"])
        return codes.contiguous().view(F8), sf
    if op == "swiglu":
        g, u = s["gu"].float().chunk(2, dim=1)
        codes, sf = _quantize_rows(g / (1.0 + torch.exp(-g)) * u)
        return codes.contiguous().view(F8), sf
    if op == "linear":
        a = _values_of_rows(s["a_codes"], s["a_sf"])
        w = _values_of_weights(s["w_codes"][None], s["w_sf"][None])[0]
        return (a @ w.t()).to(TYPES[c["out"]])
    if op == "grouped":
        return _plain_grouped(s)
    return _plain_sort(s) if op == "sort" else _plain_unsort(s)


def run(s):
    if not own:
        return _plain(s)
    from nvfp4_block_scaled_05_gb300 import binding as B
    c = s["c"]
    op = c["op"]
    if op == "quantize":
        if c["k"] > 1:
            codes, sf = B.fp8_quantize(s["x"], flat_to_perm=s["flat_to_perm"], k=s["w"].shape[1])
        else:
            codes, sf = B.fp8_quantize(s["x"])
        return codes.view(F8), sf
    if op == "weight":
        codes, sf = B.fp8_quantize_weight(s["w"])
        return codes.view(F8), sf
    if op == "swiglu":
        codes, sf = B.fp8_swiglu_quantize(s["gu"])
        return codes.view(F8), sf
    if op == "linear":
        return B.fp8_linear(s["a_codes"], s["a_sf"], s["w_codes"], s["w_sf"], out_dtype=TYPES[c["out"]])
    if op == "grouped":
        return B.fp8_grouped_gemm(s["a_codes"], s["a_sf"], s["w_codes"], s["w_sf"], s["offsets"],
                                  out_dtype=TYPES[c["out"]])
    k, w, f2p = s["w"].shape[1], s["w"] if c["weighted"] else None, s["flat_to_perm"]
    if op == "sort":
        rows = B.moe_sort_tokens(s["x"], f2p, k, topk_w=w)
        dx, d_w = B.moe_sort_tokens_backward(s["d_rows"], f2p, k, topk_w=w, x=s["x"] if c["weighted"] else None)
        out = {"rows": rows, "dx": dx}
    else:
        y = B.moe_unsort_tokens(s["rows"], f2p, k, topk_w=w)
        d_rows, d_w = B.moe_unsort_tokens_backward(s["dy"], f2p, k, topk_w=w,
                                                   rows=s["rows"] if c["weighted"] else None)
        out = {"y": y, "d_rows": d_rows}
    if c["weighted"]:
        out["d_w"] = d_w
    return out


# ------------------------------------------------------------------ 64 bits

def _round_e4m3(q):
    """The nearest E4M3 value of each 64-bit number, ties to the even one, at most 448."""
    mag = q.abs().clamp_max(448.0)
    step = torch.exp2(torch.floor(torch.log2(mag.clamp_min(2.0 ** -6))) - 3)
    return torch.copysign(torch.round(mag / step) * step, q)


def _exact_blocks(x, dims):
    """The E4M3 values and scales of 64-bit numbers in blocks that span `dims`."""
    amax = x.abs().amax(dims, keepdim=True)
    live = amax >= TINY
    q = torch.where(live, x * (448.0 / amax.clamp_min(TINY)), 0.0)
    return _round_e4m3(q), torch.where(live, amax / 448.0, 0.0)


def _exact_rows(x):
    codes, sf = [], []
    for p in x.split(2048):
        b = _padded(p, -1)
        v, f = _exact_blocks(b.view(b.shape[0], -1, BLOCK), -1)
        codes.append(v.view(b.shape[0], -1)[:, :x.shape[1]].float())
        sf.append(f[..., 0])
    return torch.cat(codes), torch.cat(sf)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op in ("quantize", "swiglu"):
        if op == "quantize":
            codes, sf = _exact_rows(s["x"].double())
            if c["k"] > 1:
                token = s["perm_to_flat"].long() // s["w"].shape[1]
                codes, sf = codes[token], sf[token]
            return codes.double(), sf
        h = []
        for p in s["gu"].split(2048):
            g, u = p.double()[:, :c["I"]], p.double()[:, c["I"]:]
            h.append(g * torch.sigmoid(g) * u)
        codes, sf = _exact_rows(torch.cat(h))
        return codes.double(), sf
    if op == "weight":
        codes, sf = [], []
        for w in s["w"]:
            b = _padded(w.double(), -1, -2)
            n, k = b.shape
            v, f = _exact_blocks(b.view(n // BLOCK, BLOCK, k // BLOCK, BLOCK), (1, 3))
            codes.append(v.reshape(n, k)[:c["N"], :c["K"]])
            sf.append(f[:, 0, :, 0])
        return torch.stack(codes), torch.stack(sf)
    if op == "linear":
        a = _values_of_rows(s["a_codes"], s["a_sf"], torch.float64)
        return a @ _values_of_weights(s["w_codes"][None], s["w_sf"][None], torch.float64)[0].t()
    if op == "grouped":
        off = s["offsets"].tolist()
        out = []
        for e in range(c["E"]):
            lo, hi = off[e], off[e + 1]
            if hi > lo:
                a = _values_of_rows(s["a_codes"][lo:hi], s["a_sf"][lo:hi], torch.float64)
                out.append(a @ _values_of_weights(s["w_codes"][e:e + 1], s["w_sf"][e:e + 1], torch.float64)[0].t())
        return torch.cat(out)
    T, K, k = c["T"], c["K"], s["w"].shape[1]
    place, w = s["flat_to_perm"].long().view(T, k), s["w"].double()
    scale = w if c["weighted"] else torch.ones_like(w)
    token, rows = (s["x"], s["d_rows"]) if op == "sort" else (s["dy"], s["rows"])
    spread = torch.empty((T * k, K), dtype=torch.float64, device="cuda")
    sums, dots = [], []
    for lo in range(0, T, 512):
        p, x, v = place[lo:lo + 512], token[lo:lo + 512].double(), scale[lo:lo + 512]
        r = rows[p.reshape(-1)].double().view(p.shape[0], k, K)
        spread[p.reshape(-1)] = (x[:, None, :] * v[..., None]).reshape(-1, K)
        sums.append(torch.einsum("tk,tkc->tc", v, r))
        dots.append(torch.einsum("tkc,tc->tk", r, x))
    out = dict(zip(("rows", "dx") if op == "sort" else ("d_rows", "y"), (spread, torch.cat(sums))))
    if c["weighted"]:
        out["d_w"] = torch.cat(dots)
    return out
