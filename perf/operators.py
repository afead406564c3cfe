"""What is measured of the layer's 8-bit floating point operators.

The operators (e4m3 values, one fp32 scale for each block of 128):
  rows     rows of activations -> e4m3 with a scale for each 128 columns of a row
  permute  the same for token rows, each written to the bucket rows of its kept picks
  weights  expert weights -> e4m3 with a scale for each 128 x 128 block
  gemm     products of ragged expert buckets with their expert's weight, both in that form
  ffn      the SwiGLU expert FFN on such products, its hidden rows quantised in between

Quantisation of a block with largest magnitude m (at least 2^-100): scale = m / 448 in fp32,
q = the e4m3 number nearest to 448 x / m, the quotient taken exactly, ties to even.

A case's routing is drawn at random: each token picks k different experts, expert ranks
weighted by (rank + 1)^-skew; a share `drop` of the picks gets no row (capacity).
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100


def listed():
    return [
        # one token of a decode step, before the experts of the Mixtral-8x7B shaped layer
        dict(name="permute_T1_d4096", op="permute", T=1, k=2, E=8, d=4096, drop=0.0, skew=0.0,
             dtype="bf16"),
        # the DeepSeek-shaped prefill batch, a tenth of its picks over capacity
        dict(name="permute_T16384_d7168", op="permute", T=16384, k=8, E=256, d=7168, drop=0.1,
             skew=0.1, dtype="bf16"),
        # rows in fp32, odd count, the last block of 128 columns partly filled
        dict(name="rows_fp32_1111x1520", op="rows", rows=1111, d=1520, dtype="f32"),
        # the gate weights of the Mixtral-8x7B shaped layer, quantised once at load
        dict(name="weights_E8_14336x4096", op="weights", E=8, n=14336, d=4096, dtype="bf16"),
        # fp32 master weights with partly filled blocks on both axes
        dict(name="weights_fp32_E3_1000x1520", op="weights", E=3, n=1000, d=1520, dtype="f32"),
        # one dense product: a shared expert's projection over a prefill batch
        dict(name="gemm_dense_4096x4096x7168", op="gemm", T=4096, k=1, E=1, d=7168, n=4096,
             skew=0.0),
        # ragged buckets, some of them empty, no size a multiple of a tile
        dict(name="gemm_E13_odd", op="gemm", T=1501, k=2, E=13, d=1520, n=1000, skew=3.0),
        # down projection of 32 experts of one rank in a decode step
        dict(name="gemm_E32_decode", op="gemm", T=16, k=8, E=32, d=2048, n=7168, skew=0.0),
        # a single token through the Mixtral-8x7B shaped experts
        dict(name="ffn_mixtral8x7b_T1", op="ffn", T=1, k=2, E=8, d=4096, f=14336, skew=0.0),
        # the DeepSeek-shaped decode step
        dict(name="ffn_dsv3_T128", op="ffn", T=128, k=8, E=256, d=7168, f=2048, skew=0.0),
        # the Mixtral-8x7B shaped prefill
        dict(name="ffn_mixtral8x7b_T4096", op="ffn", T=4096, k=2, E=8, d=4096, f=14336, skew=0.1),
        # the DeepSeek-shaped prefill
        dict(name="ffn_dsv3_T16384", op="ffn", T=16384, k=8, E=256, d=7168, f=2048, skew=0.1),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], even over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["permute", "rows", "weights", "gemm", "gemm", "ffn", "ffn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = _spread(rng, 256, 7168, 16)
    E = _spread(rng, 1, 256)
    k = rng.randint(1, min(8, E))
    skew = rng.choice([0.0, 0.1, 1.0])
    if op == "rows":
        return dict(op=op, rows=_spread(rng, 1, 65536), d=d, dtype=dtype)
    if op == "permute":
        return dict(op=op, T=_spread(rng, 1, 16384), k=k, E=E, d=d, drop=rng.choice([0.0, 0.1]),
                    skew=skew, dtype=dtype)
    n = _spread(rng, 256, 14336, 16)
    E = _spread(rng, 1, max(1, min(256, int(1.5e9 / (d * n)))))
    k = rng.randint(1, min(8, E))
    if op == "weights":
        return dict(op=op, E=E, n=n, d=d, dtype=dtype)
    T = _spread(rng, 1, 8192)
    if E * T * (d + 2 * n) > 3e9:  # a few experts would hold most rows of a large batch
        skew = min(skew, 0.1)
    if op == "gemm":
        return dict(op=op, T=T, k=k, E=E, d=d, n=n, skew=skew)
    return dict(op=op, T=T, k=k, E=E, d=d, f=n, skew=skew)


# ------------------------------------------------------------------ plain arithmetic
def _blocks(d):
    return -(-d // BLOCK)


def _pad_last(x, d):
    """x with its last axis padded by zeros to whole blocks of 128."""
    return torch.nn.functional.pad(x, (0, _blocks(d) * BLOCK - d))


def _quantize_rows(x):
    """(q, scale) of rows of numbers: a scale for each 128 columns of a row.  Quotients of
    bf16 numbers often lie on the border of two e4m3 numbers, so they are taken in 64 bits."""
    d = x.shape[-1]
    b = _pad_last(x.float(), d).unflatten(-1, (_blocks(d), BLOCK))
    m = b.abs().amax(-1).clamp_min(AMAX_FLOOR)
    q = (b.double() * E4M3_MAX / m[..., None]).to(torch.float8_e4m3fn)
    return q.flatten(-2)[..., :d].contiguous(), m / E4M3_MAX


def _quantize_weights(w):
    """(q, scale) of [E, n, d] weights: a scale for each 128 x 128 block."""
    _, n, d = w.shape
    w = torch.nn.functional.pad(w.float(), (0, _blocks(d) * BLOCK - d, 0, _blocks(n) * BLOCK - n))
    b = w.unflatten(-1, (_blocks(d), BLOCK)).unflatten(1, (_blocks(n), BLOCK))
    m = b.abs().amax((2, 4)).clamp_min(AMAX_FLOOR)  # [E, nb, kb]
    q = (b.double() * E4M3_MAX / m[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.flatten(3).flatten(1, 2)[:, :n, :d].contiguous(), m / E4M3_MAX


def _rows_value(q, s, to=torch.float32):
    """The numbers that quantised rows stand for."""
    d = q.shape[-1]
    return q.to(to) * s.to(to).repeat_interleave(BLOCK, -1)[..., :d]


def _weights_value(q, s, to=torch.float32):
    """The numbers that quantised weights stand for."""
    _, n, d = q.shape
    out = q.to(to)
    s = s.to(to).repeat_interleave(BLOCK, 1)[:, :n]
    full = d // BLOCK * BLOCK
    out[..., :full].unflatten(-1, (-1, BLOCK)).mul_(s[..., :full // BLOCK, None])
    if full < d:
        out[..., full:].mul_(s[..., -1:])
    return out


def _bucket_rows(counts, offsets):
    """[E, M] row of each bucket slot (M the longest bucket), and which slots are rows."""
    slot = torch.arange(max(1, int(counts.max())), device=counts.device)
    there = slot[None, :] < counts[:, None]
    return torch.where(there, offsets[:-1, None] + slot, 0).long(), there


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _routing(case, g):
    """Bucket sizes and starts, and the bucket row of each kept pick (-1: dropped)."""
    T, k, E = case["T"], case["k"], case["E"]
    rank = torch.randperm(E, generator=g, device="cuda").float()
    noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda")
                                  .clamp(1e-7, 1 - 1e-7)))
    picks = (noise - case["skew"] * torch.log(rank + 1)).topk(k, dim=1).indices.flatten()
    drops = int(case.get("drop", 0.0) * T * k)
    kept = torch.ones(T * k, dtype=torch.bool, device="cuda")
    kept[torch.randperm(T * k, generator=g, device="cuda")[:drops]] = False
    group = torch.where(kept, picks, E)
    order = torch.sort(group, stable=True).indices
    counts = torch.bincount(group, minlength=E + 1)[:E].int()
    row = torch.empty(T * k, dtype=torch.int32, device="cuda")
    row[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    row = torch.where(kept, row, -1).int().view(T, k)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return counts, offsets, row


def _activations(rows, d, g, dtype):
    """Rows as a norm leaves them: unit scale, a few columns much larger than the rest."""
    gain = 1 + 9 * (torch.rand(d, generator=g, device="cuda") < 0.01)
    return (torch.randn((rows, d), generator=g, device="cuda") * gain).to(dtype)


def _weights(E, n, d, g):
    """Quantised weights of unit gain, an expert at a time."""
    q = torch.empty((E, n, d), dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty((E, _blocks(n), _blocks(d)), device="cuda")
    for e in range(E):
        w = torch.randn((1, n, d), generator=g, device="cuda") / math.sqrt(d)
        q[e:e + 1], s[e:e + 1] = _quantize_weights(w.bfloat16())
    return q, s


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "rows":
        s["x"] = _activations(case["rows"], case["d"], g, _dtype(case))
        s["q"] = torch.zeros((case["rows"], case["d"]), dtype=torch.float8_e4m3fn, device="cuda")
        s["s"] = torch.zeros((case["rows"], _blocks(case["d"])), device="cuda")
    elif op == "weights":
        E, n, d = case["E"], case["n"], case["d"]
        s["w"] = torch.empty((E, n, d), dtype=_dtype(case), device="cuda")
        for e in range(E):
            s["w"][e] = torch.randn((n, d), generator=g, device="cuda") / math.sqrt(d)
        s["q"] = torch.zeros((E, n, d), dtype=torch.float8_e4m3fn, device="cuda")
        s["s"] = torch.zeros((E, _blocks(n), _blocks(d)), device="cuda")
    else:
        d = case["d"]
        s["counts"], s["offsets"], s["row"] = _routing(case, g)
        rows = case["T"] * case["k"]
        if op == "permute":
            s["x"] = _activations(case["T"], d, g, _dtype(case))
            s["q"] = torch.zeros((rows, d), dtype=torch.float8_e4m3fn, device="cuda")
            s["s"] = torch.zeros((rows, _blocks(d)), device="cuda")
            return s
        s["x_q"], s["x_s"] = _quantize_rows(_activations(rows, d, g, torch.bfloat16))
        if op == "gemm":
            s["w_q"], s["w_s"] = _weights(case["E"], case["n"], d, g)
            s["y"] = torch.zeros((rows, case["n"]), dtype=torch.bfloat16, device="cuda")
        else:
            f = case["f"]
            s["gate_q"], s["gate_s"] = _weights(case["E"], f, d, g)
            s["up_q"], s["up_s"] = _weights(case["E"], f, d, g)
            s["down_q"], s["down_s"] = _weights(case["E"], d, f, g)
            s["y"] = torch.zeros((rows, d), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    op = s["case"]["op"]
    if op == "rows":
        q, scale = _quantize_rows(s["x"])
        return {"q": q, "scale": scale}
    if op == "weights":
        q, scale = _quantize_weights(s["w"])
        return {"q": q, "scale": scale}
    if op == "permute":
        q, scale = _quantize_rows(s["x"])
        token, pick = torch.nonzero(s["row"] >= 0, as_tuple=True)
        at = s["row"][token, pick].long()
        out_q, out_s = torch.zeros_like(s["q"]), torch.zeros_like(s["s"])
        out_q.view(torch.uint8)[at] = q.view(torch.uint8)[token]
        out_s[at] = scale[token]
        return {"q": out_q, "scale": out_s}
    rows, there = _bucket_rows(s["counts"], s["offsets"])
    x = _rows_value(s["x_q"], s["x_s"])[rows]  # [E, M, d], the buckets side by side
    y = torch.zeros_like(s["y"])
    if op == "gemm":
        out = torch.bmm(x, _weights_value(s["w_q"], s["w_s"]).transpose(1, 2))
    else:
        g = torch.bmm(x, _weights_value(s["gate_q"], s["gate_s"]).transpose(1, 2))
        u = torch.bmm(x, _weights_value(s["up_q"], s["up_s"]).transpose(1, 2))
        h = _rows_value(*_quantize_rows(g / (1 + torch.exp(-g)) * u))
        out = torch.bmm(h, _weights_value(s["down_q"], s["down_s"]).transpose(1, 2))
    y[rows[there]] = out[there].bfloat16()
    return y


def _run_own(s):
    import routing_dispatch_expert_warp_b200 as M
    case, op = s["case"], s["case"]["op"]
    if op == "rows":
        M.moe_fp8_quantize_rows(s["x"], s["q"], s["s"])
        return {"q": s["q"], "scale": s["s"]}
    if op == "weights":
        M.moe_fp8_quantize_weights(s["w"], s["q"], s["s"])
        return {"q": s["q"], "scale": s["s"]}
    if op == "permute":
        if "cfg" not in s:
            s["cfg"] = M.make_config(case["T"], case["d"], 128, case["E"], case["k"],
                                     dtype=M.F32 if case["dtype"] == "f32" else M.BF16)
        M.moe_fp8_permute_rows(s["cfg"], s["x"], s["row"], s["q"], s["s"])
        return {"q": s["q"], "scale": s["s"]}
    if "ws" not in s:  # what the program keeps from call to call
        s["ws"] = M.alloc_fp8_workspace()
        if op == "ffn":
            s["cfg"] = M.make_config(case["T"], case["d"], case["f"], case["E"], case["k"])
            s["experts"] = M.Fp8Experts(s["gate_q"], s["gate_s"], s["up_q"], s["up_s"],
                                        s["down_q"], s["down_s"])
            rows = case["T"] * case["k"]
            s["h_q"] = torch.empty((rows, case["f"]), dtype=torch.float8_e4m3fn, device="cuda")
            s["h_s"] = torch.empty((rows, _blocks(case["f"])), device="cuda")
    if op == "gemm":
        M.moe_fp8_grouped_gemm(s["x_q"], s["x_s"], s["offsets"], s["counts"], s["w_q"], s["w_s"],
                               s["y"], s["ws"])
    else:
        M.moe_expert_ffn_fp8(s["cfg"], s["x_q"], s["x_s"], s["offsets"], s["counts"],
                             s["experts"], s["h_q"], s["h_s"], s["y"], s["ws"])
    return s["y"]


# ------------------------------------------------------------------ what a pass needs
def work(case):
    op, d = case["op"], case["d"]
    elem = 4 if case.get("dtype") == "f32" else 2
    row = d + 4 * _blocks(d)  # bytes of a quantised row
    if op == "rows":
        return {"bytes": case["rows"] * (d * elem + row), "flops": 0}
    if op == "weights":
        E, n = case["E"], case["n"]
        return {"bytes": E * (n * d * (elem + 1) + 4 * _blocks(n) * _blocks(d)), "flops": 0}
    T, k, E = case["T"], case["k"], case["E"]
    if op == "permute":
        kept = T * k - int(case["drop"] * T * k)
        return {"bytes": T * d * elem + kept * row + 4 * T * k, "flops": 0}
    # experts that some token is expected to have picked
    touched = E * (1 - (1 - k / E) ** T)
    n = case["n"] if op == "gemm" else case["f"]
    weight = n * d + 4 * _blocks(n) * _blocks(d)
    if op == "gemm":
        return {"bytes": touched * weight + T * k * (row + 2 * n) + 8 * E,
                "flops": 2 * T * k * n * d}
    return {"bytes": 3 * touched * weight + T * k * (row + 2 * d) + 8 * E,
            "flops": 6 * T * k * n * d}


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3_64(v):
    """v rounded to the nearest e4m3 number (ties to even), in 64 bits: 3 bits behind the
    leading one, steps of 2^-9 below 2^-6, at most 448."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_rows(x):
    """(q, scale) of float64 rows; one block of 128 columns at a time."""
    d = x.shape[1]
    q, s = torch.empty_like(x), x.new_empty((x.shape[0], _blocks(d)))
    for b in range(_blocks(d)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        m = part.abs().max(dim=1).values.clamp(min=AMAX_FLOOR)
        s[:, b] = m / 448
        q[:, b * BLOCK:(b + 1) * BLOCK] = _e4m3_64(448 * part / m[:, None])
    return q, s


def _expand(s, n, d):
    """A weight's [nb, kb] scales, one for each of its n x d entries."""
    i = torch.arange(n, device=s.device) // BLOCK
    j = torch.arange(d, device=s.device) // BLOCK
    return s.double()[i][:, j]


def _exact_product(a, q, s):
    """a (float64 rows) times the transpose of one expert's weight."""
    return a @ (q.double() * _expand(s, *q.shape)).T


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rows":
        q, scale = _exact_rows(s["x"].double())
        return {"q": q, "scale": scale}
    if op == "weights":
        E, n, d = s["w"].shape
        q = torch.empty((E, n, d), dtype=torch.float64, device="cuda")
        scale = torch.empty((E, _blocks(n), _blocks(d)), dtype=torch.float64, device="cuda")
        for e in range(E):
            w = s["w"][e].double()
            for i in range(0, n, BLOCK):
                for_rows = w[i:i + BLOCK]
                peak = for_rows.abs().max(dim=0).values
                peak = torch.cat([peak, peak.new_zeros(_blocks(d) * BLOCK - d)])
                m = peak.view(-1, BLOCK).max(dim=1).values.clamp(min=AMAX_FLOOR)
                scale[e, i // BLOCK] = m / 448
                col = torch.arange(d, device="cuda") // BLOCK
                q[e, i:i + BLOCK] = _e4m3_64(448 * for_rows / m[col])
        return {"q": q, "scale": scale}
    if op == "permute":
        T, d = s["x"].shape
        q = torch.zeros((s["q"].shape[0], d), dtype=torch.float64, device="cuda")
        scale = torch.zeros(s["s"].shape, dtype=torch.float64, device="cuda")
        tq, ts = _exact_rows(s["x"].double())
        for j in range(case["k"]):
            kept = s["row"][:, j] >= 0
            at = s["row"][kept, j].long()
            q[at] = tq[kept]
            scale[at] = ts[kept]
        return {"q": q, "scale": scale}
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    first = s["offsets"].tolist()
    for e, c in enumerate(s["counts"].tolist()):
        if c == 0:
            continue
        at = slice(first[e], first[e] + c)
        x = s["x_q"][at].double()
        for b in range(_blocks(case["d"])):
            x[:, b * BLOCK:(b + 1) * BLOCK] *= s["x_s"][at, b:b + 1].double()
        if op == "gemm":
            y[at] = _exact_product(x, s["w_q"][e], s["w_s"][e])
            continue
        g = _exact_product(x, s["gate_q"][e], s["gate_s"][e])
        u = _exact_product(x, s["up_q"][e], s["up_s"][e])
        hq, hs = _exact_rows(g * torch.sigmoid(g) * u)
        for b in range(hs.shape[1]):
            hq[:, b * BLOCK:(b + 1) * BLOCK] *= hs[:, b:b + 1]
        y[at] = _exact_product(hq, s["down_q"][e], s["down_s"][e])
    return y
