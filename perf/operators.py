"""Cases of the matrix products with a fused epilogue, of the expert-grouped products and of the two row
operators beside them (grouping rows by expert, joining the experts' rows per token), in plain torch form and
as calls of the package.

    z[t][r] = s[r] sum_k sigma[r][k] u[t][k] + bias[r]
    epilogue:  o = act(z) + residual, or gated on interleaved rows  o[i] = act(z[2i]) z[2i+1] + residual[i]
    grouped:   slot i of expert e (offsets[e] <= i < offsets[e+1]) takes row rows[i] of u and expert e's layer
    group:     expert ids [tokens][topk] -> offsets [experts+1], rows (token of each slot, -1 past the last), slots
    combine:   o[t] = residual[t] + sum_j weights[t][j] y[slots[t][j]]

A layer is LQ-D/d: in channels give K = (in/d) D sign bits per output row, padded to a multiple of 32.
"""

import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
CODES = ((10, 24), (8, 16), (8, 19), (8, 20), (8, 22), (8, 24))


def _k(case):
    return -(-(case["in"] // case["d"] * case["D"]) // 32) * 32


def _layer(name, d, D, in_dim, out, tokens, u, o, act, glu, bias, residual):
    return {"name": name, "op": "epilogue", "d": d, "D": D, "in": in_dim, "out": out, "tokens": tokens, "u": u, "o": o,
            "act": act, "glu": glu, "bias": bias, "residual": residual}


def _grouped(name, d, D, in_dim, out, tokens, topk, experts, gather, skew, o, act, glu, bias):
    return {"name": name, "op": "grouped", "d": d, "D": D, "in": in_dim, "out": out, "tokens": tokens, "topk": topk,
            "experts": experts, "gather": gather, "skew": skew, "o": o, "act": act, "glu": glu, "bias": bias}


def listed():
    return [
        # one decoded token, full precision, an output projection back into an fp32 residual stream
        _layer("epilogue f32 1 token", 10, 24, 5120, 13824, 1, "f32", "f32", "none", False, True, True),
        # a small decode batch through the gate and up rows of an MLP, bf16 activations
        _layer("epilogue bf16 8 tokens gated", 8, 20, 8192, 28672, 8, "bf16", "bf16", "silu", True, False, False),
        # a short prompt (or a chunk of drafted tokens) with odd sizes
        _layer("epilogue bf16 61 tokens odd", 8, 19, 4096, 11007, 61, "bf16", "bf16", "gelu_tanh", False, True, True),
        # a long prompt, gate and up rows
        _layer("epilogue bf16 2048 tokens", 10, 24, 5120, 13824, 2048, "bf16", "bf16", "silu", True, True, False),
        # one decoded token: two experts of eight are read
        _grouped("grouped 1 token", 8, 20, 4096, 11008, 1, 2, 8, True, 0.0, "bf16", "silu", True, False),
        # a decode batch over many small experts, a few rows each, some with none
        _grouped("grouped 32 tokens", 8, 16, 2048, 2816, 32, 4, 32, True, 1.0, "bf16", "silu", True, False),
        # a short prompt's second product: rows already in slot order, uneven experts, odd sizes
        _grouped("grouped 300 tokens uneven", 8, 22, 1408, 2050, 300, 2, 8, False, 2.0, "f32", "none", False, True),
        # a long prompt's first product
        _grouped("grouped 4096 tokens", 8, 20, 4096, 4096, 4096, 2, 8, True, 0.5, "bf16", "silu", True, False),
        # routing of a decode batch
        {"name": "group 16 tokens", "op": "group", "tokens": 16, "topk": 2, "experts": 8, "skew": 0.0, "drop": 0.0},
        # routing of a long prompt, a tenth of the choices dropped (experts of other ranks, full experts)
        {"name": "group 16384 tokens", "op": "group", "tokens": 16384, "topk": 8, "experts": 128, "skew": 1.0, "drop": 0.1},
        # the end of the experts' block of a decode batch and of a long prompt
        {"name": "combine 16 tokens", "op": "combine", "tokens": 16, "topk": 2, "width": 5120, "o": "f32",
         "residual": True, "drop": 0.2},
        {"name": "combine 4096 tokens", "op": "combine", "tokens": 4096, "topk": 4, "width": 4096, "o": "bf16",
         "residual": True, "drop": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """Any operator of the four, sizes spread over their logarithm, odd ones among them."""
    op = rng.choice(("epilogue", "epilogue", "grouped", "grouped", "group", "combine"))
    o = rng.choice(("f32", "bf16"))
    if op == "group":
        return {"op": op, "tokens": _log(rng, 1, 16384), "topk": rng.randint(1, 8), "experts": _log(rng, 8, 128),
                "skew": rng.choice((0.0, 1.0, 2.0)), "drop": rng.choice((0.0, 0.0, 0.3))}
    if op == "combine":
        return {"op": op, "tokens": _log(rng, 1, 4096), "topk": rng.randint(1, 4), "width": _log(rng, 100, 4096),
                "o": o, "residual": rng.random() < 0.5, "drop": rng.choice((0.0, 0.0, 0.3))}
    d, D = rng.choice(CODES)
    in_dim = 128 * d // 2 * _log(rng, 1, 8192 // (64 * d)) if rng.random() < 0.5 else d * _log(rng, 16, 8192 // d)
    out = 2 * _log(rng, 64, 8192) + rng.choice((0, 0, 1))
    glu = out % 2 == 0 and rng.random() < 0.5
    act = rng.choice(ACTS)
    if op == "epilogue":
        u = rng.choice(("f32", "bf16", "bf16"))
        tokens = rng.randint(1, 16) if u == "f32" else _log(rng, 1, 2048)
        while tokens > 1 and tokens * out * _k({"in": in_dim, "d": d, "D": D}) > 3.4e11:
            tokens = tokens // 2
        case = _layer("", d, D, in_dim, out, tokens, u, o, act, glu, rng.random() < 0.5, rng.random() < 0.5)
    else:
        experts, topk = _log(rng, 4, 64), rng.randint(1, 4)
        tokens = _log(rng, 1, 4096)
        # all experts' signs, and all rows if they met one expert, stay below the listed cases'
        while experts * out * _k({"in": in_dim, "d": d, "D": D}) > 8e8:
            out = 2 * (out // 4) + out % 2
        while tokens > 1 and tokens * max(experts, 2 * topk) * out * _k({"in": in_dim, "d": d, "D": D}) > 6e11:
            tokens = tokens // 2
        case = _grouped("", d, D, in_dim, out, tokens, topk, experts, rng.random() < 0.6,
                        rng.choice((0.0, 1.0, 2.0)), o, act, glu, rng.random() < 0.5)
    del case["name"]
    return case


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _lifted(case, tokens, dtype, gen):
    """u = blockdiag(M^T) a of activations a ~ N(0, 1) (orthogonal whitening leaves them so), M ~ N(0, 1/D)."""
    d, D, blocks = case["d"], case["D"], case["in"] // case["d"]
    a = torch.randn((tokens, blocks, d), device="cuda", generator=gen)
    M = torch.randn((d, D), device="cuda", generator=gen) / math.sqrt(D)
    u = torch.zeros((tokens, _k(case)), device="cuda")
    u[:, : blocks * D] = (a @ M).reshape(tokens, blocks * D)
    return u.to(dtype)


def _signs(shape, gen):
    """Random packed signs: one word is 32 signs, least significant bit first, bit 1 = +1."""
    return torch.randint(-2**31, 2**31, shape, device="cuda", generator=gen, dtype=torch.int64).to(torch.int32)


def _choices(case, gen):
    """Each token's topk distinct experts, the likelier ones more often with more skew; dropped choices are -1."""
    T, E, k = case["tokens"], case["experts"], case["topk"]
    liking = case["skew"] * torch.randn(E, device="cuda", generator=gen)
    noise = -torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=gen).clamp(1e-7, 1 - 1e-6)))
    ids = (liking + noise).topk(k, dim=1).indices.to(torch.int32)
    if case.get("drop"):
        ids = torch.where(torch.rand((T, k), device="cuda", generator=gen) < case["drop"], -1, ids)
    return ids.contiguous()


def _slots(ids, experts):
    """(offsets, rows, slots) of expert ids [tokens][topk]: a stable sort by expert, ids outside 0..experts-1 left out."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.argsort(key, stable=True)
    counts = (key[:, None] == torch.arange(experts, device=ids.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    place = torch.arange(T * k, device=ids.device)
    kept = place < offsets[-1]
    rows = torch.where(kept, order // k, -1)
    slots = torch.empty_like(place)
    slots[order] = torch.where(kept, place, -1)
    return offsets.to(torch.int32), rows.to(torch.int32), slots.reshape(T, k).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case}
    op = case["op"]
    if op == "group":
        st["ids"] = _choices(case, gen)
        return st
    o = _dtype(case["o"])
    if op == "combine":
        T, k, n = case["tokens"], case["topk"], case["tokens"] * case["topk"]
        slots = torch.randperm(n, device="cuda", generator=gen).reshape(T, k)
        slots = torch.where(torch.rand((T, k), device="cuda", generator=gen) < case["drop"], -1, slots)
        w = torch.rand((T, k), device="cuda", generator=gen) + 0.05
        st["slots"], st["weights"] = slots.to(torch.int32), w / w.sum(1, keepdim=True)
        st["y"] = torch.randn((n, case["width"]), device="cuda", generator=gen).to(o)
        st["residual"] = torch.randn((T, case["width"]), device="cuda", generator=gen).to(o) if case["residual"] else None
        return st
    K, out = _k(case), case["out"]
    lead = (case["experts"],) if op == "grouped" else ()
    st["packed"] = _signs(lead + (out, K // 32), gen)
    st["s"] = torch.empty(lead + (out,), device="cuda").uniform_(0.01, 0.03, generator=gen)
    st["bias"] = 0.2 * torch.randn(lead + (out,), device="cuda", generator=gen) if case["bias"] else None
    if op == "epilogue":
        T = case["tokens"]
        st["u"] = _lifted(case, T, _dtype(case["u"]), gen)
        width = out // 2 if case["glu"] else out
        st["residual"] = torch.randn((T, width), device="cuda", generator=gen).to(o) if case["residual"] else None
        return st
    st["offsets"], rows, _ = _slots(_choices(case, gen), case["experts"])
    st["n"] = n = case["tokens"] * case["topk"]
    st["most"] = int((st["offsets"][1:] - st["offsets"][:-1]).max())
    st["rows"] = rows if case["gather"] else None
    st["u"] = _lifted(case, case["tokens"] if case["gather"] else n, torch.bfloat16, gen)
    return st


def _unpacked(packed):
    """The signs as +-1 in fp32, [..., out, K]."""
    bits = (packed[..., None] >> torch.arange(32, device=packed.device, dtype=torch.int32)) & 1
    return bits.to(torch.float32).mul_(2).sub_(1).flatten(-2)


def _activated(z, act):
    if act == "relu":
        return torch.where(z < 0, 0.0, z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _epilogue(z, case, residual):
    y = _activated(z[..., 0::2], case["act"]) * z[..., 1::2] if case["glu"] else _activated(z, case["act"])
    if residual is not None:
        y = y + residual.float()
    return y.to(_dtype(case["o"]))


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    if case["op"] == "group":
        return _slots(st["ids"], case["experts"])
    if case["op"] == "combine":
        slots, n = st["slots"].long(), st["y"].shape[0]
        there = (slots >= 0) & (slots < n)
        picked = st["y"][torch.where(there, slots, 0)].float() * torch.where(there, st["weights"], 0.0)[..., None]
        total = picked.sum(1)
        if st["residual"] is not None:
            total = total + st["residual"].float()
        return total.to(st["y"].dtype)
    if case["op"] == "epilogue":
        z = st["s"] * (st["u"].float() @ _unpacked(st["packed"]).T)
        if st["bias"] is not None:
            z = z + st["bias"]
        return _epilogue(z, case, st["residual"])
    # grouped: every expert's rows padded to the most that one has, one batched product
    n, E = st["n"], case["experts"]
    slot = torch.arange(n, device="cuda")
    expert = torch.bucketize(slot, st["offsets"][1:].long(), right=True)
    place = slot - st["offsets"].long()[expert]
    picked = (st["u"] if st["rows"] is None else st["u"][st["rows"].long()]).float()
    x = picked.new_zeros((E, st["most"], picked.shape[1]))
    x[expert, place] = picked
    z = torch.bmm(x, _unpacked(st["packed"]).transpose(1, 2))[expert, place] * st["s"][expert]
    if st["bias"] is not None:
        z = z + st["bias"][expert]
    return _epilogue(z, case, None)


def _run_own(st):
    import bit_lifted_gemm_b200 as lq
    case = st["case"]
    if case["op"] == "group":
        return lq.group_rows(st["ids"], case["experts"])
    if case["op"] == "combine":
        return lq.combine_rows(st["y"], st["slots"], st["weights"], residual=st["residual"])
    how = {"bias": st["bias"], "act": case["act"], "glu": case["glu"], "o_dtype": case["o"]}
    if case["op"] == "grouped":
        return lq.gemm_grouped(st["packed"], st["s"], st["u"], st["offsets"], st["n"], rows=st["rows"], **how)
    call = lq.gemv_epilogue if case["u"] == "f32" else lq.gemm_epilogue
    return call(st["packed"], st["s"], st["u"], residual=st["residual"], **how)


def work(case):
    op = case["op"]
    if op == "group":
        n = case["tokens"] * case["topk"]
        return {"bytes": 12 * n + 4 * (case["experts"] + 1), "flops": 0}
    e = 4 if case["o"] == "f32" else 2
    if op == "combine":
        n = case["tokens"] * case["topk"]
        kept = n * (1 - case["drop"])
        width = case["width"]
        return {"bytes": kept * width * e + 8 * n + case["tokens"] * width * e * (2 if case["residual"] else 1),
                "flops": 2 * kept * width}
    K, out = _k(case), case["out"]
    width = out // 2 if case["glu"] else out
    layer = out * K // 8 + 4 * out * (2 if case["bias"] else 1)
    if op == "epilogue":
        T = case["tokens"]
        return {"bytes": layer + T * K * (4 if case["u"] == "f32" else 2) + T * width * e * (2 if case["residual"] else 1),
                "flops": 2 * T * out * K}
    # the experts that have rows: as many as there are choices, at most all
    n = case["tokens"] * case["topk"]
    rows = case["tokens"] if case["gather"] else n
    return {"bytes": min(n, case["experts"]) * layer + rows * K * 2 + n * width * e, "flops": 2 * n * out * K}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "group":
        ids = st["ids"].cpu().reshape(-1).tolist()
        E, k = case["experts"], case["topk"]
        lists = [[] for _ in range(E)]
        for i, e in enumerate(ids):
            if 0 <= e < E:
                lists[e].append(i)
        offsets, rows, slots = [0], [], [-1] * len(ids)
        for members in lists:
            for i in members:
                slots[i] = len(rows)
                rows.append(i // k)
            offsets.append(len(rows))
        rows += [-1] * (len(ids) - len(rows))
        whole = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
        return whole(offsets), whole(rows), whole(slots).reshape(-1, k)
    if op == "combine":
        y, w, total = st["y"].double(), st["weights"].double(), None
        total = torch.zeros((case["tokens"], case["width"]), dtype=torch.float64, device="cuda")
        for j in range(case["topk"]):
            s = st["slots"][:, j]
            at = torch.nonzero(s >= 0)[:, 0]
            total[at] += w[at, j, None] * y[s[at].long()]
        return total if st["residual"] is None else total + st["residual"].double()

    def layer(packed, s, u, bias, residual):
        words = packed.to(torch.int64) & 0xFFFFFFFF
        acc = torch.zeros((u.shape[0], packed.shape[0]), dtype=torch.float64, device="cuda")
        u = u.double().reshape(u.shape[0], packed.shape[1], 32)
        for bit in range(32):  # the words' bit by bit: sum of +-u over every 32nd element
            sign = torch.where((words >> bit) % 2 == 1, 1.0, -1.0).double()
            acc += torch.einsum("tw,rw->tr", u[:, :, bit], sign)
        z = acc * s.double() + (0 if bias is None else bias.double())
        x = z[:, 0::2] if case["glu"] else z
        if case["act"] == "relu":
            x = x.clamp(min=0)
        elif case["act"] == "gelu":
            x = x * 0.5 * torch.special.erfc(-x / math.sqrt(2.0))
        elif case["act"] == "gelu_tanh":
            x = x * torch.sigmoid(2 * math.sqrt(2 / math.pi) * x * (1 + 0.044715 * x ** 2))
        elif case["act"] == "silu":
            x = x * torch.sigmoid(x)
        x = x * z[:, 1::2] if case["glu"] else x
        return x if residual is None else x + residual.double()

    if op == "epilogue":
        return layer(st["packed"], st["s"], st["u"], st["bias"], st["residual"])
    at = st["offsets"].tolist()
    parts = []
    for e in range(case["experts"]):
        rows = torch.arange(at[e], at[e + 1], device="cuda") if st["rows"] is None else st["rows"][at[e]: at[e + 1]].long()
        parts.append(layer(st["packed"][e], st["s"][e], st["u"][rows], None if st["bias"] is None else st["bias"][e], None))
    return torch.cat(parts)
