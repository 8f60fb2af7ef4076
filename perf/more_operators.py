"""Work for the operators that take a batch through experts whose products run
apart, in 8-bit integers or not: tokens sorted by expert (quantised on the
way), rows brought back with the router's weights and the gradient of that,
rows quantised to int8 with one scale each, and dense and grouped int8
products with a scale per token and per output channel.

``run`` computes each operator in plain torch (``own`` false) or through
``moe_layer_amd.ops`` (``own`` true); ``exact`` evaluates the definitions in
64 bits.  An int8 row stands for codes times its scale.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one decoded token on its way to 8 of 256 experts
        {"name": "sort_token", "op": "sort", "tokens": 1, "experts": 256, "topk": 8, "cols": 7168, "type": "bf16",
         "quant": "none", "away": 0.0, "skew": 0.5},
        # a serving batch of an odd number of tokens for int8 experts
        {"name": "sort_batch", "op": "sort", "tokens": 1031, "experts": 256, "topk": 8, "cols": 4096, "type": "bf16",
         "quant": "int8", "away": 0.0, "skew": 0.7},
        # a prefill chunk of a bf16 layer, some experts much fuller than others
        {"name": "sort_prefill", "op": "sort", "tokens": 8192, "experts": 256, "topk": 8, "cols": 7168, "type": "bf16",
         "quant": "none", "away": 0.0, "skew": 1.0},
        # the experts' rows back at their tokens: a decode batch, a prefill chunk, and a training step's gradients
        {"name": "combine_batch", "op": "combine", "tokens": 64, "experts": 128, "topk": 8, "cols": 4096,
         "weights": True, "grad": False, "away": 0.0},
        {"name": "combine_prefill", "op": "combine", "tokens": 8192, "experts": 256, "topk": 8, "cols": 7168,
         "weights": True, "grad": False, "away": 0.0},
        {"name": "combine_grad", "op": "combine", "tokens": 4096, "experts": 128, "topk": 8, "cols": 4096,
         "weights": True, "grad": True, "away": 0.0},
        # the gated multiply between two int8 products: a decode batch, and an odd number of prefill rows
        {"name": "act8_batch", "op": "act8", "rows": 128, "cols": 1536, "gated": True, "clamp": 0.0},
        {"name": "act8_prefill", "op": "act8", "rows": 32771, "cols": 1536, "gated": True, "clamp": 7.0},
        # dense products of one token and of a prefill chunk
        {"name": "dense8_token", "op": "dense8", "rows": 1, "n": 4096, "k": 7168},
        {"name": "dense8_prefill", "op": "dense8", "rows": 8192, "n": 4096, "k": 7168},
        # products of sorted rows: decode (most experts one row or none) and prefill
        {"name": "grouped8_decode", "op": "grouped8", "rows": 131, "experts": 128, "n": 4096, "k": 1536, "skew": 0.5},
        {"name": "grouped8_prefill", "op": "grouped8", "rows": 32768, "experts": 128, "n": 4096, "k": 1536, "skew": 0.7},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("sort", "combine", "act8", "dense8", "grouped8"))
    if op in ("sort", "combine"):
        experts = rng.choice((4, 8, 32, 100, 128, 256))
        topk = rng.randint(1, min(experts, 8))
        case = {"op": op, "tokens": _spread(rng, 1, 8192), "experts": experts, "topk": topk,
                # half of the experts on another rank, in one case of three
                "away": rng.choice((0.0, 0.0, 0.5))}
        if op == "sort":
            kind, quant = rng.choice((("bf16", "none"), ("bf16", "int8"), ("bf16", "fp8"), ("fp8", "none"), ("int8", "none")))
            fine = 128 if "fp8" in (kind, quant) else 16
            return {**case, "cols": fine * _spread(rng, max(1, 256 // fine), 7168 // fine), "type": kind, "quant": quant,
                    "skew": rng.choice((0.0, 0.7, 1.5))}
        return {**case, "cols": 8 * _spread(rng, 16, 896), "weights": rng.random() < 0.7, "grad": rng.random() < 0.5}
    if op == "act8":
        return {"op": op, "rows": _spread(rng, 1, 32768), "cols": 16 * _spread(rng, 4, 160),
                "gated": rng.random() < 0.6, "clamp": rng.choice((0.0, 0.0, 7.0))}
    if op == "dense8":
        n = 8 * _spread(rng, 8, 896) if rng.random() < 0.5 else _spread(rng, 64, 7168)
        # whole 128-byte steps of K half of the time, 16-byte ones else
        k = 128 * _spread(rng, 2, 56) if rng.random() < 0.5 else 16 * _spread(rng, 4, 448)
        return {"op": op, "rows": _spread(rng, 1, min(8192, 8192 * 4096 * 7168 // (n * k))), "n": n, "k": k}
    experts = rng.choice((4, 8, 32, 100, 128, 256))
    n, k = 8 * _spread(rng, 16, 512), 16 * _spread(rng, 8, 256)
    while experts * n * k > 2 ** 30:     # 1 Gi weights at most
        experts //= 2
    return {"op": op, "rows": _spread(rng, 1, 16384), "experts": experts, "n": n, "k": k, "skew": rng.choice((0.0, 0.7, 1.5))}


def _live(case):
    """Routed slots: all of them, or on average the share that stays on this rank."""
    return case["tokens"] * case["topk"] * (1 - case["away"])


def work(case):
    op = case["op"]
    if op == "sort":
        cols, slots = case["cols"], case["tokens"] * case["topk"]
        width = {"bf16": 2 * cols, "fp8": cols + 4 * (cols // 128), "int8": cols + 4}
        source = width[case["type"]]
        target = source if case["quant"] == "none" else width[case["quant"]]
        return {"bytes": 8 * slots + case["tokens"] * source + _live(case) * target + 4 * (case["experts"] + 1), "flops": 0}
    if op == "combine":
        cols, slots, live = case["cols"], case["tokens"] * case["topk"], _live(case)
        once, many = 2 * cols * case["tokens"], 2 * cols * live
        meta = slots * (8 if case["weights"] else 4)
        if not case["grad"]:
            return {"bytes": meta + many + once, "flops": 2 * cols * live}
        weights = case["weights"]                             # without weights there is no gradient of theirs
        return {"bytes": meta + once + many * (2 if weights else 1) + (4 * slots if weights else 0),
                "flops": (3 if weights else 0) * cols * live}
    if op == "act8":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (5 if case["gated"] else 3) + 4 * case["rows"], "flops": n * (9 if case["gated"] else 2)}
    rows, n, k = case["rows"], case["n"], case["k"]
    if op == "dense8":
        return {"bytes": rows * k + n * k + 4 * (rows + n) + 2 * rows * n, "flops": 2 * rows * n * k}
    live = sum(1 for r in _group_rows(case, 0) if r)          # weights of experts without rows are not read
    return {"bytes": rows * (k + 4) + live * n * (k + 4) + 2 * rows * n + 4 * (case["experts"] + 1), "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ inputs ---

def _group_rows(case, seed):
    """Rows per expert: a multinomial over exp(skew * N(0, 1)) loads."""
    g = torch.Generator().manual_seed(6007 * int(seed) + 29)
    load = torch.softmax(case["skew"] * torch.randn(case["experts"], generator=g), 0)
    pick = torch.multinomial(load, case["rows"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=case["experts"]).tolist()


def _router(case, g, d, skew):
    """Expert ids of every token, the topk largest of random logits, and softmax weights; ids of experts
    that another rank holds are -1."""
    total = case["experts"] * (2 if case["away"] else 1)
    bias = skew * torch.randn(total, generator=g, device=d)
    logits = torch.randn(case["tokens"], total, generator=g, device=d) + bias
    top, ids = logits.topk(case["topk"], 1)
    ids = torch.where(ids < case["experts"], ids, -1).to(torch.int32)
    return ids.contiguous(), torch.softmax(top, 1).contiguous()


def _int8_rows(v):
    """Rows of any values as int8 codes and scales (how inputs are made; not the operator's rounding)."""
    s = v.float().abs().amax(-1, keepdim=True).clamp_min(1e-10) / 127
    return torch.round(v.float() / s).to(torch.int8), s[..., 0].contiguous()


def _fp8_rows(v):
    g = v.float().unflatten(-1, (-1, 128))
    s = _pow2_scale(g.abs().amax(-1))
    return (g / s[..., None]).flatten(-2).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    d = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=d).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=d, dtype=torch.bfloat16)

    st = dict(case)
    op = case["op"]
    if op == "sort":
        tokens, cols, slots = case["tokens"], case["cols"], case["tokens"] * case["topk"]
        st["ids"], _ = _router(case, g, d, case["skew"])
        # a normed row: a few channels many times the others
        x = randn(tokens, cols) * (1 + 15 * (torch.rand(cols, generator=g, device=d) < 0.01)).bfloat16()
        st["x"], st["x_scale"] = (x, None) if case["type"] == "bf16" else _fp8_rows(x) if case["type"] == "fp8" else _int8_rows(x)
        out = case["type"] if case["quant"] == "none" else case["quant"]
        st["rows"] = torch.zeros(slots, cols, device=d, dtype=torch.uint8 if out == "fp8" else torch.int8 if out == "int8" else torch.bfloat16)
        if out == "fp8":
            st["rows"] = st["rows"].view(torch.float8_e4m3fn)
        st["scales"] = None
        if out != "bf16":
            st["scales"] = torch.zeros((slots, cols // 128) if out == "fp8" else (slots,), device=d)
        st["offsets"] = torch.empty(case["experts"] + 1, dtype=torch.int32, device=d)
        st["inv"] = torch.empty(tokens, case["topk"], dtype=torch.int32, device=d)
        # what a serving program allocates once; more than the call needs
        st["scratch"] = torch.empty(8 * (slots // 256 + 2) * (case["experts"] + 2) + 1024, dtype=torch.uint8, device=d)
        return st
    if op == "combine":
        tokens, cols, slots = case["tokens"], case["cols"], case["tokens"] * case["topk"]
        ids, weights = _router(case, g, d, 0.5)
        key = torch.where(ids >= 0, ids, case["experts"]).flatten()
        place = torch.empty(slots, dtype=torch.int32, device=d)
        place[torch.argsort(key, stable=True)] = torch.arange(slots, dtype=torch.int32, device=d)
        st["inv"] = torch.where(key < case["experts"], place, -1).view(tokens, case["topk"])
        st["weights"] = weights if case["weights"] else None
        st["rows"] = randn(slots, cols)
        if case["grad"]:
            st["grad_out"] = randn(tokens, cols)
            st["grad_rows"] = torch.zeros(slots, cols, dtype=torch.bfloat16, device=d)
            st["grad_weights"] = torch.empty(tokens, case["topk"], device=d) if case["weights"] else None
        else:
            st["out"] = torch.empty(tokens, cols, dtype=torch.bfloat16, device=d)
        return st
    if op == "act8":
        rows, cols = case["rows"], case["cols"]
        st["x"] = randn(rows, 2 * cols if case["gated"] else cols) * 2
        st["codes"] = torch.empty(rows, cols, dtype=torch.int8, device=d)
        st["scales"] = torch.empty(rows, device=d)
        return st
    rows, n, k = case["rows"], case["n"], case["k"]
    st["a"], st["a_scale"] = _int8_rows(randn(rows, k))
    if op == "dense8":
        st["w"], st["w_scale"] = _int8_rows(randn(n, k) * k ** -0.5)
    else:
        parts = [_int8_rows(randn(min(32, case["experts"] - i), n, k) * k ** -0.5) for i in range(0, case["experts"], 32)]
        st["w"], st["w_scale"] = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
        per = _group_rows(case, seed)
        st["offsets"] = torch.tensor([0] + per, device=d).cumsum(0).to(torch.int32)
        st["most"] = max(per)
    st["out"] = torch.empty(rows, n, dtype=torch.bfloat16, device=d)
    return st


# -------------------------------------------------------------- plain forms ---

def _pow2_scale(amax):
    """The smallest power of two >= max(amax, 1e-10) * fl32(1 / 448)."""
    raw = amax.clamp_min(1e-10) * torch.tensor(1 / E4M3_MAX, dtype=torch.float32, device=amax.device)
    # a carry out of the fraction bits steps to the next power of two
    return ((raw.view(torch.int32) + 0x7fffff) & 0x7f800000).view(torch.float32)


def _plain_int8(v):
    most = v.float().abs().amax(-1, keepdim=True).clamp_min(1e-10).double()
    # 64 bits: fp32 quotients rounded to the nearest (torch divides by a number through its inverse), and products
    # next to a half rounded once
    codes = torch.round(v.double() * (127 / most).float().double()).to(torch.int8)
    return codes, (most / 127).float()[..., 0]


def _plain_fp8(v):
    g = v.float().unflatten(-1, (-1, 128))
    s = _pow2_scale(g.abs().amax(-1))
    return (g / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(-2).to(torch.float8_e4m3fn), s


def _plain_sort(st):
    ids, experts, topk = st["ids"].flatten(), st["experts"], st["topk"]
    key = torch.where((ids >= 0) & (ids < experts), ids, experts)
    order = torch.argsort(key, stable=True)
    offsets = torch.searchsorted(key[order], torch.arange(experts + 1, dtype=key.dtype, device=key.device)).to(torch.int32)
    row = torch.arange(len(ids), dtype=torch.int32, device=key.device)
    inv = torch.empty_like(row)
    inv[order] = row
    inv = torch.where(key < experts, inv, -1).view(-1, topk)
    x, scale = st["x"], st["x_scale"]
    if st["quant"] != "none":
        x, scale = (_plain_int8 if st["quant"] == "int8" else _plain_fp8)(x)
    there, token = (row < offsets[-1])[:, None], torch.div(order, topk, rounding_mode="floor")
    if x.dtype == torch.float8_e4m3fn:
        rows = torch.where(there, x.view(torch.uint8)[token], st["rows"].view(torch.uint8)).view(torch.float8_e4m3fn)
    else:
        rows = torch.where(there, x[token], st["rows"])
    out = {"rows": rows, "offsets": offsets, "inv": inv}
    if scale is not None:
        out["scales"] = torch.where(there if scale.dim() == 2 else there[:, 0], scale[token], st["scales"])
    return out


def _plain_combine(st):
    inv = st["inv"].long()
    there = (inv >= 0)[..., None]
    rows = torch.where(there, st["rows"][inv.clamp_min(0)].float(), 0.0)
    if st["weights"] is not None:
        rows = rows * st["weights"][..., None]
    return {"out": rows.sum(1).bfloat16()}


def _plain_combine_grad(st):
    inv = st["inv"].long()
    there = inv >= 0
    grad = st["grad_out"].float()[:, None, :].expand(-1, st["topk"], -1)
    weighted = grad if st["weights"] is None else grad * st["weights"][..., None]
    slots = inv.numel()
    # slots without a row go to a row behind the last one
    target = torch.cat([st["grad_rows"], st["grad_rows"][:1]])
    target[torch.where(there, inv, slots).flatten()] = weighted.reshape(slots, -1).bfloat16()
    out = {"grad_rows": target[:slots]}
    if st["weights"] is not None:
        dots = (grad * st["rows"][inv.clamp_min(0)].float()).sum(-1)
        out["grad_weights"] = torch.where(there, dots, 0.0)
    return out


def _plain_act8(st):
    v = st["x"]
    if st["gated"]:
        gate, up = v.float().chunk(2, -1)
        if st["clamp"] > 0:
            gate, up = gate.clamp_max(st["clamp"]), up.clamp(-st["clamp"], st["clamp"])
        gd = gate.double()                                    # 64 bits: bf16 borders
        v = ((gd / (1 + torch.exp(-gd))).float().bfloat16().float() * up).bfloat16()
    codes, scales = _plain_int8(v)
    return {"codes": codes, "scales": scales}


def _plain_dense8(st):
    # sums of whole numbers, exact as long as they stay below 2^24
    total = torch.mm(st["a"].float(), st["w"].float().t())
    return {"out": (total * st["a_scale"][:, None] * st["w_scale"]).bfloat16()}


def _plain_grouped8(st):
    off = st["offsets"].long()
    row = torch.arange(st["rows"], device=off.device)
    expert = torch.searchsorted(off, row, right=True) - 1     # the last expert starting at or before the row
    place = row - off[expert]
    slab = torch.zeros(st["experts"], st["most"], st["k"], device=off.device)
    slab[expert, place] = st["a"].float()
    total = torch.bmm(slab, st["w"].float().transpose(1, 2).contiguous())[expert, place]
    return {"out": (total * st["a_scale"][:, None] * st["w_scale"][expert]).bfloat16()}


# --------------------------------------------------------------------- run ---

def run(st):
    op = st["op"]
    if own:
        from moe_layer_amd import ops
        if op == "sort":
            rows, scales, offsets, inv = ops.moe_sort_rows(
                st["x"], st["ids"], st["experts"], x_scale=st["x_scale"],
                quant=None if st["quant"] == "none" else st["quant"], rows=st["rows"], scales=st["scales"],
                offsets=st["offsets"], inv=st["inv"], scratch=st["scratch"])
            out = {"rows": rows, "offsets": offsets, "inv": inv}
            return out if scales is None else {**out, "scales": scales}
        if op == "combine" and not st["grad"]:
            return {"out": ops.moe_combine_rows(st["rows"], st["inv"], st["weights"], out=st["out"])}
        if op == "combine":
            grad_rows, grad_weights = ops.moe_combine_rows_bwd(
                st["grad_out"], st["inv"], rows=st["rows"] if st["weights"] is not None else None,
                weights=st["weights"], grad_rows=st["grad_rows"], grad_weights=st["grad_weights"])
            return {"grad_rows": grad_rows} if grad_weights is None else {"grad_rows": grad_rows, "grad_weights": grad_weights}
        if op == "act8" and st["gated"]:
            codes, scales = ops.moe_silu_mul_int8(st["x"], clamp_limit=st["clamp"], codes=st["codes"], scales=st["scales"])
            return {"codes": codes, "scales": scales}
        if op == "act8":
            codes, scales = ops.moe_quant_act_int8(st["x"], codes=st["codes"], scales=st["scales"])
            return {"codes": codes, "scales": scales}
        if op == "dense8":
            return {"out": ops.moe_gemm_int8(st["a"], st["a_scale"], st["w"], st["w_scale"], out=st["out"])}
        return {"out": ops.moe_grouped_gemm(st["a"], st["w"], st["offsets"], st["a_scale"], st["w_scale"], out=st["out"])}
    if op == "combine":
        return _plain_combine_grad(st) if st["grad"] else _plain_combine(st)
    return {"sort": _plain_sort, "act8": _plain_act8, "dense8": _plain_dense8, "grouped8": _plain_grouped8}[op](st)


# ------------------------------------------------- the definitions in 64 bits ---

def _exact_int8(v):
    """Codes and scales of rows: the scale and its inverse are fp32 quotients, the code the nearest whole
    number (ties to even) of the value times the inverse."""
    most = v.abs().max(-1).values.clamp_min(1e-10).float().double()
    scale, inverse = (most / 127).float().double(), (127 / most).float().double()
    return torch.round(v * inverse[:, None]).to(torch.int8), scale


def _exact_fp8(v):
    rows, cols = v.shape
    v = v.reshape(rows, cols // 128, 128)
    mant, e = torch.frexp(v.abs().max(-1).values.clamp_min(1e-10) / E4M3_MAX)
    scale = ((e - (mant == 0.5).int() + 1023).long() << 52).view(torch.float64)
    q = (v / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    step = ((torch.frexp(q)[1].clamp_min(-5) - 4 + 1023).long() << 52).view(torch.float64)
    return (torch.round(q / step) * step).reshape(rows, cols), scale


def exact(case, seed):
    st = prepare(case, seed)
    op, f64 = case["op"], torch.float64
    if op == "sort":
        ids, topk, slots = st["ids"].flatten(), case["topk"], case["tokens"] * case["topk"]
        inv = torch.full((slots,), -1, dtype=torch.int32, device=ids.device)
        offsets, order = [0], []
        for e in range(case["experts"]):
            mine = torch.nonzero(ids == e)[:, 0]
            inv[mine] = torch.arange(offsets[-1], offsets[-1] + len(mine), dtype=torch.int32, device=ids.device)
            offsets.append(offsets[-1] + len(mine))
            order.append(mine)
        token = torch.cat(order) // topk
        x, scale = st["x"].to(f64), st["x_scale"]
        if case["quant"] != "none":
            x, scale = (_exact_int8 if case["quant"] == "int8" else _exact_fp8)(x)
        whole = x.dtype == torch.int8 or case["type"] == "int8"
        rows = torch.zeros(slots, case["cols"], dtype=torch.int8 if whole else f64, device=ids.device)
        rows[: len(token)] = x[token].to(rows.dtype)
        out = {"rows": rows, "offsets": torch.tensor(offsets, dtype=torch.int32, device=ids.device), "inv": inv.view(-1, topk)}
        if scale is not None:
            out["scales"] = torch.zeros(slots, *scale.shape[1:], dtype=f64, device=ids.device)
            out["scales"][: len(token)] = scale[token].to(f64)
        return out
    if op == "combine":
        tokens, topk, slots = case["tokens"], case["topk"], case["tokens"] * case["topk"]
        w = torch.ones(tokens, topk, dtype=f64, device=st["inv"].device) if st["weights"] is None else st["weights"].to(f64)
        if not case["grad"]:
            total = torch.zeros(tokens, case["cols"], dtype=f64, device=w.device)
        else:
            grad = st["grad_out"].to(f64)
            d_rows = torch.zeros(slots, case["cols"], dtype=f64, device=w.device)
            d_weights = torch.zeros(tokens, topk, dtype=f64, device=w.device)
        for j in range(topk):
            t = torch.nonzero(st["inv"][:, j] >= 0)[:, 0]
            r = st["inv"][t, j].long()
            if not case["grad"]:
                total[t] += w[t, j, None] * st["rows"][r].to(f64)
            else:
                d_rows[r] = w[t, j, None] * grad[t]
                d_weights[t, j] = torch.einsum("th,th->t", grad[t], st["rows"][r].to(f64))
        if not case["grad"]:
            return {"out": total}
        return {"grad_rows": d_rows, "grad_weights": d_weights} if case["weights"] else {"grad_rows": d_rows}
    if op == "act8":
        v = st["x"].to(f64)
        if case["gated"]:
            gate, up = v[:, : case["cols"]], v[:, case["cols"]:]
            if case["clamp"] > 0:
                gate, up = gate.clamp(max=case["clamp"]), up.clamp(-case["clamp"], case["clamp"])
            v = ((gate * torch.sigmoid(gate)).bfloat16().to(f64) * up).bfloat16().to(f64)
        codes, scales = _exact_int8(v)
        return {"codes": codes, "scales": scales}

    def product(a, a_scale, w, w_scale):
        return (a.to(f64) @ w.to(f64).T) * a_scale.to(f64)[:, None] * w_scale.to(f64)

    if op == "dense8":
        return {"out": product(st["a"], st["a_scale"], st["w"], st["w_scale"])}
    off = st["offsets"].tolist()
    out = torch.empty(case["rows"], case["n"], dtype=f64, device=st["a"].device)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            out[lo:hi] = product(st["a"][lo:hi], st["a_scale"][lo:hi], st["w"][e], st["w_scale"][e])
    return {"out": out}
