"""Work for the operators around the fused MoE layer: the quantising
residual-add + RMSNorm, the quantising SiLU-gated multiply, the dense
block-scaled fp8 product and the ragged products grouped by expert.

``run`` computes each operator in plain torch (``own`` false) or through
``moe_layer_amd.ops`` (``own`` true); ``exact`` evaluates the definitions in
64 bits.  fp8 values are OCP E4M3FN; a scale covers 128 columns of a row
(activations, a power of two), a 128 x 128 block (weights, any fp32), or 32
columns as an E8M0 byte (MXFP8).  A quantised output comes back as its two
tensors, the float8 codes and their scales.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one decoded token entering a layer: residual added, normed, quantised for the fp8 products
        {"name": "norm_token", "op": "norm", "rows": 1, "cols": 7168, "residual": True, "quant": "fp8", "y": False},
        # a decode batch of a bf16 layer, which reads the normed row itself
        {"name": "norm_batch", "op": "norm", "rows": 64, "cols": 4096, "residual": True, "quant": "none", "y": True},
        # prefill: the router reads the normed row, the fp8 products its codes
        {"name": "norm_prefill", "op": "norm", "rows": 8192, "cols": 7168, "residual": True, "quant": "fp8", "y": True},
        # odd row count, no residual yet (a model's first norm), MXFP8 codes
        {"name": "norm_mx", "op": "norm", "rows": 1537, "cols": 4096, "residual": False, "quant": "mxfp8", "y": False},
        # a shared expert's activation at decode, and a routed batch's in prefill (ragged row total)
        {"name": "act_token", "op": "act", "rows": 16, "cols": 2048, "quant": "fp8", "clamp": 0.0},
        {"name": "act_prefill", "op": "act", "rows": 20011, "cols": 2048, "quant": "fp8", "clamp": 7.0},
        # dense products: one token, a decode batch on a narrow projection, a prefill chunk, an odd one
        {"name": "dense_token", "op": "dense", "rows": 1, "n": 4096, "k": 7168},
        {"name": "dense_batch", "op": "dense", "rows": 64, "n": 7168, "k": 2048},
        {"name": "dense_prefill", "op": "dense", "rows": 8192, "n": 4096, "k": 7168},
        # products of an expert-parallel rank's routed rows: decode (most experts one row), the fp8
        # layer's gate/up shape, and a bf16 prefill down projection
        {"name": "grouped_decode", "op": "grouped", "rows": 131, "experts": 128, "n": 4096, "k": 1536, "type": "bf16", "skew": 0.5},
        {"name": "grouped_fp8", "op": "grouped", "rows": 8192, "experts": 256, "n": 512, "k": 4096, "type": "fp8", "skew": 0.7},
        {"name": "grouped_prefill", "op": "grouped", "rows": 32768, "experts": 128, "n": 4096, "k": 1536, "type": "bf16", "skew": 0.7},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "act", "dense", "dense", "grouped", "grouped"))
    if op == "norm":
        rows, cols = _spread(rng, 1, 8192), 128 * rng.randint(2, 56)
        quant = rng.choice(("none", "fp8", "fp8", "mxfp8"))
        return {"op": op, "rows": rows, "cols": cols, "residual": rng.random() < 0.7, "quant": quant,
                "y": quant == "none" or rng.random() < 0.5}
    if op == "act":
        return {"op": op, "rows": _spread(rng, 1, 20000), "cols": 128 * rng.randint(1, 16),
                "quant": rng.choice(("none", "fp8", "fp8", "mxfp8")), "clamp": rng.choice((0.0, 0.0, 7.0))}
    if op == "dense":
        # output widths are whole 16-byte rows half of the time, any number else
        n = 8 * _spread(rng, 8, 896) if rng.random() < 0.5 else _spread(rng, 64, 7168)
        k = 128 * _spread(rng, 2, 56)
        return {"op": op, "rows": _spread(rng, 1, min(8192, 8192 * 4096 * 7168 // (n * k))), "n": n, "k": k}
    experts = rng.choice((4, 8, 32, 128, 256))
    n, k = 64 * _spread(rng, 4, 64), 128 * _spread(rng, 2, 32)
    while experts * n * k > 2 ** 30:     # 1 Gi weights at most
        experts //= 2
    return {"op": op, "rows": _spread(rng, 1, 16384), "experts": experts, "n": n, "k": k,
            "type": rng.choice(("bf16", "fp8")), "skew": rng.choice((0.0, 0.7, 1.5))}


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["rows"] * case["cols"]
        scale = {"none": 0.0, "fp8": 1 + 4 / 128, "mxfp8": 1 + 1 / 32}[case["quant"]]
        per = 2 + (4 if case["residual"] else 0) + (2 if case["y"] else 0) + scale
        return {"bytes": n * per + 2 * case["cols"], "flops": 6 * n}
    if op == "act":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (4 + {"none": 2.0, "fp8": 1 + 4 / 128, "mxfp8": 1 + 1 / 32}[case["quant"]]), "flops": 8 * n}
    rows, n, k = case["rows"], case["n"], case["k"]
    if op == "dense":
        return {"bytes": rows * k * (1 + 4 / 128) + n * k + -(-n // 128) * (k // 128) * 4 + 2 * rows * n,
                "flops": 2 * rows * n * k}
    live = sum(1 for r in _group_rows(case, 0) if r)          # weights of experts without rows are not read
    fp8 = case["type"] == "fp8"
    wbytes = n * k * (1 if fp8 else 2) + (-(-n // 128) * (k // 128) * 4 if fp8 else 0)
    abytes = rows * k * (1 + 4 / 128 if fp8 else 2)
    return {"bytes": abytes + live * wbytes + 2 * rows * n + 4 * (case["experts"] + 1), "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ inputs ---

def _group_rows(case, seed):
    """Rows per expert: a multinomial over exp(skew * N(0, 1)) loads."""
    g = torch.Generator().manual_seed(7919 * int(seed) + 13)
    load = torch.softmax(case["skew"] * torch.randn(case["experts"], generator=g), 0)
    pick = torch.multinomial(load, case["rows"], replacement=True, generator=g)
    return torch.bincount(pick, minlength=case["experts"]).tolist()


def _act_codes(a):
    """E4M3 codes of bf16 activations with a power-of-two scale per row and 128 columns."""
    g = a.float().unflatten(-1, (-1, 128))
    s = _pow2_scale(g.abs().amax(-1))
    q = (g / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(-2)
    return q.to(torch.float8_e4m3fn), s


def _weight_codes(w):
    """E4M3 codes of bf16 weights [..., n, k] with an amax / 448 scale per 128 x 128 block."""
    *lead, n, k = w.shape
    pad = -n % 128
    wf = torch.nn.functional.pad(w.float(), (0, 0, 0, pad)).view(*lead, (n + pad) // 128, 128, k // 128, 128)
    s = (wf.abs().amax((-3, -1)) / E4M3_MAX).clamp_min(1e-12)
    q = (wf / s[..., :, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX).view(*lead, n + pad, k)
    return q[..., :n, :].to(torch.float8_e4m3fn).contiguous(), s


def prepare(case, seed):
    d = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=d).manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=d, dtype=torch.bfloat16)

    st = dict(case)
    op, rows = case["op"], case["rows"]
    if op in ("norm", "act"):
        cols = case["cols"]
        if op == "norm":
            # a residual stream several times the layer's own output, with a few large channels
            boost = 1 + 15 * (torch.rand(cols, generator=g, device=d) < 0.01)
            st["x"] = (0.5 * randn(rows, cols) * boost).bfloat16()
            st["residual"] = (2 * randn(rows, cols) * boost).bfloat16() if case["residual"] else None
            st["weight"] = (1 + 0.1 * randn(cols)).bfloat16()
            st["eps"] = 1e-6
            st["residual_out"] = torch.empty_like(st["x"]) if case["residual"] else None
            st["out"] = torch.empty_like(st["x"]) if case["y"] else None
        else:
            st["x"] = randn(rows, 2 * cols) * 2
            st["out"] = torch.empty(rows, cols, dtype=torch.bfloat16, device=d) if case["quant"] == "none" else None
        if case["quant"] != "none":
            mx = case["quant"] == "mxfp8"
            st["codes"] = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=d)
            st["scales"] = torch.empty(rows, cols // (32 if mx else 128), device=d,
                                       dtype=torch.uint8 if mx else torch.float32)
        return st
    n, k = case["n"], case["k"]
    a = randn(rows, k)
    w = (randn(n, k) if op == "dense" else randn(case["experts"], n, k)).mul_(k ** -0.5)
    if op == "dense" or case["type"] == "fp8":
        st["a"], st["a_scale"] = _act_codes(a)
        if op == "dense":
            st["w"], st["w_scale"] = _weight_codes(w)
        else:
            parts = [_weight_codes(w[i:i + 32]) for i in range(0, case["experts"], 32)]
            st["w"] = torch.cat([p[0].view(torch.uint8) for p in parts]).view(torch.float8_e4m3fn)
            st["w_scale"] = torch.cat([p[1] for p in parts])
    else:
        st["a"], st["w"], st["a_scale"], st["w_scale"] = a, w, None, None
    st["out"] = torch.empty(rows, n, dtype=torch.bfloat16, device=d)
    if op == "grouped":
        per = _group_rows(case, seed)
        st["offsets"] = torch.tensor([0] + per, device=d).cumsum(0).to(torch.int32)
        st["most"] = max(per)
    return st


# -------------------------------------------------------------- plain forms ---

def _pow2_scale(amax):
    """The smallest power of two >= max(amax, 1e-10) * fl32(1 / 448)."""
    raw = amax.clamp_min(1e-10) * torch.tensor(1 / E4M3_MAX, dtype=torch.float32, device=amax.device)
    # a carry out of the fraction bits steps to the next power of two
    return ((raw.view(torch.int32) + 0x7fffff) & 0x7f800000).view(torch.float32)


def _plain_quant(y, quant):
    group = 32 if quant == "mxfp8" else 128
    g = y.float().unflatten(-1, (-1, group))
    s = _pow2_scale(g.abs().amax(-1))
    codes = (g / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).flatten(-2).to(torch.float8_e4m3fn)
    if quant == "mxfp8":                                      # the E8M0 byte is the biased exponent
        s = (s.view(torch.int32) >> 23).to(torch.uint8)
    return codes, s


def _plain_norm(st):
    s = st["x"].float()
    if st["residual"] is not None:
        s = s + st["residual"].float()
    # 64 bits: the bf16 row and the codes are roundings of a long sum's result
    v = s.double()
    v = v * (1 / torch.sqrt(v.square().mean(-1, keepdim=True) + st["eps"])) * st["weight"].double()
    y = v.float().bfloat16()
    out = {"y": y} if st["out"] is not None else {}
    if st["residual"] is not None:
        out["residual_out"] = s.bfloat16()
    if st["quant"] != "none":
        out["codes"], out["scales"] = _plain_quant(y, st["quant"])
    return out


def _plain_act(st):
    gate, up = st["x"].float().chunk(2, -1)
    if st["clamp"] > 0:
        gate, up = gate.clamp_max(st["clamp"]), up.clamp(-st["clamp"], st["clamp"])
    gd = gate.double()                                        # 64 bits: bf16 borders, as in _plain_norm
    silu = (gd / (1 + torch.exp(-gd))).float().bfloat16().float()
    a = (silu * up).bfloat16()
    if st["quant"] == "none":
        return {"y": a}
    codes, scales = _plain_quant(a, st["quant"])
    return {"codes": codes, "scales": scales}


def _plain_values(codes, scale):
    return (codes.float().unflatten(-1, (-1, 128)) * scale[..., None]).flatten(-2)


def _plain_weights(w, scale):
    n, k = w.shape[-2:]
    full = scale.repeat_interleave(128, -2)[..., :n, :]
    return (w.float().unflatten(-1, (-1, 128)) * full[..., None]).flatten(-2)


def _plain_dense(st):
    a, w = _plain_values(st["a"], st["a_scale"]), _plain_weights(st["w"], st["w_scale"])
    return torch.mm(a, w.t()).bfloat16()


def _plain_grouped(st):
    off = st["offsets"].long()
    row = torch.arange(st["rows"], device=off.device)
    expert = torch.searchsorted(off, row, right=True) - 1     # the last expert starting at or before the row
    place = row - off[expert]
    fp8 = st["a_scale"] is not None
    a = _plain_values(st["a"], st["a_scale"]) if fp8 else st["a"].float()
    w = _plain_weights(st["w"], st["w_scale"]) if fp8 else st["w"].float()
    slab = torch.zeros(st["experts"], st["most"], st["k"], device=a.device)
    slab[expert, place] = a
    return torch.bmm(slab, w.transpose(1, 2).contiguous())[expert, place].bfloat16()


# --------------------------------------------------------------------- run ---

def _scale_values(scales):
    """E8M0 bytes as the float8 powers of two they stand for."""
    return scales.view(torch.float8_e8m0fnu) if scales.dtype == torch.uint8 else scales


def run(st):
    op = st["op"]
    if own:
        from moe_layer_amd import ops
        if op == "norm":
            quant = None if st["quant"] == "none" else st["quant"]
            y, res, codes, scales = ops.moe_rmsnorm(
                st["x"], st["weight"], st["eps"], residual=st["residual"], quant=quant, with_y=st["out"] is not None,
                y=st["out"], residual_out=st["residual_out"], codes=st.get("codes"), scales=st.get("scales"))
            out = {"y": y, "residual_out": res, "codes": codes, "scales": scales}
        elif op == "act":
            quant = None if st["quant"] == "none" else st["quant"]
            y, codes, scales = ops.moe_silu_mul(st["x"], quant=quant, clamp_limit=st["clamp"], y=st["out"],
                                                codes=st.get("codes"), scales=st.get("scales"))
            out = {"y": y, "codes": codes, "scales": scales}
        elif op == "dense":
            return ops.moe_gemm_fp8(st["a"], st["a_scale"], st["w"], st["w_scale"], out=st["out"])
        else:
            return ops.moe_grouped_gemm(st["a"], st["w"], st["offsets"], st["a_scale"], st["w_scale"], out=st["out"])
    else:
        out = {"norm": _plain_norm, "act": _plain_act, "dense": _plain_dense, "grouped": _plain_grouped}[op](st)
        if op in ("dense", "grouped"):
            return out
    out = {name: t for name, t in out.items() if t is not None}
    if "scales" in out:
        out["scales"] = _scale_values(out["scales"])
    return out


# ------------------------------------------------- the definitions in 64 bits ---

def _near_even(v, least, bits):
    """v to the grid of floats with ``bits`` fraction bits and least normal exponent ``least``, ties to even."""
    e = torch.frexp(v)[1].clamp_min(least + 1) - 1
    step = ((e - bits + 1023).long() << 52).view(torch.float64)   # 2^(e - bits), exact
    return torch.round(v / step) * step


def _exact_codes(v, quant):
    rows, cols = v.shape
    width = 32 if quant == "mxfp8" else 128
    v = v.reshape(rows, cols // width, width)
    least = v.abs().max(-1).values.clamp_min(1e-10) / E4M3_MAX
    mant, e = torch.frexp(least)                              # least = mant 2^e, mant in [1/2, 1)
    scale = ((e - (mant == 0.5).int() + 1023).long() << 52).view(torch.float64)
    codes = _near_even((v / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX), -6, 3)
    return codes.reshape(rows, cols), scale


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = st["x"].to(torch.float64)
        if st["residual"] is not None:
            v += st["residual"]
        total = v.clone()
        power = torch.einsum("rc,rc->r", v, v) / case["cols"]
        v = v * torch.rsqrt(power + st["eps"])[:, None] * st["weight"].to(torch.float64)
        out = {"y": v} if case["y"] else {}
        if case["residual"]:
            out["residual_out"] = total
        if case["quant"] != "none":
            out["codes"], out["scales"] = _exact_codes(_near_even(v, -126, 7), case["quant"])
        return out
    if op == "act":
        cols = case["cols"]
        gate, up = st["x"][:, :cols].to(torch.float64), st["x"][:, cols:].to(torch.float64)
        if case["clamp"] > 0:
            gate, up = gate.minimum(torch.full_like(gate, case["clamp"])), up.clamp(-case["clamp"], case["clamp"])
        v = _near_even(gate * torch.sigmoid(gate), -126, 7) * up
        if case["quant"] == "none":
            return {"y": v}
        codes, scales = _exact_codes(_near_even(v, -126, 7), case["quant"])
        return {"codes": codes, "scales": scales}

    def product(a, a_scale, w, w_scale):
        a, w = a.to(torch.float64), w.to(torch.float64)
        if a_scale is not None:
            a = a * a_scale.to(torch.float64).repeat_interleave(128, 1)
            blocks = torch.kron(w_scale.to(torch.float64), torch.ones(128, 128, dtype=torch.float64, device=w.device))
            w = w * blocks[: w.shape[0]]
        return a @ w.T

    if op == "dense":
        return product(st["a"], st["a_scale"], st["w"], st["w_scale"])
    off = st["offsets"].tolist()
    out = torch.empty(case["rows"], case["n"], dtype=torch.float64, device=st["a"].device)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if hi > lo:
            fp8 = case["type"] == "fp8"
            out[lo:hi] = product(st["a"][lo:hi], st["a_scale"][lo:hi] if fp8 else None, st["w"][e],
                                 st["w_scale"][e] if fp8 else None)
    return out
