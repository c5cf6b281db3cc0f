"""Timing cases of the feed-forward half that follows wo_b and its norm, on e4m3 codes with block scales: the product with
bias, activation and residual in its epilogue (gemm_blockscale_act) and its backward pass, and the experts' layer for a
few tokens (moe_route, moe_apply).

`run` computes a case with the library's entry points where `own` is true, and with elementary torch operations in
fp32 where it is not.  `exact` computes the definition in fp64.
"""
import math

import torch

own = False

#: Width of the residual stream (wo_b's N), and the width between the two products (one K-slice of wo_b).
HIDDEN, INNER = 7168, 2048
F8_MAX = 448.0
#: Most rows of a call (the context's), and most tokens of the experts' layer.
ROWS, FEW = 16384, 128


def listed():
    act = {"op": "act", "M": 1, "N": INNER, "K": HIDDEN, "act": "silu", "gated": True, "bias": False, "res": "none", "out": "codes", "keep": False}
    bwd = {"op": "act_bwd", "M": 4096, "N": INNER, "act": "silu", "gated": True, "bias": False, "d32": False, "out": "both"}
    route = {"op": "route", "T": 1, "H": HIDDEN, "E": 64, "k": 8, "score": "softmax", "bias": False, "w32": False}
    moe = {"op": "moe", "T": 1, "H": HIDDEN, "I": INNER, "E": 64, "k": 8, "score": "softmax", "bias": False, "w32": False, "away": 0.0, "y": True}
    return [
        # one decoded token through the gated up-projection, codes for the down-projection: the weights are read once
        {**act, "name": "act_decode_1"},
        # the down-projection of a decode batch, joined with the residual stream
        {**act, "name": "act_decode_48", "M": 48, "N": HIDDEN, "K": INNER, "act": "none", "gated": False, "res": "bf16", "out": "bf16"},
        # a training step's forward pass at prefill size: the pre-activations are kept
        {**act, "name": "act_prefill_4096", "M": 4096, "keep": True},
        # the full chunk's down-projection with a bias and the residual stream
        {**act, "name": "act_chunk_16384", "M": 16384, "N": HIDDEN, "K": INNER, "act": "none", "gated": False, "bias": True, "res": "bf16", "out": "bf16"},
        # a ragged batch of an ungated layer, an odd number of 128-column blocks, fp32 stream
        {**act, "name": "act_ragged_531", "M": 531, "N": 1920, "K": 1152, "act": "gelu", "gated": False, "bias": True, "res": "fp32", "out": "fp32"},
        # the gated activation's backward pass at prefill size: rows for the adapters, codes for the input's gradient
        {**bwd, "name": "act_bwd_4096"},
        # a ragged batch, an ungated layer with a bias, an fp32 gradient
        {**bwd, "name": "act_bwd_ragged_1531", "M": 1531, "N": 1920, "act": "gelu", "gated": False, "bias": True, "d32": True, "out": "bf16"},
        # one token's choice of experts: latency
        {**route, "name": "route_1"},
        # a decode batch's choice among many experts, scored apart and chosen with a balancing bias
        {**route, "name": "route_96", "T": 96, "E": 256, "score": "sigmoid", "bias": True, "w32": True},
        # one token's layer: the weights of eight experts are read
        {**moe, "name": "moe_1"},
        # a small model, a ragged batch, some experts on another GPU
        {**moe, "name": "moe_23", "T": 23, "H": 2944, "I": 1152, "E": 20, "k": 3, "away": 0.25, "y": False},
        # a decode batch that meets nearly every expert
        {**moe, "name": "moe_96", "T": 96, "E": 128, "score": "sigmoid", "bias": True, "w32": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 3.8e15)


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), _cost(c))
    while True:
        op = rng.choice(["act", "act", "act_bwd", "route", "moe"])
        if op.startswith("act"):
            c = {"op": op, "M": _log(rng, 1, ROWS), "N": 128 * _log(rng, 1, HIDDEN // 128), "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                 "gated": rng.random() < 0.5, "bias": rng.random() < 0.5}
            if op == "act":
                c.update(K=128 * _log(rng, 1, HIDDEN // 128), res=rng.choice(["none", "bf16", "fp32"]), out=rng.choice(["bf16", "fp32", "codes", "both"]), keep=rng.random() < 0.3)
            else:
                c.update(d32=rng.random() < 0.3, out=rng.choice(["bf16", "codes", "both"]))
        else:
            E = _log(rng, 4, 256)
            c = {"op": op, "T": _log(rng, 1, FEW), "H": 128 * _log(rng, 2, HIDDEN // 128), "E": E, "k": rng.randint(1, min(8, E)),
                 "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "w32": rng.random() < 0.5}
            if op == "moe":
                c.update(I=128 * _log(rng, 1, INNER // 128), away=rng.choice([0.0, 0.25, 0.75]), y=rng.random() < 0.5)
        if _cost(c) <= most[op]:
            return c


def work(case):
    c = case
    if c["op"] == "act":
        M, N, K = c["M"], c["N"], c["K"]
        P = 2 * N if c["gated"] else N
        out = {"bf16": 2, "fp32": 4, "codes": 1 + 4 / 128, "both": 3 + 4 / 128}[c["out"]] + {"none": 0, "bf16": 2, "fp32": 4}[c["res"]]
        return {"bytes": M * K * (1 + 4 / 128) + P * K * (1 + 4 / 128 ** 2) + M * N * out + (2 * M * P if c["keep"] else 0) + (4 * P if c["bias"] else 0),
                "flops": 2.0 * M * P * K + 8.0 * M * P}
    if c["op"] == "act_bwd":
        M, N = c["M"], c["N"]
        P = 2 * N if c["gated"] else N
        out = {"bf16": 2, "codes": 1 + 4 / 128, "both": 3 + 4 / 128}[c["out"]]
        return {"bytes": M * N * (4 if c["d32"] else 2) + M * P * (2 + out) + (4 * P if c["bias"] else 0), "flops": 12.0 * M * P}
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    route = {"bytes": E * H * (4 if c["w32"] else 2) + T * H * 2 + 8 * T * k + (4 * E if c["bias"] else 0), "flops": 2.0 * T * E * H}
    if c["op"] == "route":
        return route
    picks = T * k * (1.0 - c["away"])
    # experts that get a token, on average, and their two products
    used = E * (1.0 - (1.0 - (1.0 - c["away"]) * k / E) ** T)
    weights = 3 * H * c["I"] * (1 + 4 / 128 ** 2)
    return {"bytes": route["bytes"] + used * weights + T * H * (1 + 4 / 128 + 2 + (2 if c["y"] else 0)), "flops": route["flops"] + 6.0 * picks * H * c["I"]}


_handle = None


def _context():
    """The library's context, kept by a program for all its calls."""
    global _handle
    if _handle is None:
        import block_scaled_fp8_gemm_gb300 as g
        _handle = g.gemmar_create(torch.cuda.current_device(), ROWS, HIDDEN, INNER, 1, flags=g.GEMMAR_NO_SELF_TEST)
    return _handle


def _codes_1x128(x):
    """Codes and scales of activations, one scale per row and 128 columns."""
    groups = x.view(x.shape[0], -1, 128)
    scales = groups.abs().amax(2) / F8_MAX
    return (groups / scales[..., None]).view(x.shape).to(torch.float8_e4m3fn).view(torch.uint8), scales.contiguous()


def _codes_128x128(w):
    """Codes and scales of a weight, one scale per block of 128 rows and 128 columns."""
    blocks = w.view(w.shape[0] // 128, 128, w.shape[1] // 128, 128)
    scales = blocks.abs().amax((1, 3)) / F8_MAX
    return (blocks / scales[:, None, :, None]).view(w.shape).to(torch.float8_e4m3fn).view(torch.uint8), scales.contiguous()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed * 65537 + 1)
    c = case

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    s = {"case": case, "ctx": _context() if own else None}   # only the handle goes by `own`
    if c["op"] == "act":
        M, N, K = c["M"], c["N"], c["K"]
        P = 2 * N if c["gated"] else N
        s["A"], s["sa"] = _codes_1x128(normal(M, K))
        s["B"], s["sb"] = _codes_128x128(normal(P, K, scale=1.5 * K ** -0.5))
        s["bias"] = normal(P, scale=0.3) if c["bias"] else None
        s["res"] = None if c["res"] == "none" else normal(M, N, scale=2.0).to(torch.bfloat16 if c["res"] == "bf16" else torch.float32)
        return s
    if c["op"] == "act_bwd":
        M, N = c["M"], c["N"]
        s["z"] = normal(M, 2 * N if c["gated"] else N, scale=1.5).bfloat16()
        s["dout"] = normal(M, N).to(torch.float32 if c["d32"] else torch.bfloat16)
        return s
    T, H, E = c["T"], c["H"], c["E"]
    # the router sees the norm's rows, the experts their codes
    rows = normal(T, H)
    s["x"] = rows.bfloat16()
    s["router"] = normal(E, H, scale=H ** -0.5).to(torch.float32 if c["w32"] else torch.bfloat16)
    s["bias"] = normal(E, scale=0.1) if c["bias"] else None
    if c["op"] == "moe":
        inner = c["I"]
        s["q"], s["sx"] = _codes_1x128(rows)
        s["w13"] = torch.empty(E, 2 * inner, H, dtype=torch.uint8, device="cuda")
        s["s13"] = torch.empty(E, 2 * inner // 128, H // 128, device="cuda")
        s["w2"] = torch.empty(E, H, inner, dtype=torch.uint8, device="cuda")
        s["s2"] = torch.empty(E, H // 128, inner // 128, device="cuda")
        for e in range(E):
            s["w13"][e], s["s13"][e] = _codes_128x128(normal(2 * inner, H, scale=1.5 * H ** -0.5))
            s["w2"][e], s["s2"][e] = _codes_128x128(normal(H, inner, scale=inner ** -0.5))
        s["y"] = normal(T, H).bfloat16() if c["y"] else None
        # this GPU's number of each expert: -1 for those of another one
        s["place"] = torch.arange(E, dtype=torch.int32, device="cuda")
        s["place"][torch.rand(E, generator=gen, device="cuda") < c["away"]] = -1
    return s


# ---------------------------------------------------------------- plain forms

def _plain_rows(q, scales):
    return (q.view(torch.float8_e4m3fn).float().view(*scales.shape, 128) * scales[..., None]).view(q.shape)


def _plain_weight(q, scales):
    blocks = q.view(torch.float8_e4m3fn).float().view(*scales.shape[:-1], 128, scales.shape[-1], 128)
    return (blocks * scales[..., :, None, :, None]).view(q.shape)


def _erf(x):
    return torch.erf(x * 0.7071067811865476)


def _plain_act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + _erf(z))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    return z


def _plain_slope(name, z):
    if name == "relu":
        return (z > 0).float()
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + _erf(z)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    if name == "gelu_tanh":
        t = torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * 0.7978845608028654 * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_codes(x):
    scales = x.view(x.shape[0], -1, 128).abs().amax(2) / F8_MAX
    groups = x.view(x.shape[0], -1, 128)
    codes = torch.where(scales[..., None] > 0, groups / scales[..., None], torch.zeros_like(groups))
    return codes.view(x.shape).to(torch.float8_e4m3fn), scales


def _plain_gemm_act(s):
    c = s["case"]
    z = _plain_rows(s["A"], s["sa"]) @ _plain_weight(s["B"], s["sb"]).T
    if c["bias"]:
        z = z + s["bias"]
    out = {"z": z.bfloat16()} if c["keep"] else {}
    a = _plain_act(c["act"], z[:, :c["N"]]) * z[:, c["N"]:] if c["gated"] else _plain_act(c["act"], z)
    if c["res"] != "none":
        a = s["res"].float() + a
    if c["out"] in ("codes", "both"):
        out["q"], out["scales"] = _plain_codes(a)
    if c["out"] != "codes":
        out["C"] = a if c["out"] == "fp32" else a.bfloat16()
    return out


def _plain_act_bwd(s):
    c = s["case"]
    z, d = s["z"].float(), s["dout"].float()
    if c["gated"]:
        gate, up = z[:, :c["N"]], z[:, c["N"]:]
        dz = torch.cat([d * up * _plain_slope(c["act"], gate), d * _plain_act(c["act"], gate)], 1)
    else:
        dz = d * _plain_slope(c["act"], z)
    out = {"dbias": dz.sum(0)} if c["bias"] else {}
    if c["out"] in ("codes", "both"):
        out["q"], out["scales"] = _plain_codes(dz)
    if c["out"] != "codes":
        out["dz"] = dz.bfloat16()
    return out


def _plain_route(s):
    c = s["case"]
    # 64 bits: which expert comes next hangs on the last digits of a score
    logits = s["x"].double() @ s["router"].double().T
    if c["score"] == "softmax":
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-logits))
    by = p + s["bias"].double() if c["bias"] else p
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = torch.gather(p, 1, ids)
    return {"ids": ids.to(torch.int32), "weights": (w / w.sum(1, keepdim=True)).float()}


def _plain_moe(s):
    c = s["case"]
    out = _plain_route(s)
    x = _plain_rows(s["q"], s["sx"])
    total = s["y"].float() if c["y"] else torch.zeros_like(x)
    for j in range(c["k"]):
        # each token's expert, one of its k at a time
        e = s["place"][out["ids"][:, j].long()].long()
        w = torch.where(e >= 0, out["weights"][:, j], torch.zeros_like(out["weights"][:, j]))
        e = e.clamp(min=0)
        for t in range(0, c["T"], 16):
            p = e[t:t + 16]
            z = (_plain_weight(s["w13"][p], s["s13"][p]) @ x[t:t + 16, :, None])[..., 0]
            h = _plain_act("silu", z[:, :c["I"]]) * z[:, c["I"]:]
            total[t:t + 16] += w[t:t + 16, None] * (_plain_weight(s["w2"][p], s["s2"][p]) @ h[:, :, None])[..., 0]
    return {**out, "out": total.bfloat16()}


# ---------------------------------------------------------------- the library's calls

_ACTS = {"none": "GEMMAR_ACT_NONE", "relu": "GEMMAR_ACT_RELU", "silu": "GEMMAR_ACT_SILU", "gelu": "GEMMAR_ACT_GELU", "gelu_tanh": "GEMMAR_ACT_GELU_TANH"}


def _own_codes(M, N):
    return torch.empty(M, N, dtype=torch.uint8, device="cuda"), torch.empty(M, N // 128, device="cuda")


def _own_gemm_act(g, s):
    c, M, N = s["case"], s["case"]["M"], s["case"]["N"]
    q, scales = _own_codes(M, N) if c["out"] in ("codes", "both") else (None, None)
    C = None if c["out"] == "codes" else torch.empty(M, N, dtype=torch.float32 if c["out"] == "fp32" else torch.bfloat16, device="cuda")
    z = torch.empty(M, s["B"].shape[0], dtype=torch.bfloat16, device="cuda") if c["keep"] else None
    g.gemm_blockscale_act(s["ctx"], s["A"], s["sa"], s["B"], s["sb"], C, act=getattr(g, _ACTS[c["act"]]), gated=c["gated"], bias=s["bias"],
                          residual=s["res"], q=q, scales=scales, z=z)
    out = {"z": z, "q": None if q is None else q.view(torch.float8_e4m3fn), "scales": scales, "C": C}
    return {name: t for name, t in out.items() if t is not None}


def _own_act_bwd(g, s):
    c, (M, P) = s["case"], s["z"].shape
    dz = None if c["out"] == "codes" else torch.empty(M, P, dtype=torch.bfloat16, device="cuda")
    q, scales = _own_codes(M, P) if c["out"] in ("codes", "both") else (None, None)
    dbias = torch.empty(P, device="cuda") if c["bias"] else None
    g.gemm_blockscale_act_bwd(s["ctx"], s["dout"], s["z"], dz, act=getattr(g, _ACTS[c["act"]]), gated=c["gated"], dbias=dbias, q=q, scales=scales)
    out = {"dbias": dbias, "q": None if q is None else q.view(torch.float8_e4m3fn), "scales": scales, "dz": dz}
    return {name: t for name, t in out.items() if t is not None}


def _own_route(g, s):
    c = s["case"]
    ids = torch.empty(c["T"], c["k"], dtype=torch.int32, device="cuda")
    weights = torch.empty(c["T"], c["k"], device="cuda")
    g.moe_route(s["ctx"], s["x"], s["router"], ids, weights, bias=s["bias"], score=g.GEMMAR_SCORE_SOFTMAX if c["score"] == "softmax" else g.GEMMAR_SCORE_SIGMOID,
                renorm=True)
    return {"ids": ids, "weights": weights}


def _own_moe(g, s):
    out = _own_route(g, s)
    out["out"] = torch.empty(s["q"].shape, dtype=torch.bfloat16, device="cuda")
    g.moe_apply(s["ctx"], s["q"], s["sx"], out["ids"], out["weights"], s["w13"], s["s13"], s["w2"], s["s2"], out["out"], act=g.GEMMAR_ACT_SILU,
                place=s["place"], y=s["y"])
    return out


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"act": _plain_gemm_act, "act_bwd": _plain_act_bwd, "route": _plain_route, "moe": _plain_moe}[op](state)
    import block_scaled_fp8_gemm_gb300 as g
    return {"act": _own_gemm_act, "act_bwd": _own_act_bwd, "route": _own_route, "moe": _own_moe}[op](g, state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _table():
    """The value of each e4m3 code."""
    values = []
    for code in range(256):
        exponent, fraction = (code >> 3) & 15, code & 7
        v = (fraction / 8) * 2.0 ** -6 if exponent == 0 else (1 + fraction / 8) * 2.0 ** (exponent - 7)
        values.append(math.nan if code & 127 == 127 else -v if code & 128 else v)
    return torch.tensor(values, dtype=torch.float64, device="cuda")


def _decode(codes, scales, rows):
    """Values of codes under scales of `rows` x 128."""
    v = _table()[codes.int()]
    for j in range(codes.shape[1] // 128):
        v[:, 128 * j:128 * j + 128] *= scales[:, j].double().repeat_interleave(rows)[:, None]
    return v


def _value(name, z):
    """act(z), in place."""
    if name == "relu":
        return z.clamp_(min=0)
    if name == "silu":
        return z.mul_(torch.sigmoid(z))
    if name == "gelu":
        return z.mul_(torch.special.ndtr(z))
    if name == "gelu_tanh":
        # (1 + tanh u) / 2 = sigmoid(2 u)
        return z.mul_(torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def _grouped(out, x):
    # a code stands for the value before its rounding, in units of its group's scale
    scales = x.view(x.shape[0], -1, 128).abs().max(2).values / F8_MAX
    units = torch.where(scales > 0, 1 / scales, torch.zeros_like(scales))
    return {**out, "scales": scales, "q": (x.view(*scales.shape, 128) * units[..., None]).view(x.shape)}


def _exact_act(c, s):
    N = c["N"]
    z = torch.matmul(_decode(s["A"], s["sa"], 1), _decode(s["B"], s["sb"], 128).T)
    if c["bias"]:
        z += s["bias"].double()
    out = {"z": z.clone()} if c["keep"] else {}
    a = _value(c["act"], z[:, :N].contiguous())
    if c["gated"]:
        a.mul_(z[:, N:])
    if c["res"] != "none":
        a.add_(s["res"].double())
    if c["out"] != "codes":
        out["C"] = a
    return _grouped(out, a) if c["out"] in ("codes", "both") else out


def _exact_act_bwd(c, s):
    # by torch's own differentiation of the forward definition, in rows that fit
    parts = []
    for z, d in zip(s["z"].split(2048), s["dout"].split(2048)):
        leaf = z.double().requires_grad_()
        if c["gated"]:
            a, b = leaf.split(c["N"], 1)
        else:
            a, b = leaf, 1.0
        if c["act"] == "relu":
            v = torch.relu(a)
        elif c["act"] == "silu":
            v = a * torch.sigmoid(a)
        elif c["act"] == "gelu":
            v = a * 0.5 * torch.erfc(-a * math.sqrt(0.5))
        elif c["act"] == "gelu_tanh":
            v = a * torch.sigmoid(math.sqrt(8 / math.pi) * (a + 0.044715 * a ** 3))
        else:
            v = a * 1.0
        parts.append(torch.autograd.grad(v * b, leaf, d.double())[0])
    dz = torch.cat(parts)
    out = {"dbias": dz.sum(0)} if c["bias"] else {}
    if c["out"] != "codes":
        out["dz"] = dz
    return _grouped(out, dz) if c["out"] in ("codes", "both") else out


def _exact_route(c, s):
    logits = torch.einsum("th,eh->te", s["x"].double(), s["router"].double())
    p = torch.softmax(logits, 1) if c["score"] == "softmax" else torch.sigmoid(logits)
    by = p + (s["bias"].double() if c["bias"] else 0.0)
    ids, at = [], torch.arange(c["T"], device="cuda")
    for _ in range(c["k"]):
        # the first of the largest, then without it
        best = (by == by.amax(1, keepdim=True)).int().argmax(1)
        ids.append(best)
        by[at, best] = -math.inf
    ids = torch.stack(ids, 1)
    w = p.gather(1, ids)
    return {"ids": ids.to(torch.int32), "weights": w / w.sum(1)[:, None]}


def _exact_moe(c, s):
    out = _exact_route(c, s)
    total = s["y"].double() if c["y"] else torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    x = _decode(s["q"], s["sx"], 1)
    place = s["place"].tolist()
    for e in range(c["E"]):
        t, j = (out["ids"] == e).nonzero(as_tuple=True)
        here = place[e]
        if len(t) and here >= 0:
            z = x[t] @ _decode(s["w13"][here], s["s13"][here], 128).T
            h = _value("silu", z[:, :c["I"]].contiguous()) * z[:, c["I"]:]
            total[t] += out["weights"][t, j][:, None] * (h @ _decode(s["w2"][here], s["s2"][here], 128).T)
    return {**out, "out": total}


def exact(case, seed):
    s = prepare(case, seed)
    return {"act": _exact_act, "act_bwd": _exact_act_bwd, "route": _exact_route, "moe": _exact_moe}[case["op"]](case, s)
