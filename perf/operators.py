"""Timing cases of the operators around the wo_b projection: the norms and residual that follow it
(norm_gate_residual and its backward pass) and the low-rank adapters beside it (lora_apply and its backward pass).

`run` computes a case with the library's entry points where `own` is true, and with elementary torch operations in
fp32 where it is not.  `exact` computes the definition in fp64.
"""
import math

import torch

own = False

#: Row width and reduction lengths of wo_b: N = 7168, 2048 per K-slice, eight slices.
N_WO, K_SLICE, K_ALL = 7168, 2048, 16384
F8_MAX = 448.0


def listed():
    norm = {"op": "norm", "M": 1, "N": N_WO, "post": True, "gate": "row", "h32": False, "quant": True, "alpha": 1.0, "beta": 1.0}
    nbwd = {"op": "norm_bwd", "M": 4096, "N": N_WO, "post": True, "gate": "row", "h32": False, "alpha": 1.0, "beta": 1.0}
    lora = {"op": "lora", "T": 64, "K": K_SLICE, "N": N_WO, "R": 8, "r": 16, "spread": False, "bare": 0.0}
    lbwd = {"op": "lora_bwd", "T": 4096, "K": K_SLICE, "N": N_WO, "R": 4, "r": 16, "spread": False, "bare": 0.0}
    return [
        # one decoded token after wo_b: latency is all there is
        {**norm, "name": "norm_decode_1"},
        # a decode batch without a post norm (add, norm, quantise)
        {**norm, "name": "norm_decode_96", "M": 96, "post": False, "gate": "none"},
        # a prefill of wo_b's 4096 rows with an fp32 residual stream, codes for the next block-scaled GEMM
        {**norm, "name": "norm_prefill_4096", "M": 4096, "h32": True, "alpha": 0.5},
        # the full chunk of 16384 rows with a gate per token, bf16 rows for the next layer
        {**norm, "name": "norm_chunk_16384", "M": 16384, "gate": "token", "quant": False, "beta": 0.25},
        # a training step's backward pass at prefill size, a learned gate row
        {**nbwd, "name": "norm_bwd_4096"},
        # a ragged batch, width off the 128 grid, gate per token, fp32 residual
        {**nbwd, "name": "norm_bwd_ragged", "M": 1531, "N": 2056, "gate": "token", "h32": True, "alpha": 0.7},
        # one decoded token with an adapter on one K-slice
        {**lora, "name": "lora_decode_1", "T": 1, "R": 4},
        # a decode batch, tokens of 48 adapters in any order, a few without one, whole attention output
        {**lora, "name": "lora_decode_96", "T": 96, "K": K_ALL, "R": 48, "spread": True, "bare": 0.1},
        # a prefill of requests of uneven lengths
        {**lora, "name": "lora_prefill_4096", "T": 4096, "R": 6, "r": 32},
        # the full chunk, whole attention output, large odd-sized ranks, some requests without an adapter
        {**lora, "name": "lora_chunk_16384", "T": 16384, "K": K_ALL, "R": 7, "r": 64, "bare": 0.1},
        # training a few adapters at once on one K-slice
        {**lbwd, "name": "lora_bwd_4096"},
        # training more, larger ones on the whole attention output, tokens mixed
        {**lbwd, "name": "lora_bwd_8191", "T": 8191, "K": K_ALL, "R": 9, "r": 64, "spread": True, "bare": 0.05},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["norm", "norm_bwd", "lora", "lora_bwd"])
        if op.startswith("norm"):
            c = {"op": op, "M": _log(rng, 1, 16384), "N": 8 * _log(rng, 16, N_WO // 8), "post": rng.random() < 0.6,
                 "gate": rng.choice(["none", "row", "token"]), "h32": rng.random() < 0.4, "alpha": rng.choice([1.0, 0.5, 0.7071]), "beta": rng.choice([1.0, 0.25])}
            if op == "norm":
                c["quant"] = rng.random() < 0.5
                if c["quant"]:
                    c["N"] = 128 * max(1, c["N"] // 128)
        else:
            c = {"op": op, "T": _log(rng, 1, 16384), "K": 8 * _log(rng, 32, K_ALL // 8), "N": 8 * _log(rng, 32, N_WO // 8),
                 "R": _log(rng, 1, 64), "r": _log(rng, 4, 64), "spread": rng.random() < 0.5, "bare": rng.choice([0.0, 0.1, 0.5])}
        if work(c)["bytes"] <= most:
            return c


def work(case):
    c = case
    if c["op"] in ("norm", "norm_bwd"):
        M, N, hb = c["M"], c["N"], 4 if c["h32"] else 2
        token = 2 if c["gate"] == "token" else 0
        row = 2 * N if c["gate"] == "row" else 0
        weights = N * 4 * (2 if c["post"] else 1) + row
        if c["op"] == "norm":
            out = hb + (1 + 4 / 128 if c["quant"] else 2)
            return {"bytes": M * N * (2 + hb + token + out) + weights + 8 * M, "flops": 14.0 * M * N}
        return {"bytes": M * N * (2 + hb + 2 + hb + 2 + hb + 2 * token) + 2 * weights + row + 8 * M, "flops": 36.0 * M * N}
    T, K, N, R, r = c["T"], c["K"], c["N"], c["R"], c["r"]
    tokens = T * (1 - c["bare"])
    used = min(R, max(1, int(round(tokens)))) if c["spread"] or T < R else R
    weights = used * r * (K + N) * 2
    if c["op"] == "lora":
        return {"bytes": tokens * 2 * K + T * 4 * N + weights + 4 * T * (1 + r), "flops": 2.0 * tokens * r * (K + N)}
    return {"bytes": tokens * (2 * K + 2 * N) + T * 4 * K + weights + R * r * (K + N) * 2 + 4 * T * (1 + r), "flops": 4.0 * tokens * r * (K + N)}


_handle = None


def _context():
    """The library's context, kept by a program for all its calls."""
    global _handle
    if _handle is None:
        import block_scaled_fp8_gemm_gb300 as g
        _handle = g.gemmar_create(torch.cuda.current_device(), 16384, N_WO, K_SLICE, 1, flags=g.GEMMAR_NO_SELF_TEST)
    return _handle


def _assignment(case, seed):
    """Adapter of each token (-1: none), and the tokens in the order of their adapters with each adapter's offsets."""
    T, R = case["T"], case["R"]
    gen = torch.Generator().manual_seed(seed * 7919 + 17)
    if case["spread"]:
        ids = torch.randint(0, R, (T,), generator=gen)
        ids[torch.rand(T, generator=gen) < case["bare"]] = -1
    else:
        # whole requests of uneven lengths, one after another
        cuts = torch.sort(torch.randint(0, T + 1, (2 * R - 1,), generator=gen)).values
        ids = torch.randint(0, R, (2 * R,), generator=gen)[torch.searchsorted(cuts, torch.arange(T), right=True)]
        if case["bare"]:
            ids[torch.arange(T) >= T - int(T * case["bare"])] = -1
    key = torch.where(ids < 0, torch.full_like(ids, R), ids)
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[order].contiguous(), torch.arange(R + 1))
    return ids.cuda(), order.to(torch.int32).cuda(), offsets.to(torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed * 65537 + 1)

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    s = {"case": case, "ctx": _context() if own else None}   # only the handle goes by `own`
    if case["op"] in ("norm", "norm_bwd"):
        M, N = case["M"], case["N"]
        s["y"] = normal(M, N, scale=3.0).bfloat16()
        s["h"] = normal(M, N, scale=2.0).to(torch.float32 if case["h32"] else torch.bfloat16)
        s["w_post"] = 1.0 + normal(N, scale=0.2) if case["post"] else None
        s["w_pre"] = 1.0 + normal(N, scale=0.2)
        s["gate"] = {"none": None, "row": lambda: normal(N, scale=0.5).bfloat16(), "token": lambda: torch.sigmoid(normal(M, N)).bfloat16()}[case["gate"]]
        s["gate"] = s["gate"]() if s["gate"] else None
        s["eps"] = 1e-6
        if case["op"] == "norm_bwd":
            s["du"] = normal(M, N).bfloat16()
            s["dt"] = normal(M, N).to(s["h"].dtype)
            # the forward pass's reciprocal norms, kept for the backward pass
            y, h = s["y"].float(), s["h"].float()
            r1 = torch.rsqrt(y.square().mean(1, keepdim=True) + s["eps"]) if case["post"] else torch.ones(M, 1, device="cuda")
            z = y * r1 * s["w_post"] if case["post"] else y
            t = case["alpha"] * h + case["beta"] * (z if s["gate"] is None else z * s["gate"].float())
            s["rstd"] = torch.cat([r1, torch.rsqrt(t.square().mean(1, keepdim=True) + s["eps"])], 1).contiguous()
        return s
    T, K, N, R, r = (case[k] for k in "TKNRr")
    s["ids"], s["order"], s["offsets"] = _assignment(case, seed)
    s["A"] = normal(R, r, K, scale=K ** -0.5).bfloat16()
    s["B"] = normal(R, r, N, scale=0.3).bfloat16()
    s["scales"] = 0.25 + torch.rand(R, generator=gen, device="cuda")
    s["ranks"] = torch.randint((r + 1) // 2, r + 1, (R,), generator=gen, device="cuda", dtype=torch.int32)
    s["ranks"][0] = r
    s["x"] = normal(T, K).bfloat16()
    if case["op"] == "lora":
        s["y"] = normal(T, N).bfloat16()
    else:
        s["dy"] = normal(T, N).bfloat16()
        s["dx0"] = normal(T, K).bfloat16()
        # v as the forward pass left it: row i belongs to token order[i]
        v = torch.zeros(T, r, device="cuda")
        at = s["offsets"].tolist()
        for a in range(R):
            v[at[a]:at[a + 1]] = s["x"][s["order"][at[a]:at[a + 1]].long()].float() @ s["A"][a].float().T
        s["v"] = v
    return s


# ---------------------------------------------------------------- plain forms

def _plain_norm(s):
    c = s["case"]
    y, h = s["y"].float(), s["h"].float()
    r1 = torch.rsqrt(y.square().mean(1, keepdim=True) + s["eps"]) if c["post"] else torch.ones(c["M"], 1, device="cuda")
    z = y * r1 * s["w_post"] if c["post"] else y
    if s["gate"] is not None:
        z = z * s["gate"].float()
    t = c["alpha"] * h + c["beta"] * z
    r2 = torch.rsqrt(t.square().mean(1, keepdim=True) + s["eps"])
    u = t * r2 * s["w_pre"]
    out = {"t": t.to(s["h"].dtype), "rstd": torch.cat([r1, r2], 1)}
    if not c["quant"]:
        out["u"] = u.bfloat16()
        return out
    grouped = u.view(c["M"], -1, 128)
    scales = grouped.abs().amax(2) / F8_MAX
    codes = torch.where(scales[..., None] > 0, grouped / scales[..., None], torch.zeros_like(grouped))
    return {**out, "q": codes.view(c["M"], -1).to(torch.float8_e4m3fn), "scales": scales}


def _plain_norm_bwd(s):
    c = s["case"]
    y, h, du, dt = s["y"].float(), s["h"].float(), s["du"].float(), s["dt"].float()
    r1, r2 = s["rstd"][:, :1], s["rstd"][:, 1:]
    yhat = y * r1
    w1 = s["w_post"] if c["post"] else torch.ones(c["N"], device="cuda")
    g = s["gate"].float() if s["gate"] is not None else torch.ones(c["N"], device="cuda")
    t = c["alpha"] * h + c["beta"] * (g * (yhat * w1))
    that = t * r2
    dv = du * s["w_pre"]
    dt = dt + r2 * (dv - that * (dv * that).mean(1, keepdim=True))
    dz = c["beta"] * g * dt
    dn = dz * w1
    out = {"dh": (c["alpha"] * dt).to(s["h"].dtype), "dw_pre": (du * that).sum(0)}
    if c["post"]:
        out["dy"] = (r1 * (dn - yhat * (dn * yhat).mean(1, keepdim=True))).bfloat16()
        out["dw_post"] = (dz * yhat).sum(0)
    else:
        out["dy"] = dn.bfloat16()
    if c["gate"] == "row":
        out["dgate"] = (c["beta"] * yhat * w1 * dt).sum(0)
    elif c["gate"] == "token":
        out["dgate"] = (c["beta"] * yhat * w1 * dt).bfloat16()
    return out


def _chosen(s):
    """[T, R, r]: whether row j of adapter a is the token's."""
    R, r = s["case"]["R"], s["case"]["r"]
    return (s["ids"][:, None] == torch.arange(R, device="cuda"))[:, :, None] & (torch.arange(r, device="cuda") < s["ranks"][:, None])[None]


def _plain_lora(s):
    T, K, N, R, r = (s["case"][k] for k in "TKNRr")
    v = (s["x"].float() @ s["A"].float().view(R * r, K).T).view(T, R, r) * s["scales"][:, None]
    v = torch.where(_chosen(s), v, torch.zeros_like(v)).view(T, R * r)
    return {"out": (s["y"].float() + v @ s["B"].float().view(R * r, N)).bfloat16()}


def _plain_lora_bwd(s):
    T, K, N, R, r = (s["case"][k] for k in "TKNRr")
    chosen = _chosen(s)
    x, dy = s["x"].float(), s["dy"].float()
    w = (dy @ s["B"].float().view(R * r, N).T).view(T, R, r) * s["scales"][:, None]
    w = torch.where(chosen, w, torch.zeros_like(w)).view(T, R * r)
    v = torch.empty_like(s["v"])
    v[s["order"].long()] = s["v"]
    v = torch.where(chosen, v[:, None, :] * s["scales"][:, None], torch.zeros(T, R, r, device="cuda")).view(T, R * r)
    return {"dx": (s["dx0"].float() + w @ s["A"].float().view(R * r, K)).bfloat16(),
            "dA": (w.T @ x).bfloat16().view(R, r, K), "dB": (v.T @ dy).bfloat16().view(R, r, N)}


# ---------------------------------------------------------------- the library's calls

def _own_norm(g, s):
    c, N = s["case"], s["case"]["N"]
    out = {"t": torch.empty_like(s["h"]), "rstd": torch.empty(c["M"], 2, device="cuda")}
    if c["quant"]:
        q = torch.empty(c["M"], N, dtype=torch.uint8, device="cuda")
        out["scales"] = torch.empty(c["M"], N // 128, device="cuda")
        out["q"] = q.view(torch.float8_e4m3fn)
    else:
        out["u"] = torch.empty(c["M"], N, dtype=torch.bfloat16, device="cuda")
    g.norm_gate_residual(s["ctx"], s["y"], s["h"], s["w_pre"], out["t"], w_post=s["w_post"], gate=s["gate"], alpha=c["alpha"], beta=c["beta"], eps=s["eps"],
                         u=out.get("u"), q=out.get("q"), scales=out.get("scales"), rstd=out["rstd"])
    return out


def _own_norm_bwd(g, s):
    c, N = s["case"], s["case"]["N"]
    out = {"dy": torch.empty_like(s["y"]), "dh": torch.empty_like(s["h"]), "dw_pre": torch.empty(N, device="cuda")}
    if c["post"]:
        out["dw_post"] = torch.empty(N, device="cuda")
    if c["gate"] != "none":
        out["dgate"] = torch.empty(N, device="cuda") if c["gate"] == "row" else torch.empty_like(s["gate"])
    g.norm_gate_residual_bwd(s["ctx"], s["y"], s["h"], s["rstd"], s["dt"], out["dy"], out["dh"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"],
                             alpha=c["alpha"], beta=c["beta"], du=s["du"], dw_post=out.get("dw_post"), dw_pre=out["dw_pre"], dgate=out.get("dgate"))
    return out


def _own_lora(g, s):
    out = torch.empty_like(s["y"])
    g.lora_apply(s["ctx"], s["x"], s["order"], s["offsets"], s["A"], s["B"], s["scales"], s["ranks"], out, y=s["y"])
    return {"out": out}


def _own_lora_bwd(g, s):
    out = {"dx": torch.empty_like(s["x"]), "dA": torch.empty_like(s["A"]), "dB": torch.empty_like(s["B"])}
    g.lora_apply_bwd(s["ctx"], s["x"], s["dy"], s["order"], s["offsets"], s["A"], s["B"], s["scales"], s["ranks"], s["v"], out["dx"], out["dA"], out["dB"], dx0=s["dx0"])
    return out


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "lora": _plain_lora, "lora_bwd": _plain_lora_bwd}[op](state)
    import block_scaled_fp8_gemm_gb300 as g
    return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "lora": _own_lora, "lora_bwd": _own_lora_bwd}[op](g, state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm(c, s):
    y, t = s["y"].double(), s["h"].double().mul_(c["alpha"])
    r1 = (y.pow(2).sum(1) / c["N"] + s["eps"]).pow(-0.5) if c["post"] else torch.ones(c["M"], dtype=torch.float64, device="cuda")
    y.mul_(r1[:, None]).mul_(c["beta"])
    for f in (s["w_post"], s["gate"]):
        if f is not None:
            y.mul_(f.double())
    t.add_(y)
    del y
    r2 = (t.pow(2).sum(1) / c["N"] + s["eps"]).pow(-0.5)
    out = {"t": t.clone(), "rstd": torch.stack([r1, r2], 1)}
    u = t.mul_(r2[:, None]).mul_(s["w_pre"].double())
    if not c["quant"]:
        return {**out, "u": u}
    # a code stands for the value before its rounding, in units of its group's scale
    scales = u.view(c["M"], -1, 128).abs().max(2).values / F8_MAX
    return {**out, "scales": scales, "q": (u.view(c["M"], -1, 128) / scales[..., None]).view(c["M"], -1)}


def _exact_norm_bwd(c, s):
    # by the Jacobian of each step in turn: u -> t -> (h, g, n = yhat w1) -> y
    M, N = c["M"], c["N"]
    r1, r2 = s["rstd"].double().unbind(1)
    one = torch.ones(N, dtype=torch.float64, device="cuda")
    w1 = s["w_post"].double() if c["post"] else one
    g = s["gate"].double() if s["gate"] is not None else one
    yhat = s["y"].double() * r1[:, None]
    t = s["h"].double() * c["alpha"] + yhat * (w1 * c["beta"]) * g
    up = s["du"].double()
    out = {"dw_pre": torch.einsum("mn,mn,m->n", up, t, r2)}
    up = up * s["w_pre"].double()
    d = up * r2[:, None] - t * (torch.einsum("mn,mn->m", up, t) * r2 ** 3 / N)[:, None] + s["dt"].double()
    del up, t
    out["dh"] = d * c["alpha"]
    d = d * c["beta"]
    if c["gate"] != "none":
        dg = d * yhat * w1
        out["dgate"] = dg.sum(0) if c["gate"] == "row" else dg
    d = d * g
    if c["post"]:
        out["dw_post"] = torch.einsum("mn,mn->n", d, yhat)
        d = d * w1
        out["dy"] = (d - yhat * (torch.einsum("mn,mn->m", d, yhat) / N)[:, None]) * r1[:, None]
    else:
        out["dy"] = d
    return out


def _exact_lora(c, s):
    out, at = s["y"].double(), s["offsets"].tolist()
    for a in range(c["R"]):
        rows, k = s["order"][at[a]:at[a + 1]].long(), int(s["ranks"][a])
        if len(rows):
            out[rows] += float(s["scales"][a]) * (s["x"][rows].double() @ s["A"][a, :k].double().T) @ s["B"][a, :k].double()
    return {"out": out}


def _exact_lora_bwd(c, s):
    dx, at = s["dx0"].double(), s["offsets"].tolist()
    dA, dB = torch.zeros(s["A"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["B"].shape, dtype=torch.float64, device="cuda")
    for a in range(c["R"]):
        rows, k, scale = s["order"][at[a]:at[a + 1]].long(), int(s["ranks"][a]), float(s["scales"][a])
        if len(rows):
            dy = s["dy"][rows].double()
            w = scale * dy @ s["B"][a, :k].double().T
            dx[rows] += w @ s["A"][a, :k].double()
            dA[a, :k] = w.T @ s["x"][rows].double()
            dB[a, :k] = scale * s["v"][at[a]:at[a + 1], :k].double().T @ dy
    return {"dx": dx, "dA": dA, "dB": dB}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "lora": _exact_lora, "lora_bwd": _exact_lora_bwd}[case["op"]](case, s)
