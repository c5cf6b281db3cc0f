"""The end of an attention block and the start of the next, as a serving step and as a training step.

    python examples/adapted_block.py            # wo_b's widths, a few hundred tokens
    python examples/adapted_block.py --tokens 4 # a decode step

Serving: wo_b over P K-slices (fused_gemm_reduce), the requests' low-rank adapters on top (lora_plan,
lora_apply), the residual stream with its norms and gate (norm_gate_residual), whose codes and scales are the
A operand of the next block's GEMM (gemm_blockscale_fp8).  Training: the gradients of everything after the
frozen wo_b (norm_gate_residual_bwd, lora_apply_bwd).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_gemm_gb300 as g  # noqa: E402


def make(tokens, N, K, P, adapters, rank, seed=0):
    """Random activations and weights; the GEMMs' operands are quantised by the library."""
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s, scale=1.0: torch.randn(s, generator=gen, device="cuda") * scale
    m = {"x": rnd(tokens, P * K).bfloat16(), "h": rnd(tokens, N), "gate": torch.sigmoid(rnd(tokens, N)).bfloat16(),
         "w_post": 1 + 0.1 * rnd(N), "w_pre": 1 + 0.1 * rnd(N),
         "A": rnd(adapters, rank, P * K, scale=(P * K) ** -0.5).bfloat16(), "B": rnd(adapters, rank, N, scale=0.05).bfloat16(),
         "scales": torch.full((adapters,), 2.0, device="cuda"),
         "ranks": torch.randint(1, rank + 1, (adapters,), generator=gen, device="cuda", dtype=torch.int32),
         "ids": torch.randint(-1, adapters, (tokens,), generator=gen, device="cuda", dtype=torch.int32),
         "wo": [rnd(N, K, scale=0.02) for _ in range(P)], "next": rnd(N, N, scale=0.02)}
    return m


def quantise(ctx, w, rows):
    R, C = w.shape
    q = torch.empty(R, C, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-R // rows), C // 128, device="cuda")
    g.quant_blockscale_e4m3(ctx, w, rows, q, s)
    return q, s


def forward(ctx, next_ctx, m, P, K, alpha, beta):
    T, N = m["h"].shape
    bf16 = dict(dtype=torch.bfloat16, device="cuda")
    acts = [quantise(ctx, m["x"][:, p * K:(p + 1) * K].contiguous(), 1) for p in range(P)]
    weights = [quantise(ctx, w, 128) for w in m["wo"]]
    y = torch.empty(T, N, **bf16)
    g.fused_gemm_reduce(ctx, [a[0] for a in acts], [a[1] for a in acts], [w[0] for w in weights], [w[1] for w in weights], y, bands=1)
    out = {"wo_b": y.clone()}
    # one plan serves every layer of the batch
    R, r, _ = m["A"].shape
    out["order"] = torch.empty(T, dtype=torch.int32, device="cuda")
    out["offsets"] = torch.empty(R + 1, dtype=torch.int32, device="cuda")
    g.lora_plan(ctx, m["ids"], out["order"], out["offsets"])
    out["v"] = torch.zeros(T, r, device="cuda")
    g.lora_apply(ctx, m["x"], out["order"], out["offsets"], m["A"], m["B"], m["scales"], m["ranks"], y, y=y, v=out["v"])
    out["y"] = y
    out["t"], out["rstd"] = torch.empty_like(m["h"]), torch.empty(T, 2, device="cuda")
    out["q"], out["s"] = torch.empty(T, N, dtype=torch.uint8, device="cuda"), torch.empty(T, N // 128, device="cuda")
    g.norm_gate_residual(ctx, y, m["h"], m["w_pre"], out["t"], w_post=m["w_post"], gate=m["gate"], alpha=alpha, beta=beta,
                         q=out["q"], scales=out["s"], rstd=out["rstd"])
    # the codes are the next GEMM's operand as they are
    B, sb = quantise(next_ctx, m["next"], 128)
    out["next"] = torch.empty(T, N, **bf16)
    g.gemm_blockscale_fp8(next_ctx, out["q"], out["s"], B, sb, out["next"])
    return out


def backward(ctx, m, out, dt, du, alpha, beta):
    T, N = m["h"].shape
    dy, dh, dgate = torch.empty_like(out["y"]), torch.empty_like(m["h"]), torch.empty_like(m["gate"])
    dw_post, dw_pre = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    g.norm_gate_residual_bwd(ctx, out["y"], m["h"], out["rstd"], dt, dy, dh, w_post=m["w_post"], w_pre=m["w_pre"], gate=m["gate"],
                             alpha=alpha, beta=beta, du=du, dw_post=dw_post, dw_pre=dw_pre, dgate=dgate)
    dx, dA, dB = torch.empty_like(m["x"]), torch.empty_like(m["A"]), torch.empty_like(m["B"])
    g.lora_apply_bwd(ctx, m["x"], dy, out["order"], out["offsets"], m["A"], m["B"], m["scales"], m["ranks"], out["v"], dx, dA, dB)
    return {"dy": dy, "dh": dh, "dgate": dgate, "dw_post": dw_post, "dw_pre": dw_pre, "dx": dx, "dA": dA, "dB": dB}


def plain(m, wo_b, alpha, beta, eps=1e-6):
    """The same, after wo_b, in fp64 with autograd."""
    leaf = {k: m[k].double().requires_grad_() for k in ("x", "h", "gate", "w_post", "w_pre", "A", "B")}
    R, r, _ = m["A"].shape
    v = torch.einsum("tk,ajk->taj", leaf["x"], leaf["A"])
    own = (m["ids"][:, None] == torch.arange(R, device="cuda"))[:, :, None] & (torch.arange(r, device="cuda") < m["ranks"][:, None])[None]
    y = wo_b.double() + torch.einsum("taj,ajn->tn", torch.where(own, v * m["scales"][:, None].double(), 0.0), leaf["B"])
    n = y * (y.square().mean(1, keepdim=True) + eps).rsqrt() * leaf["w_post"]
    t = alpha * leaf["h"] + beta * leaf["gate"] * n
    return leaf, y, t, t * (t.square().mean(1, keepdim=True) + eps).rsqrt() * leaf["w_pre"]


def run(tokens=384, N=7168, K=2048, P=2, adapters=5, rank=16, alpha=1.0, beta=0.5):
    """Run both steps; returns {name: relative error against the plain fp64 computation}."""
    torch.cuda.set_device(0)
    ctx = g.gemmar_create(0, max(tokens, 128), N, K, P, flags=g.GEMMAR_NO_SELF_TEST)
    next_ctx = g.gemmar_create(0, max(tokens, 128), N, N, 1, flags=g.GEMMAR_NO_SELF_TEST)
    try:
        m = make(tokens, N, K, P, adapters, rank)
        out = forward(ctx, next_ctx, m, P, K, alpha, beta)
        gen = torch.Generator("cuda").manual_seed(1)
        dt, du = torch.randn(tokens, N, generator=gen, device="cuda"), torch.randn(tokens, N, generator=gen, device="cuda").bfloat16()
        grads = backward(ctx, m, out, dt, du, alpha, beta)
        torch.cuda.synchronize()
        for c in (ctx, next_ctx):
            code, detail = g.gemmar_status(c)
            if code != g.GEMMAR_OK:
                raise RuntimeError(f"device status {g.STATUS_NAMES.get(code)} at site {detail}")
        leaf, y, t, x = plain(m, out["wo_b"], alpha, beta)
        ((t * dt.double()).sum() + (x * du.double()).sum()).backward()
        codes = out["q"].view(torch.float8_e4m3fn).double().view(tokens, -1, 128) * out["s"].double()[..., None]
        pairs = {"y": (out["y"], y), "t": (out["t"], t), "codes": (codes.view(tokens, N), x), "next": (out["next"], x @ m["next"].double().T)}
        pairs |= {"d" + k: (grads["d" + k], v.grad) for k, v in leaf.items()}
        return {k: float((a.double() - b.detach()).norm() / b.detach().norm().clamp_min(1e-300)) for k, (a, b) in pairs.items()}
    finally:
        ctx.close()
        next_ctx.close()


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=384)
    for name, err in run(tokens=ap.parse_args().tokens).items():
        print(f"{name:8s} relative error {err:.2e}")
