"""norm_gate_residual and its backward pass against the formulas in 64 bits.

Tolerances.  A bf16 output is one rounding of an fp32 value: 2^-8 of the value (u of
an 8-bit significand).  The fp32 part: a row sum is a chain of at most 64 + 16 additions,
80 * 2^-24 = 4.8e-6 of the sum of magnitudes, and an element takes a dozen more
operations of 2^-24 each: 2e-5 of the magnitudes that enter it covers both.  A sum over
M <= 2000 rows is a chain of at most 160 additions: 1e-5 of the sum of magnitudes, on top
of its terms' own 2e-5."""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

U_BF16 = 2.0 ** -8
F32 = 2e-5


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def ctx(g):
    torch.cuda.set_device(0)
    c = g.gemmar_create(0, 2048, 16384, 128, 1, flags=g.GEMMAR_NO_SELF_TEST, wait_timeout_ns=500_000_000)
    yield c
    c.close()


def make(M, N, post, pre, gate, h32, y32=False, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    d = {"y": rnd(M, N).mul(2).to(torch.float32 if y32 else torch.bfloat16),
         "h": rnd(M, N).to(torch.float32 if h32 else torch.bfloat16),
         "w_post": 1 + 0.3 * rnd(N) if post else None, "w_pre": 1 + 0.3 * rnd(N) if pre else None,
         "gate": {"none": None, "row": rnd(N).bfloat16(), "token": rnd(M, N).bfloat16()}[gate],
         "dt": rnd(M, N).to(torch.float32 if h32 else torch.bfloat16), "du": rnd(M, N).bfloat16() if pre else None}
    return d


def dbl(t):
    return None if t is None else t.double()


def ref_forward(d, alpha, beta, eps):
    y, h = dbl(d["y"]), dbl(d["h"])
    N = y.shape[1]
    one = torch.ones((), dtype=torch.float64, device="cuda")
    w1 = dbl(d["w_post"]) if d["w_post"] is not None else one
    gate = dbl(d["gate"]) if d["gate"] is not None else one
    r1 = ((y * y).mean(1) + eps).rsqrt() if d["w_post"] is not None else torch.ones(len(y), dtype=torch.float64, device="cuda")
    branch = beta * gate * y * r1[:, None] * w1
    t = alpha * h + branch
    mag = (alpha * h).abs() + branch.abs()
    r2 = ((t * t).mean(1) + eps).rsqrt() if d["w_pre"] is not None else torch.ones_like(r1)
    x = t * r2[:, None] * dbl(d["w_pre"]) if d["w_pre"] is not None else None
    return t, x, r1, r2, mag


def close(got, ref, mag, u, what):
    err = (got.double() - ref).abs()
    bound = u * ref.abs() * (1 + 1e-3) + F32 * mag + 1e-37
    assert torch.isfinite(got.double()).all(), what
    worst = (err / bound).max().item()
    assert worst <= 1, (what, worst)


def u_of(t):
    return U_BF16 if t.dtype == torch.bfloat16 else 0.0


def forward(g, ctx, d, alpha=1.0, beta=1.0, eps=1e-6, u=True, q=False, stream=None):
    M, N = d["y"].shape
    o = {"t": torch.empty(M, N, dtype=d["h"].dtype, device="cuda"), "rstd": torch.empty(M, 2, device="cuda")}
    if u and d["w_pre"] is not None:
        o["u"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    if q:
        o["q"] = torch.empty(M, N, dtype=torch.uint8, device="cuda")
        o["scales"] = torch.empty(M, N // 128, device="cuda")
    g.norm_gate_residual(ctx, d["y"], d["h"], d["w_pre"], o["t"], w_post=d["w_post"], gate=d["gate"], alpha=alpha,
                         beta=beta, eps=eps, u=o.get("u"), q=o.get("q"), scales=o.get("scales"), rstd=o["rstd"], stream=stream)
    return o


def backward(g, ctx, d, rstd, alpha=1.0, beta=1.0, stream=None):
    M, N = d["y"].shape
    new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")
    o = {"dy": torch.empty_like(d["y"], memory_format=torch.contiguous_format),
         "dh": torch.empty_like(d["h"], memory_format=torch.contiguous_format)}
    if d["w_post"] is not None:
        o["dw_post"] = new(N)
    if d["w_pre"] is not None:
        o["dw_pre"] = new(N)
    if d["gate"] is not None:
        o["dgate"] = new(N) if d["gate"].dim() == 1 else new(M, N, dtype=torch.bfloat16)
    g.norm_gate_residual_bwd(ctx, d["y"], d["h"], rstd, d["dt"], o["dy"], o["dh"], w_post=d["w_post"], w_pre=d["w_pre"],
                             gate=d["gate"], alpha=alpha, beta=beta, du=d["du"], dw_post=o.get("dw_post"),
                             dw_pre=o.get("dw_pre"), dgate=o.get("dgate"), stream=stream)
    return o


def check_forward(d, o, alpha, beta, eps):
    t, x, r1, r2, mag = ref_forward(d, alpha, beta, eps)
    assert torch.allclose(o["rstd"][:, 0].double(), r1, rtol=F32, atol=0)
    # r2's relative error: t's own error weighs by mag/|t| in the mean square
    rel = F32 * (1 + (mag * t.abs()).mean(1) / ((t * t).mean(1) + eps))
    assert ((o["rstd"][:, 1].double() - r2).abs() <= rel * r2).all()
    close(o["t"], t, mag, u_of(o["t"]), "t")
    if x is not None:
        w2 = dbl(d["w_pre"]).abs()
        xmag = (mag * r2[:, None] + (t * r2[:, None]).abs() * (rel / F32)[:, None]) * w2
        if "u" in o:
            close(o["u"], x, xmag, U_BF16, "u")
        if "q" in o:
            s = o["scales"].double()
            amax = x.view(len(x), -1, 128).abs().amax(2)
            slack = F32 * xmag.view(len(x), -1, 128).amax(2)
            assert ((s * 448 - amax).abs() <= slack + 1e-30).all()
            got = o["q"].view(torch.float8_e4m3fn).double().view(len(x), -1, 128) * s[..., None]
            err = (got - x.view_as(got)).abs()
            # e4m3: 2^-4 of the value, 2^-10 of the scale below the normal range
            assert (err <= 2.0 ** -4 * x.view_as(got).abs() + 2.0 ** -10 * s[..., None] + F32 * 2 * xmag.view_as(got)).all()


def check_backward(d, rstd, o, alpha, beta):
    y, h = dbl(d["y"]), dbl(d["h"])
    M, N = y.shape
    r1, r2 = dbl(rstd[:, :1]), dbl(rstd[:, 1:])
    one = torch.ones(N, dtype=torch.float64, device="cuda")
    w1 = dbl(d["w_post"]) if d["w_post"] is not None else one
    gate = dbl(d["gate"]) if d["gate"] is not None else one
    n = y * r1
    tmag = (alpha * h).abs() + (beta * gate * n * w1).abs()
    that = (alpha * h + beta * gate * n * w1) * r2
    dmag = D = dbl(d["dt"]) if d["dt"] is not None else torch.zeros_like(y)
    dmag = dmag.abs()
    if d["w_pre"] is not None:
        du = dbl(d["du"])
        dv = du * dbl(d["w_pre"])
        D = D + r2 * (dv - that * (dv * that).mean(1, keepdim=True))
        hm = tmag * r2
        dmag = dmag + r2 * (dv.abs() + hm * (dv.abs() * hm).mean(1, keepdim=True))
        close(o["dw_pre"], (du * that).sum(0), 2 * (du.abs() * hm).sum(0), 0.0, "dw_pre")
    close(o["dh"], alpha * D, abs(alpha) * dmag, u_of(o["dh"]), "dh")
    c = beta * gate * w1
    e, emag = c * D, c.abs() * dmag
    if d["w_post"] is not None:
        ref = r1 * (e - n * (e * n).mean(1, keepdim=True))
        mag = r1 * (emag + n.abs() * (emag * n.abs()).mean(1, keepdim=True))
        close(o["dw_post"], (beta * gate * D * n).sum(0), 2 * (abs(beta) * gate.abs() * dmag * n.abs()).sum(0), 0.0, "dw_post")
    else:
        ref, mag = e, emag
    close(o["dy"], ref, mag, u_of(o["dy"]), "dy")
    if d["gate"] is not None:
        dg, gmag = beta * n * w1 * D, abs(beta) * n.abs() * w1.abs() * dmag
        if d["gate"].dim() == 1:
            close(o["dgate"], dg.sum(0), 2 * gmag.sum(0), 0.0, "dgate row")
        else:
            close(o["dgate"], dg, gmag, U_BF16, "dgate")


SHAPES = [(1, 7168), (3, 128), (5, 8), (33, 1032), (2, 16384), (700, 256), (161, 2056), (64, 7168), (9, 8192), (4, 8200)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("post,pre,gate,h32,y32", [(True, True, "row", False, False), (False, True, "none", True, False),
                                                   (True, True, "token", True, True), (True, False, "none", False, False),
                                                   (False, True, "token", False, False), (False, False, "row", False, True)])
def test_forward_and_backward(g, ctx, M, N, post, pre, gate, h32, y32):
    d = make(M, N, post, pre, gate, h32, y32, seed=M + N)
    alpha, beta, eps = 0.75, 1.5, 1e-5
    o = forward(g, ctx, d, alpha, beta, eps, q=pre and N % 128 == 0)
    check_forward(d, o, alpha, beta, eps)
    b = backward(g, ctx, d, o["rstd"], alpha, beta)
    check_backward(d, o["rstd"], b, alpha, beta)
    assert g.gemmar_status(ctx)[0] == 0


@pytest.mark.parametrize("M,N", [(37, 7168), (300, 384)])
def test_outputs_follow_from_the_fp32_sum_bit_for_bit(g, ctx, M, N):
    """With an fp32 stream t comes out unrounded, so x = (t r2) w2 can be formed again: u is its bf16
    rounding and the codes are quant_blockscale_e4m3's of it, whichever of them the call is asked for."""
    d = make(M, N, True, True, "token", True, seed=3)
    both = forward(g, ctx, d, q=True)
    x = (both["t"] * both["rstd"][:, 1:]) * d["w_pre"]
    assert torch.equal(both["u"].view(torch.int16), x.bfloat16().view(torch.int16))
    q, s = oracle.quant_act_1x128(x.cpu().numpy())
    assert np.array_equal(both["q"].cpu().numpy(), q) and np.array_equal(both["scales"].cpu().numpy(), s)
    only = forward(g, ctx, d, u=False, q=True)
    assert torch.equal(only["q"], both["q"]) and torch.equal(only["t"], both["t"])


def test_views_streams_and_in_place(g, ctx):
    M, N = 45, 1536
    d = make(M, N, True, True, "token", False, seed=5)
    ref, refb = forward(g, ctx, d), None
    refb = backward(g, ctx, d, ref["rstd"])
    wide = {k: torch.full((M, 2 * N + 8), float("nan"), dtype=d[k].dtype, device="cuda") for k in ("y", "h", "gate", "dt", "du")}
    v = dict(d)
    for i, k in enumerate(wide):
        v[k] = wide[k][:, 8 * (i % 2 + 1):8 * (i % 2 + 1) + N]
        v[k].copy_(d[k])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o = forward(g, ctx, v, stream=side)
    b = backward(g, ctx, v, o["rstd"], stream=side)
    side.synchronize()
    assert all(torch.equal(o[k], ref[k]) for k in ref) and all(torch.equal(b[k], refb[k]) for k in refb)
    # one row of h and of dt for every row
    w = dict(d, h=d["h"][:1].expand(M, N), dt=d["dt"][:1].expand(M, N))
    full = dict(d, h=w["h"].contiguous(), dt=w["dt"].contiguous())
    o1, o2 = forward(g, ctx, w), forward(g, ctx, full)
    assert all(torch.equal(o1[k], o2[k]) for k in o1)
    b1, b2 = backward(g, ctx, w, o1["rstd"]), backward(g, ctx, full, o1["rstd"])
    assert all(torch.equal(b1[k], b2[k]) for k in b1)
    # t over h, u over y; dh over dt
    y, h, dt = d["y"].clone(), d["h"].clone(), d["dt"].clone()
    g.norm_gate_residual(ctx, y, h, d["w_pre"], h, w_post=d["w_post"], gate=d["gate"], u=y)
    assert torch.equal(h, ref["t"]) and torch.equal(y, ref["u"])
    dy = torch.empty_like(d["y"])
    g.norm_gate_residual_bwd(ctx, d["y"], d["h"], ref["rstd"], dt, dy, dt, w_post=d["w_post"], w_pre=d["w_pre"], gate=d["gate"], du=d["du"])
    assert torch.equal(dt, refb["dh"]) and torch.equal(dy, refb["dy"])


def test_rows_are_independent_and_zero_rows_are_finite(g, ctx):
    d = make(40, 896, True, True, "token", True, seed=9)
    good = forward(g, ctx, d, q=True)
    goodb = backward(g, ctx, d, good["rstd"])
    bad = {k: (v.clone() if v is not None else None) for k, v in d.items()}
    bad["y"][3, 5] = float("nan")
    bad["h"][7, 800] = float("inf")
    bad["gate"][20] = float("-inf")
    bad["du"][25, 1] = float("nan")
    o = forward(g, ctx, bad, q=True)
    b = backward(g, ctx, bad, o["rstd"])
    keep = torch.tensor([i not in (3, 7, 20) for i in range(40)], device="cuda")
    for k in good:
        assert torch.equal(o[k][keep], good[k][keep]), k
    keep[25] = False
    for k in ("dy", "dh", "dgate"):
        assert torch.equal(b[k][keep], goodb[k][keep]), k
    assert not torch.isfinite(o["t"][3]).all() and torch.isnan(o["u"][3].float()).any()
    # zero rows, and a stream that the branch cancels exactly
    z = make(4, 256, True, True, "none", True, y32=True, seed=1)
    z["y"][0] = 0
    z["h"][:2] = 0
    z["w_post"] = None
    z["h"][2] = -z["y"][2]
    o = forward(g, ctx, z, q=True)
    check_forward(z, o, 1.0, 1.0, 1e-6)
    assert (o["t"][2] == 0).all() and (o["q"][2] == 0).all() and (o["scales"][2] == 0).all() and (o["u"][0] == 0).all()


def test_no_gradient_of_the_stream_and_repeatability(g, ctx):
    d = make(333, 512, True, True, "row", False, seed=13)
    o = forward(g, ctx, d)
    d["dt"] = None
    a, b = backward(g, ctx, d, o["rstd"]), backward(g, ctx, d, o["rstd"])
    check_backward(d, o["rstd"], a, 1.0, 1.0)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_rows_past_32_bit_offsets(g, ctx):
    M, N, stride = 131100, 64, 16400   # 2.15e9 elements from the first row to the last
    big = torch.empty(M * stride, dtype=torch.bfloat16, device="cuda")
    d = make(M, N, True, True, "row", False, seed=2)
    y = torch.as_strided(big, (M, N), (stride, 1))
    y.copy_(d["y"])
    ref = forward(g, ctx, d)
    d["y"] = y
    o = forward(g, ctx, d)
    assert all(torch.equal(o[k], ref[k]) for k in ref)


def loss(g, ctx, d, gt, gu, alpha, beta):
    o = forward(g, ctx, d, alpha, beta)
    return ((o["t"].double() * gt).sum() + (o["u"].double() * gu).sum()).item()


@pytest.mark.parametrize("post,gate", [(True, "row"), (True, "token"), (False, "none")])
def test_gradient_against_differences(g, ctx, post, gate):
    """Central differences of the forward pass along each gradient's own direction.  A step of size e
    changes the loss by 2 e |grad| sqrt(size); u's bf16 rounding adds noise of about 2^-9 an element, which
    the sum over 24576 of them puts below 1%, and the curvature e^2 ~ 1e-3: 3% covers both."""
    d = make(48, 512, post, True, gate, True, y32=True, seed=21)
    alpha, beta = 0.8, 1.2
    o = forward(g, ctx, d, alpha, beta)
    b = backward(g, ctx, d, o["rstd"], alpha, beta)
    pairs = {"y": "dy", "h": "dh", "w_pre": "dw_pre"}
    if post:
        pairs["w_post"] = "dw_post"
    if gate != "none":
        pairs["gate"] = "dgate"
    for name, grad in pairs.items():
        gr = b[grad].double()
        step = 0.03 * gr / gr.square().mean().sqrt()
        at = []
        for sign in (1, -1):
            e = dict(d)
            e[name] = (d[name].double() + sign * step).to(d[name].dtype)
            at.append(e)
        change = loss(g, ctx, at[0], dbl(d["dt"]), dbl(d["du"]), alpha, beta) - loss(g, ctx, at[1], dbl(d["dt"]), dbl(d["du"]), alpha, beta)
        expect = (gr * (at[0][name].double() - at[1][name].double())).sum().item()
        assert abs(change - expect) <= 0.03 * abs(expect), (name, change, expect)


def test_refusals(g, ctx):
    d = make(8, 256, True, True, "none", False, seed=1)
    t, u = torch.empty_like(d["h"]), torch.empty_like(d["y"])

    def code(**kw):
        a = dict(y=d["y"], h=d["h"], w_pre=d["w_pre"], t=t, u=u)
        a.update(kw)
        with pytest.raises(g.GemmarError) as e:
            g.norm_gate_residual(ctx, a.pop("y"), a.pop("h"), a.pop("w_pre"), a.pop("t"), **a)
        return e.value.code
    assert code(t=None) == g.GEMMAR_ERR_ARG
    assert code(w_pre=None) == g.GEMMAR_ERR_ARG                 # u without its weight
    assert code(q=torch.empty(8, 256, dtype=torch.uint8, device="cuda")) == g.GEMMAR_ERR_ARG   # codes without scales
    for bad in ({"eps": -1.0}, {"eps": float("nan")}, {"alpha": float("inf")}, {"beta": float("nan")}):
        assert code(**bad) == g.GEMMAR_ERR_ARG
    odd = torch.zeros(8, 260, dtype=torch.bfloat16, device="cuda")
    assert code(y=odd[:, 1:257]) == g.GEMMAR_ERR_ALIGN
    assert code(y=odd[:, 0:256]) == g.GEMMAR_ERR_ALIGN          # a row stride of 520 bytes
    narrow = torch.zeros(8, 12, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(g.GemmarError) as e:
        g.norm_gate_residual(ctx, narrow, narrow, None, torch.empty_like(narrow))
    assert e.value.code == g.GEMMAR_ERR_SHAPE
    wide = torch.zeros(1, 16392, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(g.GemmarError) as e:
        g.norm_gate_residual(ctx, wide, wide, None, torch.empty_like(wide))
    assert e.value.code == g.GEMMAR_ERR_SHAPE
    ok = torch.zeros(8, 136, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(g.GemmarError) as e:                     # codes need whole groups of 128
        g.norm_gate_residual(ctx, ok, ok, torch.ones(136, device="cuda"), torch.empty_like(ok),
                             q=torch.empty(8, 136, dtype=torch.uint8, device="cuda"), scales=torch.empty(8, 1, device="cuda"))
    assert e.value.code == g.GEMMAR_ERR_SHAPE
    with pytest.raises(ValueError):
        g.norm_gate_residual(ctx, d["y"], d["h"][:4], d["w_pre"], t)
    with pytest.raises(TypeError):
        g.norm_gate_residual(ctx, d["y"], d["h"], d["w_pre"].bfloat16(), t)
    with pytest.raises(ValueError):
        g.norm_gate_residual(ctx, d["y"], d["h"], d["w_pre"], t, gate=torch.ones(1, 256, device="cuda").bfloat16().expand(8, 256))
    rstd = torch.ones(8, 2, device="cuda")
    with pytest.raises(g.GemmarError) as e:                     # the normed rows' gradient is missing
        g.norm_gate_residual_bwd(ctx, d["y"], d["h"], rstd, d["dt"], torch.empty_like(d["y"]), torch.empty_like(d["h"]), w_pre=d["w_pre"])
    assert e.value.code == g.GEMMAR_ERR_ARG
    small = g.gemmar_create(0, 1, 128, 128, 1, flags=g.GEMMAR_NO_SELF_TEST)
    try:
        big = make(4096, 16384, False, True, "none", False, seed=4)
        with pytest.raises(g.GemmarError) as e:
            backward(g, small, big, torch.ones(4096, 2, device="cuda"))
        assert e.value.code == g.GEMMAR_ERR_WORKSPACE
    finally:
        small.close()
    assert g.gemmar_status(ctx)[0] == 0
