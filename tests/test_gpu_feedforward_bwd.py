"""gemm_blockscale_act_bwd against the formula in fp64 and against differences of the forward definition, its
column sums, its codes, and the whole way back through a gated layer with frozen weights."""
import pytest
import torch

import feedforward as ff

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def ctx(g):
    torch.cuda.set_device(0)
    c = g.gemmar_create(0, 4096, 2048, 256, 1, flags=g.GEMMAR_NO_SELF_TEST)
    yield c
    assert g.gemmar_status(c)[0] == 0
    c.close()


def reference(z, dout, act, gated):
    """dz and the bound of an fp32 evaluation: slopes and values are off by 2^-19 at most (their factors'
    errors times at most 2), products by a rounding each."""
    leaf = z.double().requires_grad_()
    out = ff.value(act, leaf[:, :leaf.shape[1] // 2]) * leaf[:, leaf.shape[1] // 2:] if gated else ff.value(act, leaf)
    dz = torch.autograd.grad(out, leaf, dout.double())[0]
    d, z = dout.double().abs(), z.double()
    if gated:
        zg, zu = z.chunk(2, 1)
        err = torch.cat([2.0 ** -19 * d * zu.abs(), d * ff.value_error(act, zg, 0 * zg)], 1)
    else:
        err = 2.0 ** -19 * d
    return dz, err + 2.0 ** -22 * dz.abs()


def inputs(M, N, gated, seed, dtype=torch.bfloat16):
    gen = torch.Generator("cuda").manual_seed(seed)
    z = (torch.randn(M, N * (2 if gated else 1), generator=gen, device="cuda") * 2).bfloat16()
    return z, torch.randn(M, N, generator=gen, device="cuda").to(dtype)


def run(g, ctx, dout, z, act, gated, codes=True):
    new = lambda *s, dtype=torch.float32: torch.full(s, 77, dtype=dtype, device="cuda")
    M, P = z.shape
    r = {"dz": new(M, P, dtype=torch.bfloat16), "dbias": new(P)}
    if codes:
        r.update(q=new(M, P, dtype=torch.uint8), scales=new(M, P // 128))
    g.gemm_blockscale_act_bwd(ctx, dout, z, act=ff.ACTS.index(act), gated=gated, **r)
    torch.cuda.synchronize()
    return r


def check(r, z, dout, act, gated):
    dz, err = reference(z, dout, act, gated)
    ff.within(r["dz"], dz, err + ff.BF16 * (dz.abs() + err), "dz")
    if "q" in r:
        ff.codes_within(r["q"], r["scales"], dz, err, "dz")
    # sums: a thread's chain over its rows, then the CTA's and the shares' (at most M / 32 + 16 additions)
    M = z.shape[0]
    ff.within(r["dbias"], dz.sum(0), err.sum(0) + (M / 32 + 16) * 2.0 ** -24 * dz.abs().sum(0) + 1e-30, "dbias")


@pytest.mark.parametrize("act", ff.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_formula(g, ctx, act, gated, dtype):
    z, dout = inputs(333, 384, gated, 1, dtype)
    check(run(g, ctx, dout, z, act, gated), z, dout, act, gated)


@pytest.mark.parametrize("M,N", [(1, 128), (2, 640), (5, 1152), (63, 256), (64, 512), (65, 128), (1000, 896), (4099, 128), (2500, 2048)])
@pytest.mark.parametrize("gated", [False, True])
def test_sizes(g, ctx, M, N, gated):
    z, dout = inputs(M, N, gated, M + N)
    check(run(g, ctx, dout, z, "silu", gated), z, dout, "silu", gated)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_against_differences(g, ctx, act):
    z, dout = inputs(16, 128, True, 5, torch.float32)
    r = run(g, ctx, dout, z, act, True, codes=False)
    h, z64 = 2.0 ** -12, z.double()
    f = lambda t: ff.value(act, t[:, :128]) * t[:, 128:]
    for half in (0, 1):
        step = torch.zeros_like(z64)
        step[:, 128 * half:128 * half + 128] = h
        diff = dout.double() * (f(z64 + step) - f(z64 - step)) / (2 * h)
        # third derivatives are below 3 |z_u|: h^2 / 6 of them, then dz's own rounding
        bound = dout.double().abs() * (z64.abs().amax() + 1) * h * h + ff.BF16 * diff.abs() * 1.01 + 1e-5
        ff.within(r["dz"][:, 128 * half:128 * half + 128], diff, bound)


def test_codes_alone_views_and_in_place(g, ctx):
    z, dout = inputs(77, 256, False, 6)
    full = run(g, ctx, dout, z, "silu", False)
    wide = torch.zeros(77, 320, dtype=torch.bfloat16, device="cuda")
    wide[:, 64:] = dout
    q, s = torch.zeros_like(full["q"]), torch.zeros_like(full["scales"])
    g.gemm_blockscale_act_bwd(ctx, wide[:, 64:], z, None, act=g.GEMMAR_ACT_SILU, q=q, scales=s)
    assert torch.equal(q, full["q"]) and torch.equal(s, full["scales"])
    inplace, z2 = dout.clone(), z.clone()
    g.gemm_blockscale_act_bwd(ctx, inplace, z, inplace, act=g.GEMMAR_ACT_SILU)
    g.gemm_blockscale_act_bwd(ctx, dout, z2, z2, act=g.GEMMAR_ACT_SILU)
    assert torch.equal(inplace, full["dz"]) and torch.equal(z2, full["dz"])
    row = dout[:1].expand(77, 256)
    a, b = torch.empty_like(z), torch.empty_like(z)
    g.gemm_blockscale_act_bwd(ctx, row, z, a, act=g.GEMMAR_ACT_SILU)
    g.gemm_blockscale_act_bwd(ctx, row.contiguous(), z, b, act=g.GEMMAR_ACT_SILU)
    assert torch.equal(a, b)


def test_far_pre_activations(g, ctx):
    z = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    z[:, 0], z[:, 1], z[:, 2], z[:, 3] = -1e30, 1e30, -float("inf"), float("inf")
    dout = torch.ones(4, 128, dtype=torch.bfloat16, device="cuda")
    for act in ("relu", "silu", "gelu", "gelu_tanh"):
        dz = run(g, ctx, dout, z, act, False)["dz"]
        assert dz[:, :4].tolist() == [[0.0, 1.0, 0.0, 1.0]] * 4, act


def test_zero_rows_and_nan(g, ctx):
    z, dout = inputs(50, 256, True, 8)
    dout[3] = 0
    clean = run(g, ctx, dout, z, "silu", True)
    assert (clean["q"][3] & 0x7F == 0).all() and (clean["scales"][3] == 0).all()
    dout[7, 9] = float("nan")
    r = run(g, ctx, dout, z, "silu", True)
    keep = torch.arange(50, device="cuda") != 7
    assert all(torch.equal(r[n][keep], clean[n][keep]) for n in ("dz", "q", "scales"))
    assert torch.isnan(r["dbias"][[9, 256 + 9]]).all() and int(torch.isnan(r["dbias"]).sum()) == 2


def test_through_frozen_weights(g, ctx):
    """Forward, backward, and the gradient of the input by the product with the transposed codes: the whole
    equals the fp64 gradient to what the two quantisations of dz and the bf16 z cost."""
    M, N, K = 300, 512, 384
    gen = torch.Generator("cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    A, sa = ff.codes_1x128(rnd(M, K))
    B, sb = ff.codes_128x128(rnd(2 * N, K) * K ** -0.5)
    bias = rnd(2 * N) * 0.1
    C = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    z = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    g.gemm_blockscale_act(ctx, A, sa, B, sb, C, act=g.GEMMAR_ACT_SILU, gated=True, bias=bias, z=z)
    dout = rnd(M, N).bfloat16()
    q, s = torch.empty(M, 2 * N, dtype=torch.uint8, device="cuda"), torch.empty(M, 2 * N // 128, device="cuda")
    dbias, dA = torch.empty(2 * N, device="cuda"), torch.empty(M, K, device="cuda")
    g.gemm_blockscale_act_bwd(ctx, dout, z, None, act=g.GEMMAR_ACT_SILU, gated=True, dbias=dbias, q=q, scales=s)
    g.gemm_blockscale_fp8(ctx, q, s, B.T.contiguous(), sb.T.contiguous(), dA)
    torch.cuda.synchronize()
    a, b = ff.values(A, sa).requires_grad_(), ff.values(B, sb)
    bias64 = bias.double().requires_grad_()
    y = a @ b.T + bias64
    da, db = torch.autograd.grad(ff.value("silu", y[:, :N]) * y[:, N:], (a, bias64), dout.double())
    # z's rounding moves dz by at most 2^-8 |z| times the slopes' slope, the codes by 2^-4 |dz|
    dz, _ = reference(y.detach(), dout, "silu", True)
    zg, zu = y.detach().chunk(2, 1)
    d = dout.double().abs()
    moved = ff.BF16 * torch.cat([d * (0.5 * zg.abs() * zu.abs() + 1.1 * zu.abs()), 1.1 * d * zg.abs()], 1)
    top = (dz.abs() + moved).view(M, -1, 128).amax(2).repeat_interleave(128, 1)
    code = torch.maximum(ff.E4M3 * (dz.abs() + moved), top * 2.0 ** -10 / 448)
    bound = (moved + 1.001 * code) @ b.abs() + 1e-5
    ff.within(dA, da, bound, "dA")
    ff.within(dbias, db, moved.sum(0) + 1e-3 * 2.0 ** -8 * dz.abs().sum(0) + 1e-6, "dbias")
