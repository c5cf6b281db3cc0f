"""gemm_blockscale_act against its definition in fp64: every activation, gated and not, each output form, rows
from one to several tiles, odd numbers of column blocks, views, a residual that is the output, and what a row
with a NaN does to the others."""
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
    c = g.gemmar_create(0, 1024, 2048, 256, 1, flags=g.GEMMAR_NO_SELF_TEST)
    yield c
    assert g.gemmar_status(c)[0] == 0
    c.close()


def operands(M, P, K, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    return (*ff.codes_1x128(rnd(M, K)), *ff.codes_128x128(rnd(P, K) * K ** -0.5 * 1.5)), rnd


def run(g, ctx, ops, N, act, gated, out=("C32",), **kw):
    M, P = ops[0].shape[0], ops[2].shape[0]
    new = lambda *s, dtype=torch.float32: torch.full(s, 77, dtype=dtype, device="cuda")
    res = {}
    C = None
    if "C32" in out:
        C = res["C"] = new(M, N)
    if "C16" in out:
        C = res["C"] = new(M, N, dtype=torch.bfloat16)
    if "q" in out:
        kw["q"] = res["q"] = new(M, N, dtype=torch.uint8)
        kw["scales"] = res["scales"] = new(M, N // 128)
    if "z" in out:
        kw["z"] = res["z"] = new(M, P, dtype=torch.bfloat16)
    g.gemm_blockscale_act(ctx, *ops, C, act=ff.ACTS.index(act), gated=gated, **kw)
    torch.cuda.synchronize()
    return res


def check(res, ops, act, gated, bias=None, residual=None):
    ref, err, z, ez = ff.act_reference(*ops, act, gated, bias, residual)
    if "C" in res:
        half = 2.0 ** -24 if res["C"].dtype == torch.float32 else ff.BF16
        ff.within(res["C"], ref, err + half * (ref.abs() + err), "C")
    if "q" in res:
        ff.codes_within(res["q"], res["scales"], ref, err, "out")
    if "z" in res:
        ff.within(res["z"], z, ez + ff.BF16 * (z.abs() + ez), "z")


@pytest.mark.parametrize("act", ff.ACTS)
@pytest.mark.parametrize("gated", [False, True])
def test_activations(g, ctx, act, gated):
    N = 256
    ops, rnd = operands(200, N * (2 if gated else 1), 384, 1)
    bias, res = rnd(ops[2].shape[0]) * 0.5, rnd(200, N)
    check(run(g, ctx, ops, N, act, gated, ("C32", "q", "z"), bias=bias, residual=res), ops, act, gated, bias, res)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 16, 17, 33, 64, 65, 96, 127, 128, 129, 300, 777])
@pytest.mark.parametrize("N,K,gated", [(128, 128, False), (640, 256, False), (384, 1152, True), (2048, 512, False)])
def test_rows(g, ctx, M, N, K, gated):
    ops, rnd = operands(M, N * (2 if gated else 1), K, M)
    res = rnd(M, N).bfloat16()
    check(run(g, ctx, ops, N, "silu", gated, ("C16", "q", "z"), residual=res), ops, "silu", gated, None, res)


@pytest.mark.parametrize("M", [1, 23, 150])
@pytest.mark.parametrize("gated", [False, True])
def test_codes_are_the_quantiser_s(g, ctx, M, gated):
    """q and scales are, bit for bit, what quant_blockscale_e4m3 makes of the fp32 C."""
    N = 384
    ops, rnd = operands(M, N * (2 if gated else 1), 256, 3)
    r = run(g, ctx, ops, N, "gelu_tanh", gated, ("C32", "q"), bias=rnd(ops[2].shape[0]))
    q, s = torch.empty_like(r["q"]), torch.empty_like(r["scales"])
    g.quant_blockscale_e4m3(ctx, r["C"], 1, q, s)
    torch.cuda.synchronize()
    assert torch.equal(s, r["scales"]) and torch.equal(q, r["q"])


@pytest.mark.parametrize("M", [5, 140])
def test_without_epilogue_is_the_plain_product(g, ctx, M):
    ops, _ = operands(M, 512, 640, 4)
    C = torch.empty(M, 512, device="cuda")
    g.gemm_blockscale_fp8(ctx, *ops, C)
    ref, err, _, _ = ff.act_reference(*ops, "none", False)
    ff.within(C, ref, err + 2.0 ** -24 * ref.abs())
    ff.within(run(g, ctx, ops, 512, "none", False)["C"], ref, err + 2.0 ** -24 * ref.abs())


@pytest.mark.parametrize("M", [3, 130])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_residual_in_place_and_views(g, ctx, M, dtype):
    N = 256
    ops, rnd = operands(M, N, 256, 5)
    wide = rnd(M, N + 64).to(dtype)
    before = wide.clone()
    view = wide[:, 32:32 + N]
    g.gemm_blockscale_act(ctx, *ops, view, act=g.GEMMAR_ACT_SILU, residual=view)
    torch.cuda.synchronize()
    check({"C": view}, ops, "silu", False, None, before[:, 32:32 + N])
    assert torch.equal(wide[:, :32], before[:, :32]) and torch.equal(wide[:, 32 + N:], before[:, 32 + N:])


def test_one_residual_row_for_all(g, ctx):
    ops, rnd = operands(40, 256, 128, 6)
    row = rnd(1, 256)
    res = row.expand(40, 256)
    check(run(g, ctx, ops, 256, "relu", False, residual=res), ops, "relu", False, None, res)


@pytest.mark.parametrize("M", [40, 200])
@pytest.mark.parametrize("gated", [False, True])
def test_a_row_of_nan_stays_alone(g, ctx, M, gated):
    N = 256
    ops, _ = operands(M, N * (2 if gated else 1), 256, 7)
    clean = run(g, ctx, ops, N, "silu", gated, ("C32", "q", "z"))
    A = ops[0].clone()
    A[11, 5] = 0x7F
    r = run(g, ctx, (A, *ops[1:]), N, "silu", gated, ("C32", "q", "z"))
    keep = torch.arange(M, device="cuda") != 11
    assert torch.isnan(r["C"][11]).all() and torch.isnan(r["z"][11]).all()
    assert all(torch.equal(r[n][keep], clean[n][keep]) for n in r)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("M", [4, 140])
def test_far_pre_activations(g, ctx, act, M):
    """Very negative z gives 0, very positive z gives z, an infinite one the limit, without NaN."""
    ops, rnd = operands(M, 256, 128, 8)
    bias = torch.zeros(256, device="cuda")
    bias[:4] = torch.tensor([-1e30, 1e30, -float("inf"), float("inf")])
    C = run(g, ctx, ops, 256, act, False, bias=bias)["C"]
    assert (C[:, 0] == 0).all() and (C[:, 2] == 0).all()
    assert (C[:, 1] > 0.99e30).all() and torch.isinf(C[:, 3]).all() and (C[:, 3] > 0).all()


@pytest.mark.parametrize("M", [6, 140])
def test_zero_scales(g, ctx, M):
    """Zero rows of A and zero blocks of B give exact zeros, and zero codes with scale 0."""
    ops, _ = operands(M, 256, 256, 9)
    A, sa, B, sb = (t.clone() for t in ops)
    A[2], sa[2] = 0, 0
    r = run(g, ctx, (A, sa, B, sb), 256, "silu", False, ("C32", "q"))
    assert (r["C"][2] == 0).all() and (r["scales"][2] == 0).all() and (r["q"][2] == 0).all()


def test_the_same_bits_twice(g, ctx):
    for M in (1, 48, 128, 500):
        ops, rnd = operands(M, 1024, 1024, M)
        res = rnd(M, 512)
        a, b = (run(g, ctx, ops, 512, "silu", True, ("C32", "q", "z"), residual=res) for _ in range(2))
        assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("M", [1, 140])
@pytest.mark.parametrize("act", ff.ACTS)
def test_values_over_the_whole_range(g, ctx, act, M):
    """Without a product z is the bias, exactly: the activation's own error from one tail to the other."""
    N = 8192
    ops, rnd = operands(M, N, 128, 1)
    ops[0].zero_()
    z = torch.linspace(-12, 12, N, device="cuda")
    ref, exact = ff.value(act, z.double()), torch.zeros(N, device="cuda", dtype=torch.float64)
    # act is z times a factor in [0, 1], and a factor below 2^-126 may be 0 (the sigmoid's divisor is past
    # 2^126, from where the fast division gives 0): off by at most 2^-126 |z|
    bound = ff.value_error(act, z.double(), exact) + 2.0 ** -24 * ref.abs() + 2.0 ** -126 * z.double().abs().clamp(min=1)
    ff.within(run(g, ctx, ops, N, act, False, bias=z)["C"], ref.expand(M, N), bound)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("M,N,K,gated", [(2500, 1920, 256, False), (2500, 1920, 256, True), (5000, 128, 128, False), (4097, 640, 640, False)])
def test_many_rows_join_a_wider_stream(g, ctx, M, N, K, gated, act, dtype):
    """Several tiles to a CTA, a ragged last one and an odd number of column blocks; the residual is columns of a
    wider matrix, read alone, in place, and as one row for all."""
    ops, rnd = operands(M, N * (2 if gated else 1), K, 12)
    wide = rnd(M, N + 40).to(dtype)
    view = wide[:, 8:8 + N]
    before, beside = view.clone(), (wide[:, :8].clone(), wide[:, 8 + N:].clone())
    got = run(g, ctx, ops, N, act, gated, ("C32", "q"), residual=view)
    check(got, ops, act, gated, None, before)
    g.gemm_blockscale_act(ctx, *ops, view, act=ff.ACTS.index(act), gated=gated, residual=view)
    torch.cuda.synchronize()
    assert torch.equal(view, got["C"].to(dtype)) and torch.equal(wide[:, :8], beside[0]) and torch.equal(wide[:, 8 + N:], beside[1])
    row = before[7:8].expand(M, N)
    check(run(g, ctx, ops, N, act, gated, ("C16",), residual=row), ops, act, gated, None, row)
