"""Calls whose waits run out at once (a context with a limit of 1 ns): they end by themselves, the status says so, and what
runs next on the same SMs is right."""
import pytest
import torch

import feedforward as ff
from test_gpu_moe import apply, check_layer, layer, picks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


def contexts(g):
    torch.cuda.set_device(0)
    return [g.gemmar_create(0, 4096, 1024, 256, 1, flags=g.GEMMAR_NO_SELF_TEST, wait_timeout_ns=ns) for ns in (0, 1)]


def done(g, ctx, hurried):
    torch.cuda.synchronize()
    assert g.gemmar_status(ctx)[0] == 0
    code, _ = g.gemmar_status(hurried)
    assert code in (0, g.GEMMAR_ERR_TIMEOUT)
    ctx.close()
    hurried.close()
    return code


@pytest.mark.parametrize("M", [1, 40, 300, 2000])
@pytest.mark.parametrize("gated", [False, True])
def test_product(g, M, gated):
    ctx, hurried = contexts(g)
    N, K = 1024, 7168
    gen = torch.Generator("cuda").manual_seed(M)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    A, sa = ff.codes_1x128(rnd(M, K))
    B, sb = ff.codes_128x128(rnd(2 * N if gated else N, K) * K ** -0.5)
    rows = torch.arange(0, M, max(1, M // 50), device="cuda")
    ref, err, _, _ = ff.act_reference(A[rows], sa[rows], B, sb, "silu", gated)
    out = torch.empty(M, N, device="cuda")
    late = torch.empty(M, N, device="cuda")
    for _ in range(4):
        g.gemm_blockscale_act(hurried, A, sa, B, sb, late, act=g.GEMMAR_ACT_SILU, gated=gated)
        g.gemm_blockscale_act(ctx, A, sa, B, sb, out, act=g.GEMMAR_ACT_SILU, gated=gated)
    torch.cuda.synchronize()
    ff.within(out[rows], ref, err)
    if done(g, ctx, hurried) == 0:
        ff.within(late[rows], ref, err)


@pytest.mark.parametrize("T", [2, 60])
def test_experts(g, T):
    ctx, hurried = contexts(g)
    s, rnd, gen = layer(T, 1024, 256, 8, T)
    ids, weights = picks(T, 3, 8, gen)
    for _ in range(4):
        apply(g, hurried, s, ids, weights)
        out = apply(g, ctx, s, ids, weights)
    check_layer(out, s, ids, weights)
    done(g, ctx, hurried)
