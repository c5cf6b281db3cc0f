"""A moe_apply whose waits run out (by the context's own limit, not by a fault) and the calls after it."""
import pytest
import torch

from test_gpu_moe import apply, check_layer, layer, picks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


def test_the_call_after_one_that_gave_up(g):
    """302 MB of the first product's weights take 45 us at the least, so the CTAs' wait for them runs out at 25; eight CTAs
    without a share have counted themselves at the first barrier by then.  The next call finds its barriers as new."""
    torch.cuda.set_device(0)
    s, rnd, gen = layer(3, 256, 128, 4, 1)
    ids, weights = picks(3, 2, 4, gen)
    ctx = g.gemmar_create(0, 1024, 4096, 256, 1, flags=g.GEMMAR_NO_SELF_TEST)
    want = apply(g, ctx, s, ids, weights)
    check_layer(want, s, ids, weights)
    ctx.close()

    H, I, E, T, k = 65536, 128, 18, 2, 9
    f32 = lambda *shape: torch.zeros(shape, device="cuda")
    u8 = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device="cuda")
    big = (u8(T, H), f32(T, H // 128), torch.arange(E, dtype=torch.int32, device="cuda").view(T, k), f32(T, k), u8(E, 2 * I, H),
           f32(E, 2 * I // 128, H // 128), u8(E, H, I), f32(E, H // 128, I // 128), torch.empty(T, H, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    hurried = g.gemmar_create(0, 1024, 4096, 256, 1, flags=g.GEMMAR_NO_SELF_TEST, wait_timeout_ns=25_000)
    for _ in range(3):
        g.moe_apply(hurried, *big)
        torch.cuda.synchronize()
        for _ in range(2):
            assert torch.equal(apply(g, hurried, s, ids, weights), want)
    assert g.gemmar_status(hurried)[0] == g.GEMMAR_ERR_TIMEOUT
    with pytest.raises(g.GemmarError) as e:   # disabled from here on
        g.moe_apply(hurried, *big)
    assert e.value.code == g.GEMMAR_ERR_DISABLED
    hurried.close()
