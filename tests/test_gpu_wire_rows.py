"""The fp8 wire's row scales are as many as the context's rows, whatever a narrower call leaves of its codes."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,refused", [(256, False), (512, True)])
def test_more_rows_than_the_context_has_scales_for(M, refused):
    import block_scaled_fp8_gemm_gb300 as g
    torch.cuda.set_device(0)
    N, K = 256, 256
    ctx = g.gemmar_create(0, 256, 512, K, 1, flags=g.GEMMAR_NO_SELF_TEST)
    try:
        a, b = (torch.full((rows, K), 0x38, dtype=torch.uint8, device="cuda") for rows in (M, N))
        sa, sb = torch.ones(M, K // 128, device="cuda"), torch.ones(N // 128, K // 128, device="cuda")
        out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        if refused:
            with pytest.raises(g.GemmarError) as e:
                g.fused_gemm_reduce(ctx, [a], [sa], [b], [sb], out, flags=g.GEMMAR_FP8_WIRE)
            assert e.value.code == g.GEMMAR_ERR_WORKSPACE and (out == 0).all()
        else:
            g.fused_gemm_reduce(ctx, [a], [sa], [b], [sb], out, flags=g.GEMMAR_FP8_WIRE)
            assert (out == K).all()   # every code 1.0, every scale 1
        assert g.gemmar_status(ctx)[0] == 0
    finally:
        ctx.close()
