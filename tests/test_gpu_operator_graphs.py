"""The residual and adapter operators captured in a CUDA graph: a replay is the eager call on whatever the
input buffers hold then, for a decode batch (one launch in a cluster) and for larger ones (launches that
overlap the one before them), and calls on two streams with a context each do not disturb one another."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


def context(g):
    torch.cuda.set_device(0)
    return g.gemmar_create(0, 1024, 1024, 256, 1, flags=g.GEMMAR_NO_SELF_TEST, wait_timeout_ns=500_000_000)


class Step:
    """wo_b's rows through adapters and norms, and back, on buffers of its own."""

    def __init__(self, g, ctx, T, seed):
        self.g, self.ctx = g, ctx
        gen = torch.Generator("cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
        K, N, R, r = 264, 1024, 3, 24
        self.x, self.y0, self.h = rnd(T, K).bfloat16(), rnd(T, N).bfloat16(), rnd(T, N)
        self.A, self.B = (rnd(R, r, K) / 16).bfloat16(), (rnd(R, r, N) / 4).bfloat16()
        self.w1, self.w2, self.scales = 1 + 0.1 * rnd(N), 1 + 0.1 * rnd(N), torch.ones(R, device="cuda")
        self.ids = torch.randint(-1, R, (T,), generator=gen, device="cuda", dtype=torch.int32)
        self.dt, self.du = rnd(T, N), rnd(T, N).bfloat16()
        e = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
        bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
        self.order, self.offsets, self.v = e(T, dtype=i32), e(R + 1, dtype=i32), e(T, r)
        self.y, self.t, self.rstd, self.q, self.s = e(T, N, dtype=bf), e(T, N), e(T, 2), e(T, N, dtype=u8), e(T, N // 128)
        self.dy, self.dh, self.dw1, self.dw2 = e(T, N, dtype=bf), e(T, N), e(N), e(N)
        self.dx, self.dA, self.dB = e(T, K, dtype=bf), e(R, r, K, dtype=bf), e(R, r, N, dtype=bf)

    def __call__(self):
        g, c = self.g, self.ctx
        g.lora_plan(c, self.ids, self.order, self.offsets)
        g.lora_apply(c, self.x, self.order, self.offsets, self.A, self.B, self.scales, None, self.y, y=self.y0, v=self.v)
        g.norm_gate_residual(c, self.y, self.h, self.w2, self.t, w_post=self.w1, q=self.q, scales=self.s, rstd=self.rstd)
        g.norm_gate_residual_bwd(c, self.y, self.h, self.rstd, self.dt, self.dy, self.dh, w_post=self.w1, w_pre=self.w2, du=self.du,
                                 dw_post=self.dw1, dw_pre=self.dw2)
        g.lora_apply_bwd(c, self.x, self.dy, self.order, self.offsets, self.A, self.B, self.scales, None, self.v, self.dx, self.dA, self.dB)

    def outputs(self):
        return [t.clone() for t in (self.order, self.offsets, self.y, self.t, self.rstd, self.q, self.s, self.dy, self.dh, self.dw1,
                                    self.dw2, self.dx, self.dA, self.dB)]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [1, 100, 700])
def test_replay_equals_eager(g, T):
    ctx = context(g)
    try:
        step = Step(g, ctx, T, T)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for seed in (11, 12):
            gen = torch.Generator("cuda").manual_seed(seed)
            step.x.copy_(torch.randn(step.x.shape, generator=gen, device="cuda"))
            step.ids.copy_(torch.randint(-1, 3, (T,), generator=gen, device="cuda", dtype=torch.int32))
            step()
            eager = step.outputs()
            for t in (step.y, step.t, step.q, step.dx, step.dA):
                t.zero_()
            for _ in range(3):
                graph.replay()
            torch.cuda.synchronize()
            assert same(step.outputs(), eager)
        assert g.gemmar_status(ctx)[0] == 0
    finally:
        ctx.close()


def test_two_streams_with_a_context_each(g):
    ctxs = [context(g), context(g)]
    try:
        steps = [Step(g, c, T, T) for c, T in zip(ctxs, (700, 613))]
        expect = []
        for s in steps:
            s()
            expect.append(s.outputs())
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(10):
            for s, st in zip(steps, streams):
                with torch.cuda.stream(st):
                    s()
        torch.cuda.synchronize()
        assert all(same(s.outputs(), e) for s, e in zip(steps, expect))
        assert all(g.gemmar_status(c)[0] == 0 for c in ctxs)
    finally:
        for c in ctxs:
            c.close()
