"""The feed-forward operators as a block calls them: behind the norm, one after another, captured and replayed, on
streams of their own, at offsets past 32 bits; and what they refuse once tensors are on the GPU."""
import os
import subprocess
import sys

import pytest
import torch

import feedforward as ff

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


def context(g, max_M=1024, N=4096):
    torch.cuda.set_device(0)
    return g.gemmar_create(0, max_M, N, 256, 1, flags=g.GEMMAR_NO_SELF_TEST, wait_timeout_ns=500_000_000)


class Block:
    """wo_b's rows join the stream; a gated feed-forward layer with frozen weights, or the experts' layer; and back."""

    def __init__(self, g, ctx, T, seed):
        self.g, self.ctx, self.T = g, ctx, T
        gen = torch.Generator("cuda").manual_seed(seed)
        self.rnd = rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
        self.H, self.I, self.E, self.k = H, I, E, k = 768, 512, 12, 3
        self.y, self.h = rnd(T, H).bfloat16(), rnd(T, H)
        self.w1, self.w2n = 1 + 0.1 * rnd(H), 1 + 0.1 * rnd(H)
        self.up, self.sup = ff.codes_128x128(rnd(2 * I, H) * H ** -0.5 * 1.5)
        self.down, self.sdown = ff.codes_128x128(rnd(H, I) * I ** -0.5)
        self.upT, self.supT = self.up.T.contiguous(), self.sup.T.contiguous()
        self.downT, self.sdownT = self.down.T.contiguous(), self.sdown.T.contiguous()
        w13, w2 = [ff.codes_128x128(rnd(2 * I, H) * H ** -0.5 * 1.5) for _ in range(E)], [ff.codes_128x128(rnd(H, I) * I ** -0.5) for _ in range(E)]
        self.w13, self.s13 = (torch.stack([a[i] for a in w13]) for i in (0, 1))
        self.w2, self.s2 = (torch.stack([a[i] for a in w2]) for i in (0, 1))
        self.router, self.bias, self.b_up = rnd(E, H) * H ** -0.5, 0.1 * rnd(E), 0.1 * rnd(2 * I)
        self.dout = rnd(T, H).bfloat16()
        e = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
        bf, u8 = torch.bfloat16, torch.uint8
        self.t, self.u, self.q, self.s = e(T, H), e(T, H, dtype=bf), e(T, H, dtype=u8), e(T, H // 128)
        self.z, self.qi, self.si, self.out = e(T, 2 * I, dtype=bf), e(T, I, dtype=u8), e(T, I // 128), e(T, H)
        self.dqo, self.dso, self.dinner = e(T, H, dtype=u8), e(T, H // 128), e(T, I, dtype=bf)
        self.dz, self.qz, self.sz, self.db, self.dx = e(T, 2 * I, dtype=bf), e(T, 2 * I, dtype=u8), e(T, 2 * I // 128), e(2 * I), e(T, H, dtype=bf)
        self.ids, self.wts, self.moe = e(T, k, dtype=torch.int32), e(T, k), e(T, H, dtype=bf)

    def __call__(self, stream=None):
        g, c, kw = self.g, self.ctx, dict(stream=stream)
        g.norm_gate_residual(c, self.y, self.h, self.w2n, self.t, w_post=self.w1, u=self.u, q=self.q, scales=self.s, **kw)
        g.gemm_blockscale_act(c, self.q, self.s, self.up, self.sup, None, act=g.GEMMAR_ACT_SILU, gated=True, bias=self.b_up, q=self.qi, scales=self.si,
                              z=self.z, **kw)
        g.gemm_blockscale_act(c, self.qi, self.si, self.down, self.sdown, self.out, residual=self.t, **kw)
        # back: the down-projection's input gradient, the activation's, the up-projection's
        g.quant_blockscale_e4m3(c, self.dout, 1, self.dqo, self.dso, **kw)
        g.gemm_blockscale_fp8(c, self.dqo, self.dso, self.downT, self.sdownT, self.dinner, **kw)
        g.gemm_blockscale_act_bwd(c, self.dinner, self.z, self.dz, act=g.GEMMAR_ACT_SILU, gated=True, dbias=self.db, q=self.qz, scales=self.sz, **kw)
        g.gemm_blockscale_fp8(c, self.qz, self.sz, self.upT, self.supT, self.dx, **kw)
        if self.T <= g.GEMMAR_MOE_MAX_TOKENS:
            g.moe_route(c, self.u, self.router, self.ids, self.wts, bias=self.bias, score=g.GEMMAR_SCORE_SIGMOID, **kw)
            g.moe_apply(c, self.q, self.s, self.ids, self.wts, self.w13, self.s13, self.w2, self.s2, self.moe, y=self.u, **kw)

    def outputs(self):
        return [t.clone() for t in (self.t, self.q, self.s, self.z, self.qi, self.si, self.out, self.dinner, self.dz, self.qz, self.sz, self.db,
                                    self.dx, self.ids, self.wts, self.moe)]

    def check(self):
        """Each step against its definition on what the step before it left."""
        ref, err, z, ez = ff.act_reference(self.q, self.s, self.up, self.sup, "silu", True, self.b_up)
        ff.within(self.z, z, ez + ff.BF16 * (z.abs() + ez), "z")
        ff.codes_within(self.qi, self.si, ref, err, "inner")
        ref, err, _, _ = ff.act_reference(self.qi, self.si, self.down, self.sdown, "none", False, None, self.t)
        ff.within(self.out, ref, err + 2.0 ** -24 * ref.abs(), "out")
        zg, zu = self.z.double().chunk(2, 1)
        s, d = torch.sigmoid(zg), self.dinner.double()
        dz = torch.cat([d * zu * s * (1 + zg * (1 - s)), d * zg * s], 1)
        bound = 2.0 ** -19 * d.abs() * (1 + zu.abs() + zg.abs())
        ff.within(self.dz, dz, torch.cat([bound, bound], 1) + ff.BF16 * dz.abs() * 1.01, "dz")
        dx, ex = ff.product(self.qz, self.sz, self.upT, self.supT)
        ff.within(self.dx, dx, ex + ff.BF16 * (dx.abs() + ex), "dx")
        if self.T <= 128:
            l = torch.sigmoid(self.u.double() @ self.router.double().T)
            ids = torch.sort(l + self.bias.double(), dim=1, descending=True, stable=True).indices[:, :self.k]
            assert torch.equal(self.ids, ids.int())


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T", [1, 7, 100, 600])
def test_replay_equals_eager(g, T):
    ctx = context(g)
    try:
        block = Block(g, ctx, T, T)
        block()
        torch.cuda.synchronize()
        block.check()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            block()
        for seed in (11, 12):
            gen = torch.Generator("cuda").manual_seed(seed)
            for t in (block.y, block.h, block.dout):
                t.copy_(torch.randn(t.shape, generator=gen, device="cuda"))
            block()
            eager = block.outputs()
            for t in (block.q, block.qi, block.out, block.dz, block.ids, block.moe):
                t.zero_()
            for _ in range(3):
                graph.replay()
            torch.cuda.synchronize()
            assert same(block.outputs(), eager)
            block.check()
        assert g.gemmar_status(ctx)[0] == 0
    finally:
        ctx.close()


def test_two_graphs_share_a_context(g):
    """Their workspace and counters are the context's: replayed in turn, each leaves them fit for the other."""
    ctx = context(g)
    try:
        blocks = [Block(g, ctx, T, T) for T in (3, 90)]
        graphs, eager = [], []
        for b in blocks:
            b()
            eager.append(b.outputs())
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                b()
        for _ in range(5):
            for graph in graphs:
                graph.replay()
        torch.cuda.synchronize()
        assert all(same(b.outputs(), e) for b, e in zip(blocks, eager))
        assert g.gemmar_status(ctx)[0] == 0
    finally:
        ctx.close()


def test_two_streams_with_a_context_each(g):
    ctxs = [context(g), context(g)]
    try:
        blocks = [Block(g, c, T, T) for c, T in zip(ctxs, (128, 33))]
        expect = []
        for b in blocks:
            b()
            expect.append(b.outputs())
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(10):
            for b, st in zip(blocks, streams):
                b(stream=st)
        torch.cuda.synchronize()
        assert all(same(b.outputs(), e) for b, e in zip(blocks, expect))
        assert all(g.gemmar_status(c)[0] == 0 for c in ctxs)
    finally:
        for c in ctxs:
            c.close()


def test_first_call_in_a_capture(g):
    """A process whose first call of each operator is captured."""
    code = """
import sys; sys.path[:0] = [%r, %r]
import torch, block_scaled_fp8_gemm_gb300 as g
from test_gpu_feedforward_together import Block, context
ctx = context(g)
blocks = [Block(g, ctx, T, T) for T in (5, 64)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for b in blocks: b()
graph.replay(); torch.cuda.synchronize()
for b in blocks: b.check()
assert g.gemmar_status(ctx)[0] == 0
print("captured")
""" % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_offsets_past_32_bits(g):
    """More than 2^31 elements of C, z and dz, and more than 2^32 bytes of experts."""
    ctx = context(g)
    try:
        M, N, K = 65664, 32896, 128
        gen = torch.Generator("cuda").manual_seed(1)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
        A, sa = ff.codes_1x128(rnd(M, K))
        B, sb = ff.codes_128x128(rnd(N, K) * K ** -0.5)
        C, z = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        g.gemm_blockscale_act(ctx, A, sa, B, sb, C, act=g.GEMMAR_ACT_RELU, z=z)
        rows = torch.tensor([0, 1, 65279, 65280, M - 1], device="cuda")
        ref, err, zz, ez = ff.act_reference(A[rows], sa[rows], B, sb, "relu", False)
        ff.within(C[rows], ref, err + ff.BF16 * (ref.abs() + err))
        ff.within(z[rows], zz, ez + ff.BF16 * (zz.abs() + ez))
        g.gemm_blockscale_act_bwd(ctx, C, z, C, act=g.GEMMAR_ACT_RELU)
        assert torch.equal(C[rows], torch.where(z[rows] > 0, z[rows], torch.zeros_like(z[rows])))
        del C, z
        H, I, E = 7168, 2048, 152
        w13, s13 = torch.zeros(E, 2 * I, H, dtype=torch.uint8, device="cuda"), torch.zeros(E, 2 * I // 128, H // 128, device="cuda")
        w2, s2 = torch.zeros(E, H, I, dtype=torch.uint8, device="cuda"), torch.zeros(E, H // 128, I // 128, device="cuda")
        assert w13.numel() > 1 << 32
        w13[-1], s13[-1] = ff.codes_128x128(rnd(2 * I, H) * H ** -0.5)
        w2[-1], s2[-1] = ff.codes_128x128(rnd(H, I) * I ** -0.5)
        x, sx = ff.codes_1x128(rnd(2, H))
        out = torch.empty(2, H, dtype=torch.bfloat16, device="cuda")
        big = context(g, 4096, 7168)
        g.moe_apply(big, x, sx, torch.tensor([[0, E - 1], [E - 1, 3]], dtype=torch.int32, device="cuda"), torch.ones(2, 2, device="cuda"),
                    w13, s13, w2, s2, out)
        h, eh, _, _ = ff.act_reference(x, sx, w13[-1], s13[-1], "silu", True)
        b = ff.values(w2[-1], s2[-1])
        ref = h @ b.T
        bound = (eh + h.abs().view(2, -1, 128).amax(2).repeat_interleave(128, 1) * 2.0 ** -14) @ b.abs().T + 40 * 2.0 ** -23 * (h.abs() @ b.abs().T)
        ff.within(out, ref, bound + ff.BF16 * (ref.abs() + bound))
        big.close()
    finally:
        ctx.close()


def test_refusals(g):
    ctx = context(g, 128, 256)
    e = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32

    def refused(code, call, *args, **kw):
        with pytest.raises(g.GemmarError) as info:
            call(ctx, *args, **kw)
        assert info.value.code == code, info.value

    try:
        M, N, K = 4, 256, 256
        ops = lambda P=N, K=K: (e(M, K, dtype=u8), e(M, K // 128), e(P, K, dtype=u8), e(P // 128, K // 128))
        C, q, s = e(M, N, dtype=bf), e(M, N, dtype=u8), e(M, N // 128)
        act, bwd = g.gemm_blockscale_act, g.gemm_blockscale_act_bwd
        refused(g.GEMMAR_ERR_ARG, act, *ops(), None)                                   # nowhere to go
        refused(g.GEMMAR_ERR_ARG, act, *ops(), C, q=q)                                 # codes without scales
        refused(g.GEMMAR_ERR_ARG, act, *ops(), C, scales=s)
        refused(g.GEMMAR_ERR_ARG, act, *ops(), C, act=5)
        refused(g.GEMMAR_ERR_ARG, act, *ops(), C, act=-1)
        refused(g.GEMMAR_ERR_SHAPE, act, *ops(192), e(M, 192, dtype=bf))               # columns off the 128 grid
        refused(g.GEMMAR_ERR_SHAPE, act, *ops(384), e(M, 192, dtype=bf), gated=True)
        refused(g.GEMMAR_ERR_ARG, act, *ops(), e(1, N, dtype=bf).expand(M, N))         # one row written for all
        refused(g.GEMMAR_ERR_ALIGN, act, *ops(), e(M, N + 4, dtype=bf)[:, :N])         # rows off 16 bytes
        wide = e(M + 1, N)
        refused(g.GEMMAR_ERR_ARG, act, *ops(), wide[1:], residual=wide[:M])            # a row below what it reads
        below = e(M + 1, 2 * N)
        for at, row in ((0, 2), (0, M - 1), (8, 1)):                                   # one row for all, among C's
            refused(g.GEMMAR_ERR_ARG, act, *ops(), below[:M, :N], residual=below[row:row + 1, at:at + N].expand(M, N))
        for at, row in ((N, 2), (0, M)):                                               # beside and below them is fine
            act(ctx, *ops(), below[:M, :N], residual=below[row:row + 1, at:at + N].expand(M, N))
        act(ctx, *ops(), below[1:, N:], residual=below[:1, N:].expand(M, N))           # and above
        o = ops()
        refused(g.GEMMAR_ERR_ARG, act, *o, C, q=o[0], scales=s)                        # codes over A
        refused(g.GEMMAR_ERR_ARG, act, *o, C, q=o[2][:M], scales=s)                    # over B
        both = e(M, N + N)
        act(ctx, *ops(), both[:, :N], residual=both[:, N:])                            # side by side is fine
        z, d = e(M, N, dtype=bf), e(M, N, dtype=bf)
        refused(g.GEMMAR_ERR_ARG, bwd, d, z, None)
        refused(g.GEMMAR_ERR_ARG, bwd, d, e(M, 2 * N, dtype=bf), None, gated=True, q=e(M, 2 * N, dtype=u8))
        zz = e(M + 1, N, dtype=bf)
        refused(g.GEMMAR_ERR_ARG, bwd, d, zz[:M], zz[1:])                              # dz a row below z
        refused(g.GEMMAR_ERR_ARG, bwd, zz[:M], z, zz[1:])
        refused(g.GEMMAR_ERR_ARG, bwd, zz[2:3].expand(M, N), z, zz[1:])                # one row for all, among dz's
        bwd(ctx, zz[:1].expand(M, N), z, zz[1:])                                       # above them is fine
        refused(g.GEMMAR_ERR_ARG, act, *ops(), C, z=zz[:M], residual=zz[2:3].expand(M, N))
        H, I, E, T, k = 256, 128, 4, 3, 2
        r = lambda T=T, k=k, E=E, H=H: (e(T, H, dtype=bf), e(E, H), e(T, k, dtype=i32), e(T, k))
        refused(g.GEMMAR_ERR_ARG, g.moe_route, *r(k=5))                                # more than there are
        refused(g.GEMMAR_ERR_ARG, g.moe_route, *r(), score=2)
        refused(g.GEMMAR_ERR_ARG, g.moe_route, *r(), factor=float("nan"))
        refused(g.GEMMAR_ERR_SHAPE, g.moe_route, *r(T=129))
        refused(g.GEMMAR_ERR_SHAPE, g.moe_route, *r(E=1025))
        refused(g.GEMMAR_ERR_SHAPE, g.moe_route, *r(E=20, k=17))
        refused(g.GEMMAR_ERR_SHAPE, g.moe_route, *r(H=252))
        m = lambda T=T, k=k: (e(T, H, dtype=u8), e(T, H // 128), e(T, k, dtype=i32), e(T, k), e(E, 2 * I, H, dtype=u8), e(E, 2, 2), e(E, H, I, dtype=u8),
                              e(E, 2, 1))
        refused(g.GEMMAR_ERR_SHAPE, g.moe_apply, *m(T=129), e(129, H, dtype=bf))
        refused(g.GEMMAR_ERR_SHAPE, g.moe_apply, *m(k=17), e(T, H, dtype=bf))
        refused(g.GEMMAR_ERR_ARG, g.moe_apply, *m(), e(T, H, dtype=bf), act=9)
        rows = e(T + 1, H, dtype=bf)
        refused(g.GEMMAR_ERR_ARG, g.moe_apply, *m(), rows[1:], y=rows[:T])
        refused(g.GEMMAR_ERR_ARG, g.moe_apply, *m(), rows[1:], y=rows[2:3].expand(T, H))
        g.moe_apply(ctx, *m(), rows[1:], y=rows[:1].expand(T, H))
        refused(g.GEMMAR_ERR_WORKSPACE, g.moe_apply, *m(T=100, k=4), e(100, H, dtype=bf))   # a context of 128 x 256
        torch.cuda.synchronize()
        assert g.gemmar_status(ctx)[0] == 0
    finally:
        ctx.close()
