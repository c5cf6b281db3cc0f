"""Outputs over inputs or over one another: refused by every feed-forward operator, for every pair; side by side is fine."""
import pytest
import torch

pytestmark = pytest.mark.gpu
M, N, K, T, H, INNER, E, KC = 8, 256, 256, 6, 256, 128, 5, 2
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32

# arguments: (shape, dtype, is an output)
CALLS = {
    "gemm_blockscale_act": dict(A=((M, K), U8, 0), sa=((M, K // 128), F32, 0), B=((2 * N, K), U8, 0), sb=((2 * N // 128, K // 128), F32, 0),
                                C=((M, N), BF, 1), bias=((2 * N,), F32, 0), residual=((M, N), BF, 0), q=((M, N), U8, 1),
                                scales=((M, N // 128), F32, 1), z=((M, 2 * N), BF, 1)),
    "gemm_blockscale_act_bwd": dict(dout=((M, N), BF, 0), z=((M, 2 * N), BF, 0), dz=((M, 2 * N), BF, 1), dbias=((2 * N,), F32, 1),
                                    q=((M, 2 * N), U8, 1), scales=((M, 2 * N // 128), F32, 1)),
    "moe_route": dict(x=((T, H), BF, 0), router=((E, H), F32, 0), ids=((T, KC), I32, 1), weights=((T, KC), F32, 1), bias=((E,), F32, 0)),
    "moe_apply": dict(q=((T, H), U8, 0), sx=((T, H // 128), F32, 0), ids=((T, KC), I32, 0), weights=((T, KC), F32, 0),
                      w13=((E, 2 * INNER, H), U8, 0), s13=((E, 2 * INNER // 128, H // 128), F32, 0), w2=((E, H, INNER), U8, 0),
                      s2=((E, H // 128, INNER // 128), F32, 0), out=((T, H), BF, 1), place=((9,), I32, 0), y=((T, H), BF, 0)),
}
FORM = {"gemm_blockscale_act": dict(gated=True), "gemm_blockscale_act_bwd": dict(gated=True), "moe_route": {}, "moe_apply": {}}
ITSELF = {("gemm_blockscale_act", "C", "residual"), ("gemm_blockscale_act_bwd", "dz", "z"), ("moe_apply", "out", "y")}
PAIRS = [(name, o, other) for name, args in CALLS.items() for o, (_, _, out) in args.items() if out
         for other, (_, _, also) in args.items() if other != o and not (also and other < o)]


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def ctx(g):
    torch.cuda.set_device(0)
    c = g.gemmar_create(0, 256, 512, 256, 1, flags=g.GEMMAR_NO_SELF_TEST)
    yield c
    torch.cuda.synchronize()
    assert g.gemmar_status(c)[0] == 0
    c.close()


def nbytes(shape, dtype):
    return torch.Size(shape).numel() * torch.empty(0, dtype=dtype).element_size()


def place(buf, at, shape, dtype):
    return buf[at:at + nbytes(shape, dtype)].view(dtype).view(shape)


def arguments(name):
    return {a: torch.zeros(shape, dtype=dtype, device="cuda") for a, (shape, dtype, _) in CALLS[name].items()}


def call(g, ctx, name, args):
    getattr(g, name)(ctx, **args, **FORM[name])


@pytest.mark.parametrize("name,out,other", PAIRS)
def test_every_pair(g, ctx, name, out, other):
    (os, od, _), (ts, td, _) = CALLS[name][out], CALLS[name][other]
    no, nt = nbytes(os, od), nbytes(ts, td)
    buf = torch.zeros(2 * no + nt + 64, dtype=torch.uint8, device="cuda")
    at = -(-no // 16) * 16
    args = arguments(name)
    args[other] = place(buf, at, ts, td)
    # its first and its last 16 bytes, its start, and the output's end over its start
    for o in {at, at + (nt - 1) // 16 * 16, at - (no - 1) // 16 * 16}:
        if (name, out, other) in ITSELF and o == at and no == nt and od == td:
            continue
        args[out] = place(buf, o, os, od)
        with pytest.raises(g.GemmarError) as e:
            call(g, ctx, name, args)
        assert e.value.code == g.GEMMAR_ERR_ARG, (o - at, e.value)
    for o in (at + -(-nt // 16) * 16, 0 if no % 16 == 0 else None):   # right behind and right before
        if o is not None:
            args[out] = place(buf, o, os, od)
            call(g, ctx, name, args)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name,out,other", sorted(ITSELF))
def test_itself(g, ctx, name, out, other):
    args = arguments(name)
    args[out] = args[other]
    call(g, ctx, name, args)
    torch.cuda.synchronize()


def test_gradient_over_an_ungated_one(g, ctx):
    d = torch.zeros(M, N, dtype=BF, device="cuda")
    g.gemm_blockscale_act_bwd(ctx, d, torch.zeros_like(d), d)
    g.gemm_blockscale_act_bwd(ctx, torch.zeros_like(d), d, d)
    torch.cuda.synchronize()


@pytest.mark.parametrize("name,out,other,cols", [("gemm_blockscale_act", "C", "residual", N), ("moe_apply", "out", "y", H)])
def test_rows_at_two_strides(g, ctx, name, out, other, cols):
    """Views of one buffer whose rows lie at different distances: refused where a row of one meets a row of the other."""
    rows = CALLS[name][out][0][0]
    buf = torch.zeros(64 * cols, dtype=BF, device="cuda")
    a = buf[:rows * 3 * cols].view(rows, 3 * cols)[:, :cols]               # rows 0, 3, 6, ...
    for start, step, meets in ((1, 2, True), (1, 6, False), (2, 6, False), (4, 6, False), (6, 4, True), (3 * rows, 2, False)):
        n = rows * step
        b = buf[start * cols:(start + n) * cols].view(rows, step * cols)[:, :cols]   # rows start, start + step, ...
        assert meets == bool({3 * i for i in range(rows)} & {start + step * i for i in range(rows)})
        for o, i in ((a, b), (b, a)):
            args = arguments(name)
            args[out], args[other] = o, i
            if meets:
                with pytest.raises(g.GemmarError) as e:
                    call(g, ctx, name, args)
                assert e.value.code == g.GEMMAR_ERR_ARG
            else:
                call(g, ctx, name, args)
    torch.cuda.synchronize()


def test_scales_in_the_gaps_of_wider_rows(g, ctx):
    """Contiguous outputs that lie between the rows of C touch none of them."""
    wide = torch.zeros(M, 2 * N, dtype=BF, device="cuda")
    args = arguments("gemm_blockscale_act")
    args["C"] = wide[:, :N]
    args["scales"] = wide[0, N:].view(F32)[:M * N // 128].view(M, N // 128)
    call(g, ctx, "gemm_blockscale_act", args)
    args["scales"] = wide.view(-1)[2 * N - 8:].view(F32)[:M * N // 128].view(M, N // 128)   # 16 bytes before row 1
    with pytest.raises(g.GemmarError) as e:
        call(g, ctx, "gemm_blockscale_act", args)
    assert e.value.code == g.GEMMAR_ERR_ARG
    torch.cuda.synchronize()
