"""lora_plan, lora_apply and lora_apply_bwd against the formulas in 64 bits.

Tolerances.  A bf16 output is one rounding of an fp32 value: 2^-8 of it.  An fp32 sum is a
chain of at most 256 additions (2^-16 of the sum of magnitudes), and the inner factor
enters the outer product as two bf16 parts (2^-16 of it): 2^-15 of the sums of magnitudes
covers each product."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U_BF16 = 2.0 ** -8
SUM = 2.0 ** -15


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def ctx(g):
    torch.cuda.set_device(0)
    c = g.gemmar_create(0, 4096, 7168, 2048, 1, flags=g.GEMMAR_NO_SELF_TEST, wait_timeout_ns=500_000_000)
    yield c
    c.close()


def plan(g, ctx, ids, R):
    order = torch.empty(len(ids), dtype=torch.int32, device="cuda")
    offsets = torch.empty(R + 1, dtype=torch.int32, device="cuda")
    g.lora_plan(ctx, ids, order, offsets)
    return order, offsets


def make(g, ctx, ids, R, r, K, N, seed=0, ranks="mixed"):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    T = len(ids)
    ids = torch.as_tensor(ids, dtype=torch.int32, device="cuda")
    d = {"ids": ids, "x": rnd(T, K).bfloat16(), "y": rnd(T, N).bfloat16(), "dy": rnd(T, N).bfloat16(), "dx0": rnd(T, K).bfloat16(),
         "A": (rnd(R, r, K) * K ** -0.5).bfloat16(), "B": (rnd(R, r, N) * 0.5).bfloat16(), "scales": 0.5 + torch.rand(R, generator=gen, device="cuda")}
    d["ranks"] = None if ranks is None else torch.tensor([(r, 1, (r + 1) // 2, 0)[a % 4] for a in range(R)], dtype=torch.int32, device="cuda")
    if d["ranks"] is not None:
        for a in range(R):   # rows past an adapter's rank are not read
            d["A"][a, int(d["ranks"][a]):] = float("nan")
            d["B"][a, int(d["ranks"][a]):] = float("nan")
    d["order"], d["offsets"] = plan(g, ctx, ids, R)
    return d


def weights(d, a):
    k = d["A"].shape[1] if d["ranks"] is None else int(d["ranks"][a])
    return d["A"][a, :k].double(), d["B"][a, :k].double(), float(d["scales"][a]), k


def apply(g, ctx, d, y="y", v=True, stream=None, out=None):
    T, N, r = len(d["ids"]), d["B"].shape[2], d["A"].shape[1]
    out = torch.empty(T, N, dtype=torch.bfloat16, device="cuda") if out is None else out
    v = torch.full((T, r), 77.0, device="cuda") if v else None
    g.lora_apply(ctx, d["x"], d["order"], d["offsets"], d["A"], d["B"], d["scales"], d["ranks"], out,
                 y=d[y] if y else None, v=v, stream=stream)
    return out, v


def apply_bwd(g, ctx, d, v, dx0="dx0", stream=None):
    dx, dA, dB = torch.empty_like(d["dx0"]), torch.empty_like(d["A"]), torch.empty_like(d["B"])
    g.lora_apply_bwd(ctx, d["x"], d["dy"], d["order"], d["offsets"], d["A"], d["B"], d["scales"], d["ranks"], v, dx, dA, dB,
                     dx0=d[dx0] if dx0 else None, stream=stream)
    return dx, dA, dB


def close(got, ref, mag, what, u=U_BF16):
    err = (got.double() - ref).abs()
    worst = (err / (u * ref.abs() * (1 + 1e-3) + SUM * mag + 1e-37)).max().item() if err.numel() else 0.0
    assert worst <= 1, (what, worst)


def check_apply(d, out, v, y="y"):
    base = d[y].double() if y else torch.zeros_like(d["y"], dtype=torch.float64)
    ref, mag = base.clone(), base.abs() * 0
    at = d["offsets"].tolist()
    for a in range(d["A"].shape[0]):
        rows = d["order"][at[a]:at[a + 1]].long()
        A, B, s, k = weights(d, a)
        x = d["x"][rows].double()
        vr, vm = x @ A.T, x.abs() @ A.abs().T
        if v is not None:
            close(v[at[a]:at[a + 1], :k], vr, vm, "v", 0.0)
            assert (v[at[a]:at[a + 1], k:] == 0).all()
        ref[rows] += s * vr @ B
        mag[rows] = 2 * s * vm @ B.abs()
    close(out, ref, mag, "out")
    bare = d["order"][at[-1]:].long()
    assert torch.equal(out[bare].float(), base[bare].float())
    if v is not None:
        assert (v[at[-1]:] == 77.0).all()


def check_bwd(d, v, dx, dA, dB, dx0="dx0"):
    base = d[dx0].double() if dx0 else torch.zeros_like(d["dx0"], dtype=torch.float64)
    ref, mag = base.clone(), base.abs() * 0
    at = d["offsets"].tolist()
    for a in range(d["A"].shape[0]):
        rows = d["order"][at[a]:at[a + 1]].long()
        A, B, s, k = weights(d, a)
        x, dy, va = d["x"][rows].double(), d["dy"][rows].double(), v[at[a]:at[a + 1], :k].double()
        w, wm = s * dy @ B.T, s * dy.abs() @ B.abs().T
        ref[rows] += w @ A
        mag[rows] = 2 * wm @ A.abs()
        close(dA[a, :k], w.T @ x, 2 * wm.T @ x.abs(), "dA")
        close(dB[a, :k], s * va.T @ dy, 2 * s * va.abs().T @ dy.abs(), "dB")
        assert (dA[a, k:] == 0).all() and (dB[a, k:] == 0).all()
    close(dx, ref, mag, "dx")
    bare = d["order"][at[-1]:].long()
    assert torch.equal(dx[bare].float(), base[bare].float())


def mixed_ids(T, R, seed, bare=0.2):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, R, T)
    ids[rng.random(T) < bare] = -1
    return ids.astype(np.int32)


def runs(*pairs):
    return np.concatenate([np.full(n, a, np.int32) for a, n in pairs])


CASES = [
    # ids, R, r, K, N
    ("one token", [0], 1, 16, 2048, 7168),
    ("one token without", [-1], 3, 8, 64, 64),
    ("tiny", [1, 0, 1], 2, 1, 8, 8),
    ("decode", mixed_ids(33, 20, 1), 20, 16, 1024, 1544),
    ("decode, many of one", runs((2, 40), (0, 1), (-1, 3)), 4, 24, 520, 264),
    ("ranks odd", mixed_ids(130, 5, 2), 5, 33, 264, 392),
    ("prefill runs", runs((1, 200), (0, 129), (-1, 31), (2, 128), (1, 65)), 6, 32, 2048, 512),
    ("prefill mixed", mixed_ids(1100, 7, 3), 7, 64, 520, 1032),
    ("rank 128", mixed_ids(300, 3, 4, 0.0), 3, 128, 384, 640),
    ("all without", np.full(50, -1, np.int32), 2, 16, 128, 128),
    ("many adapters", mixed_ids(700, 300, 5), 300, 8, 128, 136),
    ("one large", np.zeros(2000, np.int32), 1, 16, 256, 264),
]


@pytest.mark.parametrize("name,ids,R,r,K,N", CASES, ids=[c[0] for c in CASES])
def test_apply_and_gradients(g, ctx, name, ids, R, r, K, N):
    d = make(g, ctx, ids, R, r, K, N, seed=len(ids) + r)
    out, v = apply(g, ctx, d)
    check_apply(d, out, v)
    check_bwd(d, v, *apply_bwd(g, ctx, d, v))
    assert g.gemmar_status(ctx)[0] == 0


@pytest.mark.parametrize("T,r", [(1, 7), (50, 16), (600, 48)])
def test_without_base_ranks_or_v(g, ctx, T, r):
    d = make(g, ctx, mixed_ids(T, 4, T), 4, r, 512, 768, seed=T, ranks=None)
    out, v = apply(g, ctx, d, y=None)
    check_apply(d, out, v, y=None)
    same, _ = apply(g, ctx, d, y=None, v=False)
    assert torch.equal(out, same)
    check_bwd(d, v, *apply_bwd(g, ctx, d, v, dx0=None), dx0=None)


@pytest.mark.parametrize("T", [5, 700])
def test_views_streams_in_place_and_repeatability(g, ctx, T):
    K, N = 264, 520
    d = make(g, ctx, mixed_ids(T, 3, 8), 3, 16, K, N, seed=4)
    out, v = apply(g, ctx, d)
    grads = apply_bwd(g, ctx, d, v)
    torch.cuda.synchronize()
    w = dict(d)
    for k in ("x", "y", "dy", "dx0"):
        wide = torch.full((T, d[k].shape[1] + 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        w[k] = wide[:, 24:24 + d[k].shape[1]]
        w[k].copy_(d[k])
    big = torch.full((T, N + 40), 5.0, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    apply(g, ctx, w, stream=side, out=big[:, 8:8 + N])
    w["dx0"] = d["dx0"]
    again = apply_bwd(g, ctx, w, v, stream=side)
    side.synchronize()
    assert torch.equal(big[:, 8:8 + N], out) and (big[:, :8] == 5).all() and (big[:, 8 + N:] == 5).all()
    assert all(torch.equal(a, b) for a, b in zip(again, grads))
    y = d["y"].clone()
    d2 = dict(d, y=y)
    apply(g, ctx, d2, out=y)
    assert torch.equal(y, out)
    dx = d["dx0"].clone()
    g.lora_apply_bwd(ctx, d["x"], d["dy"], d["order"], d["offsets"], d["A"], d["B"], d["scales"], d["ranks"], v, dx,
                     torch.empty_like(d["A"]), torch.empty_like(d["B"]), dx0=dx)
    assert torch.equal(dx, grads[0])


@pytest.mark.parametrize("T,r", [(24, 16), (900, 32)])
def test_non_finite_tokens_and_adapters_stay_apart(g, ctx, T, r):
    d = make(g, ctx, mixed_ids(T, 4, 6), 4, r, 256, 384, seed=6, ranks=None)
    out, v = apply(g, ctx, d)
    grads = apply_bwd(g, ctx, d, v)
    bad = {k: (t.clone() if isinstance(t, torch.Tensor) else t) for k, t in d.items()}
    sick = torch.nonzero(d["ids"] == 1)[0, 0].item()
    other = torch.nonzero(d["ids"] < 0)[0, 0].item()
    bad["x"][sick, 3] = float("nan")
    bad["dy"][sick, 9] = float("inf")
    bad["x"][other] = float("nan")        # a token without an adapter is not read
    bad["dy"][other] = float("nan")
    bad["A"][2] = float("inf")            # an adapter of its own tokens only
    o, v2 = apply(g, ctx, bad)
    b = apply_bwd(g, ctx, bad, v2)
    rows = (d["ids"] != 2) & (torch.arange(T, device="cuda") != sick)
    assert torch.equal(o[rows], out[rows]) and torch.equal(b[0][rows], grads[0][rows])
    assert not torch.isfinite(o[sick].float()).all()
    for a in (0, 3):
        assert torch.equal(b[1][a], grads[1][a]) and torch.equal(b[2][a], grads[2][a])
    assert torch.equal(b[2][1][:, torch.arange(384, device="cuda") != 9].isnan().any(1), torch.ones(r, dtype=torch.bool, device="cuda"))


@pytest.mark.parametrize("T", [1, 3, 31, 32, 33, 1000, 4096, 100000])
@pytest.mark.parametrize("R", [1, 5, 64, 1024])
def test_plan(g, ctx, T, R):
    ids = torch.from_numpy(mixed_ids(T, R, T + R)).cuda()
    if T > 4:
        ids[2], ids[3] = R + 9, -2147483648       # outside [0, R): no adapter
    order, offsets = plan(g, ctx, ids, R)
    key = torch.where((ids < 0) | (ids >= R), torch.full_like(ids, R), ids)
    assert torch.equal(order.long(), torch.sort(key, stable=True).indices)
    assert offsets.tolist() == torch.searchsorted(torch.sort(key).values, torch.arange(R + 1, device="cuda", dtype=torch.int32)).tolist()


def test_entries_outside_the_batch_are_skipped(g, ctx):
    d = make(g, ctx, [0, 0, 1, 1, 0, 1, 0], 2, 8, 64, 64, seed=3, ranks=None)
    out, v = apply(g, ctx, d)
    d["order"][1], d["order"][6] = -5, 1 << 30
    gone = {1, 5}   # the tokens that those places named
    keep = torch.tensor([t not in gone for t in range(7)], device="cuda")
    o, _ = apply(g, ctx, d)
    assert torch.equal(o[keep], out[keep])
    dx, dA, dB = apply_bwd(g, ctx, d, v)
    assert torch.isfinite(dA.float()).all() and torch.isfinite(dB.float()).all() and torch.isfinite(dx[keep].float()).all()


def test_tokens_past_32_bit_offsets(g, ctx):
    T, K, N, stride = 131100, 64, 64, 16400   # 2.15e9 elements from the first token to the last
    big = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (T, K), (stride, 1))
    ids = torch.full((T,), -1, dtype=torch.int32)
    ids[:5] = 1
    ids[-300:] = 0
    d = make(g, ctx, ids, 2, 16, K, N, seed=8, ranks=None)
    x.copy_(d["x"])
    out, v = apply(g, ctx, d)
    grads = apply_bwd(g, ctx, d, v)
    d["x"] = x
    o, _ = apply(g, ctx, d)
    assert torch.equal(o, out)
    assert all(torch.equal(a, b) for a, b in zip(apply_bwd(g, ctx, d, v), grads))


@pytest.mark.parametrize("T,r", [(40, 16), (500, 40)])
def test_gradient_against_differences(g, ctx, T, r):
    """out is linear in x, in A and in B, so a central difference has no curvature: along a gradient's own
    direction only the bf16 rounding of out is left, below 1% of the change: 2%."""
    d = make(g, ctx, mixed_ids(T, 3, 9, 0.1), 3, r, 256, 512, seed=12, ranks=None)
    _, v = apply(g, ctx, d)
    dx, dA, dB = apply_bwd(g, ctx, d, v, dx0=None)
    for name, grad in (("x", dx), ("A", dA), ("B", dB)):
        gr = grad.double()
        step = 0.2 * gr / gr.square().mean().sqrt() * d[name].double().square().mean().sqrt()
        ends = [dict(d, **{name: (d[name].double() + sg * step).bfloat16()}) for sg in (1, -1)]
        change = sum(sg * (apply(g, ctx, e)[0].double() * d["dy"].double()).sum().item() for sg, e in zip((1, -1), ends))
        expect = (gr * (ends[0][name].double() - ends[1][name].double())).sum().item()
        assert abs(change - expect) <= 0.02 * abs(expect), (name, change, expect)


def test_refusals(g, ctx):
    d = make(g, ctx, [0, 1, -1], 2, 8, 64, 128, seed=1, ranks=None)

    def code(fn, *a, **kw):
        with pytest.raises(g.GemmarError) as e:
            fn(ctx, *a, **kw)
        return e.value.code
    ops = lambda **kw: [dict(d, **kw)[k] for k in ("x", "order", "offsets", "A", "B", "scales", "ranks")]
    out = torch.empty(3, 128, dtype=torch.bfloat16, device="cuda")
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")
    assert code(g.lora_apply, *ops(scales=None), out) == g.GEMMAR_ERR_ARG
    assert code(g.lora_apply, *ops(x=bf(3, 60), A=bf(2, 8, 60)), out) == g.GEMMAR_ERR_SHAPE
    assert code(g.lora_apply, *ops(A=bf(2, 129, 64), B=bf(2, 129, 128)), out) == g.GEMMAR_ERR_SHAPE
    assert code(g.lora_apply, *ops(x=bf(3, 72)[:, 4:68]), out) == g.GEMMAR_ERR_ALIGN
    assert code(g.lora_apply, *ops(x=bf(3, 68)[:, :64]), out) == g.GEMMAR_ERR_ALIGN      # a stride of 136 bytes
    assert code(g.lora_apply, *ops(), out[:1].expand(3, 128)) == g.GEMMAR_ERR_ARG        # one row for all outputs
    many = torch.zeros(1026, dtype=torch.int32, device="cuda")
    assert code(g.lora_plan, d["ids"], d["order"], many) == g.GEMMAR_ERR_SHAPE
    assert code(g.lora_plan, d["ids"], d["order"], many[:1]) == g.GEMMAR_ERR_ARG         # no adapter at all
    with pytest.raises(TypeError):
        g.lora_apply(ctx, *ops(x=d["x"].float()), out)
    with pytest.raises(ValueError):
        g.lora_apply(ctx, *ops(), out[:2])
    with pytest.raises(ValueError):
        g.lora_apply(ctx, *ops(B=bf(2, 9, 128)), out)
    small = g.gemmar_create(0, 1, 128, 128, 1, flags=g.GEMMAR_NO_SELF_TEST)
    try:
        e = make(g, ctx, np.zeros(4096, np.int32), 1, 64, 64, 64, seed=2, ranks=None)
        with pytest.raises(g.GemmarError) as err:
            apply(g, small, e)
        assert err.value.code == g.GEMMAR_ERR_WORKSPACE
    finally:
        small.close()
    assert g.gemmar_status(ctx)[0] == 0


def test_offsets_that_are_no_plan_stay_in_bounds(g, ctx):
    """Offsets that go back and forth name every token for every adapter: the result means nothing, but
    nothing outside the outputs is written, and the next call is right."""
    T, R, r, K, N = 900, 6, 16, 256, 384
    d = make(g, ctx, mixed_ids(T, R, 3), R, r, K, N, seed=5, ranks=None)
    out, v = apply(g, ctx, d)
    grads = apply_bwd(g, ctx, d, v)
    bad = dict(d, offsets=torch.tensor([0, T, 0, T, -7, 1 << 30, 0], dtype=torch.int32, device="cuda"))
    fenced = torch.full((T + 8, N), 3.0, dtype=torch.bfloat16, device="cuda")
    apply(g, ctx, bad, out=fenced[4:T + 4])
    assert (fenced[:4] == 3).all() and (fenced[T + 4:] == 3).all()
    fence = {k: torch.full((n + 64,), 3.0, dtype=torch.bfloat16, device="cuda") for k, n in (("dx", T * K), ("dA", R * r * K), ("dB", R * r * N))}
    inner = [fence[k][32:-32].view(s) for k, s in (("dx", (T, K)), ("dA", (R, r, K)), ("dB", (R, r, N)))]
    g.lora_apply_bwd(ctx, d["x"], d["dy"], d["order"], bad["offsets"], d["A"], d["B"], d["scales"], d["ranks"], v, *inner, dx0=d["dx0"])
    assert all((f[:32] == 3).all() and (f[-32:] == 3).all() for f in fence.values())
    assert torch.equal(apply(g, ctx, d)[0], out)
    assert all(torch.equal(a, b) for a, b in zip(apply_bwd(g, ctx, d, v), grads))
    assert g.gemmar_status(ctx)[0] == 0


@pytest.mark.parametrize("T,r", [(2900, 20), (2750, 64)])
def test_tiles_and_columns_for_four_ctas_an_sm(g, ctx, T, r):
    """The second product's shorter ring, taken where its CTAs are many; a last step of part of its columns."""
    ids = mixed_ids(T, 4, seed=T)
    d = make(g, ctx, ids, 4, r, 136, 7160, seed=T)
    out, v = apply(g, ctx, d)
    check_apply(d, out, v)
    d = make(g, ctx, ids, 4, r, 7160, 136, seed=T + 1)
    _, v = apply(g, ctx, d)
    check_bwd(d, v, *apply_bwd(g, ctx, d, v))
