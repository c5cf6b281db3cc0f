"""moe_route and moe_apply against their definitions in fp64."""
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
    c = g.gemmar_create(0, 4096, 4096, 256, 1, flags=g.GEMMAR_NO_SELF_TEST)
    yield c
    assert g.gemmar_status(c)[0] == 0
    c.close()


# ---------------------------------------------------------------- moe_route

def route(g, ctx, x, w, k, **kw):
    T = x.shape[0]
    ids = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    weights = torch.full((T, k), 77.0, device="cuda")
    g.moe_route(ctx, x, w, ids, weights, **kw)
    torch.cuda.synchronize()
    return ids, weights


def route_reference(x, w, k, bias=None, score=0, renorm=True, factor=1.0):
    l = x.double() @ w.double().T
    p = torch.softmax(l, 1) if score == 0 else torch.sigmoid(l)
    by = p if bias is None else p + bias.double()
    order = torch.sort(by, dim=1, descending=True, stable=True)
    ids, ok = order.indices[:, :k], order.values[:, :k] > -float("inf")
    wt = torch.where(ok, p.gather(1, ids), 0.0)
    if renorm:
        wt = wt / wt.sum(1, keepdim=True).clamp(min=1e-300)
    # an fp32 logit is off by the roundings of its chain, at most 64, relative to its terms' sizes
    el = 64 * 2.0 ** -24 * (x.double().abs() @ w.double().abs().T).amax(1, keepdim=True)
    return torch.where(ok, ids, -1).int(), wt * factor, (4 * el + 2.0 ** -20) * wt * abs(factor) + 1e-30


def router(T, H, E, seed, dtype=torch.bfloat16):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    return rnd(T, H).bfloat16(), (rnd(E, H) * H ** -0.5).to(dtype), rnd(E) * 0.2


def check_route(got, ref):
    assert torch.equal(got[0], ref[0])
    ff.within(got[1], ref[1], ref[2])


@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 31, 64, 127, 128])
@pytest.mark.parametrize("E,k", [(1, 1), (4, 2), (20, 3), (64, 8), (65, 8), (256, 8), (257, 16)])
def test_route_sizes(g, ctx, T, E, k):
    x, w, _ = router(T, 520, E, T * E)
    check_route(route(g, ctx, x, w, k), route_reference(x, w, k))


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("biased", [False, True])
def test_route_forms(g, ctx, score, renorm, dtype, biased):
    x, w, bias = router(33, 1024, 96, 5, dtype)
    kw = dict(bias=bias if biased else None, score=score, renorm=renorm, factor=2.5)
    check_route(route(g, ctx, x, w, 6, **kw), route_reference(x, w, 6, **kw))


@pytest.mark.parametrize("H", [8, 16, 264, 7168])
def test_route_widths_and_views(g, ctx, H):
    x, w, _ = router(12, H, 1024, H)
    wide = torch.zeros(12, H + 24, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + H] = x
    ref = route_reference(x, w, 4)
    check_route(route(g, ctx, wide[:, 16:16 + H], w, 4), ref)
    row = x[:1].expand(12, H)
    check_route(route(g, ctx, row, w, 4), route_reference(row, w, 4))


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("biased", [False, True])
def test_route_scores_that_fp32_cannot_tell_apart(g, ctx, score, biased):
    """Experts in pairs whose logits differ by less than fp32's rounding of them, in either order."""
    T, H, E = 40, 2048, 64
    x, w, _ = router(T, H, E, 6, torch.float32)
    gen = torch.Generator("cuda").manual_seed(7)
    w[1::2] = w[0::2]
    turn = torch.rand(E // 2, generator=gen, device="cuda") < 0.5
    at = torch.arange(E // 2, device="cuda") * 2 + turn
    # the smallest change of one weight moves a logit by 2^-30 or so, up or down by x's sign
    w[at, 100] = torch.nextafter(w[at, 100], w[at, 100] + 1)
    bias = torch.zeros(E, device="cuda") if biased else None
    check_route(route(g, ctx, x, w, 8, bias=bias, score=score), route_reference(x, w, 8, bias=bias, score=score))


@pytest.mark.parametrize("biased", [False, True])
def test_route_near_pairs_among_distant_ones(g, ctx, biased):
    """Some of a token's choices are told apart in fp32 and some are not, in one order."""
    T, H, E = 40, 7168, 256
    x, w, bias = router(T, H, E, 18, torch.float32)
    bias = (bias * 64).round() if biased else None
    gen = torch.Generator("cuda").manual_seed(19)
    pick = torch.randperm(E, generator=gen, device="cuda")
    w[pick[:60]] = w[pick[60:120]]
    w[pick[:60], 300] = torch.nextafter(w[pick[:60], 300], w[pick[:60], 300] - 1)
    if biased:
        bias[pick[:60]] = bias[pick[60:120]]
    check_route(route(g, ctx, x, w, 16, bias=bias, score=1), route_reference(x, w, 16, bias=bias, score=1))


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T", [1, 40])
def test_route_saturated_scores(g, ctx, score, T):
    """Logits of many tens: most scores are 0 or 1 to fp32, the order is still the logits', and no slower."""
    x, w, _ = router(T, 1024, 64, 16)
    w = (w.float() * 80).bfloat16()
    ids, weights = route(g, ctx, x, w, 8, score=score)
    l = x.double() @ w.double().T
    assert torch.equal(ids, torch.sort(l, dim=1, descending=True, stable=True).indices[:, :8].int())
    p = torch.softmax(l, 1) if score == 0 else torch.sigmoid(l)
    p = p.gather(1, ids.long())
    el = 64 * 2.0 ** -24 * (x.double().abs() @ w.double().abs().T).amax(1, keepdim=True)
    ff.within(weights, p / p.sum(1, keepdim=True), 4 * el + 2.0 ** -20)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(10):
        g.moe_route(ctx, x, w, ids, weights, score=score)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) < 10   # ms; a token that is decided in 64 bits takes some microseconds


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T", [1, 40])
def test_route_chosen_scores_too_small_for_fp32(g, ctx, score, T):
    """The bias takes out the experts that have all of the softmax, or all logits are far below 0."""
    x, w, bias = router(T, 1024, 64, 17)
    x[:, 0], w[:, 0] = 1, -150
    w[:32, 0] = 50
    bias[:] = 0
    bias[:32] = -float("inf")
    for kw in (dict(bias=bias, score=score), dict(bias=bias, score=score, factor=2.5, renorm=False)):
        check_route(route(g, ctx, x, w, 6, **kw), route_reference(x, w, 6, **kw))
    check_route(route(g, ctx, x, w[32:], 6, score=score), route_reference(x, w[32:], 6, score=score))


@pytest.mark.parametrize("score", [0, 1])
def test_route_equal_scores_take_the_lowest(g, ctx, score):
    x, w, _ = router(20, 256, 48, 8)
    x[4] = 0                                   # a padded row: every logit is 0
    w[10:30] = w[5]
    check_route(route(g, ctx, x, w, 8, score=score), route_reference(x, w, 8, score=score))
    ids, weights = route(g, ctx, x, w, 8, score=score)
    assert ids[4].tolist() == list(range(8)) and torch.allclose(weights[4], torch.full((8,), 0.125, device="cuda"))


def test_route_masked_experts(g, ctx):
    x, w, bias = router(9, 256, 12, 9)
    bias[:9] = -float("inf")
    bias[10] = float("nan")
    ids, weights = route(g, ctx, x, w, 4, bias=bias)
    assert set(ids[:, :2].flatten().tolist()) == {9, 11} and (ids[:, 2:] == -1).all() and (weights[:, 2:] == 0).all()
    assert torch.allclose(weights.sum(1), torch.ones(9, device="cuda"))
    ids, weights = route(g, ctx, x, w, 4, bias=torch.full((12,), -float("inf"), device="cuda"))
    assert (ids == -1).all() and (weights == 0).all()


def test_route_a_row_of_nan_stays_alone(g, ctx):
    x, w, _ = router(30, 256, 40, 10)
    clean = route(g, ctx, x, w, 5)
    x[13, 7] = float("nan")
    got = route(g, ctx, x, w, 5)
    keep = torch.arange(30, device="cuda") != 13
    assert all(torch.equal(a[keep], b[keep]) for a, b in zip(got, clean))
    assert (got[0][13] == -1).all() and (got[1][13] == 0).all()


# ---------------------------------------------------------------- moe_apply

def layer(T, H, I, E, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")
    w13 = [ff.codes_128x128(rnd(2 * I, H) * 1.5 * H ** -0.5) for _ in range(E)]
    w2 = [ff.codes_128x128(rnd(H, I) * I ** -0.5) for _ in range(E)]
    s = {"w13": torch.stack([a for a, _ in w13]), "s13": torch.stack([a for _, a in w13]),
         "w2": torch.stack([a for a, _ in w2]), "s2": torch.stack([a for _, a in w2])}
    s["q"], s["sx"] = ff.codes_1x128(rnd(T, H))
    s["y"] = rnd(T, H).bfloat16()
    return s, rnd, gen


def picks(T, k, E, gen, none=0.0):
    ids = torch.stack([torch.randperm(E, generator=gen, device="cuda")[:k] for _ in range(T)]).int()
    ids[torch.rand(T, k, generator=gen, device="cuda") < none] = -1
    return ids, torch.rand(T, k, generator=gen, device="cuda") + 0.1


def apply(g, ctx, s, ids, weights, act="silu", y=True, place=None):
    out = torch.full(s["q"].shape, 77, dtype=torch.bfloat16, device="cuda")
    g.moe_apply(ctx, s["q"], s["sx"], ids, weights, s["w13"], s["s13"], s["w2"], s["s2"], out, act=ff.ACTS.index(act),
                y=s["y"] if y else None, place=place)
    torch.cuda.synchronize()
    return out


def check_layer(out, s, ids, weights, act="silu", y=True):
    """The bound: both products' as in gemm_blockscale_act, the hidden values' parts 2^-14 of their group's
    largest, one addition per expert, and the one rounding to bf16."""
    T, H = s["q"].shape
    ref = s["y"].double() if y else torch.zeros(T, H, dtype=torch.float64, device="cuda")
    err, sizes = torch.zeros_like(ref), ref.abs()
    E, I = s["w2"].shape[0], s["w2"].shape[2]
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        if not len(t):
            continue
        h, eh, _, _ = ff.act_reference(s["q"][t], s["sx"][t], s["w13"][e], s["s13"][e], act, True)
        w = weights[t, j].double()[:, None]
        h, eh = h * w, eh * w.abs() + 2.0 ** -23 * (h * w).abs()
        parts = h.abs().view(len(t), -1, 128).amax(2).repeat_interleave(128, 1) * 2.0 ** -14
        b = ff.values(s["w2"][e], s["s2"][e])
        ref.index_add_(0, t, h @ b.T)
        size = h.abs() @ b.abs().T
        err.index_add_(0, t, (eh + parts) @ b.abs().T + (12 + I // 128) * 2.0 ** -23 * size)
        sizes.index_add_(0, t, size)
    err = err + (ids.shape[1] + 4) * 2.0 ** -23 * sizes
    ff.within(out, ref, err + ff.BF16 * (ref.abs() + err))


@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 16, 17, 33, 64, 65, 100, 128])
@pytest.mark.parametrize("H,I,E,k", [(256, 128, 4, 2), (640, 384, 9, 4), (1024, 512, 20, 8)])
def test_layer_sizes(g, ctx, T, H, I, E, k):
    s, rnd, gen = layer(T, H, I, E, T)
    ids, weights = picks(T, k, E, gen)
    check_layer(apply(g, ctx, s, ids, weights), s, ids, weights)


@pytest.mark.parametrize("act", ff.ACTS)
def test_layer_activations(g, ctx, act):
    s, rnd, gen = layer(21, 384, 256, 6, 1)
    ids, weights = picks(21, 3, 6, gen)
    check_layer(apply(g, ctx, s, ids, weights, act, y=False), s, ids, weights, act, y=False)


@pytest.mark.parametrize("H,I,E,k,T", [(128, 128, 1, 1, 1), (128, 128, 1, 1, 128), (7168, 128, 3, 1, 5), (128, 4096, 3, 2, 70), (2048, 768, 40, 16, 24)])
def test_layer_extremes(g, ctx, H, I, E, k, T):
    s, rnd, gen = layer(T, H, I, E, 2)
    ids, weights = picks(T, k, E, gen)
    check_layer(apply(g, ctx, s, ids, weights), s, ids, weights)


@pytest.mark.parametrize("T", [1, 40, 128])
def test_all_tokens_to_one_expert(g, ctx, T):
    s, rnd, gen = layer(T, 512, 384, 5, 3)
    ids, weights = torch.full((T, 1), 3, dtype=torch.int32, device="cuda"), torch.rand(T, 1, generator=gen, device="cuda")
    check_layer(apply(g, ctx, s, ids, weights), s, ids, weights)


@pytest.mark.parametrize("T", [1, 30, 128])
def test_tokens_without_an_expert(g, ctx, T):
    """Ids outside the experts add nothing: rows are y, or zero; NaN weights beside them are not read."""
    s, rnd, gen = layer(T, 256, 256, 6, 4)
    ids, weights = picks(T, 4, 6, gen, none=0.6)
    ids[0] = torch.tensor([-1, 6, 1 << 30, -(1 << 31)], dtype=torch.int32)
    weights[0] = float("nan")
    out = apply(g, ctx, s, ids, weights)
    assert torch.equal(out[0], s["y"][0])
    check_layer(out, s, ids, torch.nan_to_num(weights))
    none = torch.full_like(ids, -1)
    assert torch.equal(apply(g, ctx, s, none, weights), s["y"])
    assert (apply(g, ctx, s, none, weights, y=False) == 0).all()


def test_an_expert_twice(g, ctx):
    s, rnd, gen = layer(10, 256, 256, 3, 5)
    ids = torch.randint(0, 3, (10, 4), generator=gen, device="cuda", dtype=torch.int32)
    weights = torch.rand(10, 4, generator=gen, device="cuda")
    check_layer(apply(g, ctx, s, ids, weights), s, ids, weights)


def test_place(g, ctx):
    """Experts held elsewhere are left out; the router's numbers are not this GPU's rows."""
    s, rnd, gen = layer(25, 384, 256, 5, 6)
    place = torch.full((16,), -1, dtype=torch.int32, device="cuda")
    place[[2, 3, 7, 11, 15]] = torch.tensor([4, 0, 2, 1, 3], dtype=torch.int32, device="cuda")
    place[5] = 99                              # outside the experts: none
    ids, weights = picks(25, 6, 16, gen)
    ids[3, 0] = 16                             # outside the router's numbers: none
    here = torch.where(ids < 16, place[ids.clamp(max=15).long()], -1).int()
    check_layer(apply(g, ctx, s, ids, weights, place=place), s, here, weights)


def test_in_place_and_views(g, ctx):
    s, rnd, gen = layer(19, 256, 128, 4, 7)
    ids, weights = picks(19, 2, 4, gen)
    want = apply(g, ctx, s, ids, weights)
    wide = torch.zeros(19, 320, dtype=torch.bfloat16, device="cuda")
    view = wide[:, 64:]
    view.copy_(s["y"])
    g.moe_apply(ctx, s["q"], s["sx"], ids, weights, s["w13"], s["s13"], s["w2"], s["s2"], view, y=view)
    torch.cuda.synchronize()
    assert torch.equal(view, want) and (wide[:, :64] == 0).all()


def test_a_row_of_nan_stays_alone(g, ctx):
    s, rnd, gen = layer(40, 512, 256, 6, 8)
    ids, weights = picks(40, 3, 6, gen)
    clean = apply(g, ctx, s, ids, weights)
    s["q"][17, 300] = 0x7F
    out = apply(g, ctx, s, ids, weights)
    keep = torch.arange(40, device="cuda") != 17
    assert torch.isnan(out[17].float()).all() and torch.equal(out[keep], clean[keep])


def test_large_and_small_hidden_values(g, ctx):
    """Groups of hidden values of very different sizes keep their accuracy."""
    s, rnd, gen = layer(12, 256, 512, 4, 9)
    s["s13"] = s["s13"] * torch.logspace(-6, 6, 8, device="cuda").view(1, 8, 1)
    ids, weights = picks(12, 2, 4, gen)
    check_layer(apply(g, ctx, s, ids, weights, y=False), s, ids, weights, y=False)


@pytest.mark.parametrize("act", ["relu", "silu"])
@pytest.mark.parametrize("tiny", [1e-30, 1e-36, 1e-38, 1e-40, 1e-45])
def test_weights_next_to_nothing(g, ctx, act, tiny):
    """A softmax gives such weights to the experts behind a clear first: they add next to nothing."""
    s, rnd, gen = layer(12, 256, 512, 4, 10)
    ids, weights = picks(12, 3, 4, gen)
    weights[:, 1] *= tiny
    weights[6:, 2] = 0
    check_layer(apply(g, ctx, s, ids, weights, act, y=False), s, ids, weights, act, y=False)
    ids, weights = ids[:, 1:].contiguous(), weights[:, 1:].contiguous()
    check_layer(apply(g, ctx, s, ids, weights, act), s, ids, weights, act)


def test_hidden_values_near_the_largest(g, ctx):
    s, rnd, gen = layer(12, 256, 512, 4, 11)
    ids, weights = picks(12, 1, 4, gen)
    for t in range(12):
        e = int(ids[t, 0])
        h = ff.act_reference(s["q"][t:t + 1], s["sx"][t:t + 1], s["w13"][e], s["s13"][e], "silu", True)[0]
        weights[t] = 2e38 / float(h.abs().max())
    s["s2"] = s["s2"] * 1e-30
    check_layer(apply(g, ctx, s, ids, weights, y=False), s, ids, weights, y=False)


def test_the_same_bits_twice(g, ctx):
    for T in (1, 37, 128):
        s, rnd, gen = layer(T, 1024, 512, 16, T)
        ids, weights = picks(T, 5, 16, gen)
        assert torch.equal(apply(g, ctx, s, ids, weights), apply(g, ctx, s, ids, weights))
