"""The order of moe_route's experts where the logits' terms cancel: an fp32 sum is then off by its terms' sizes,
far more than the logits' own."""
import pytest
import torch

from test_gpu_moe import check_route, ctx, g, route, route_reference, router   # noqa: F401 (fixtures)

pytestmark = pytest.mark.gpu

FORMS = [(0, False), (1, False), (0, True), (1, True)]   # score, with a bias


def reference(x, w, k, bias=None, score=0):
    """route_reference, whose sigmoids are equal in 64 bits past 36 or so: without a bias the order is the logits'."""
    ids, weights, err = route_reference(x, w, k, bias=bias, score=score)
    if bias is None and score == 1:
        l = x.double() @ w.double().T
        by_logit = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
        p = torch.sigmoid(l)
        assert torch.allclose(p.gather(1, by_logit), p.gather(1, ids.long()), rtol=0, atol=2.0 ** -52)   # the same but for equal ones
        ids = by_logit.int()
    return ids, weights, err


def forms(biased, bias, score):
    return dict(bias=bias if biased else None, score=score)


@pytest.mark.parametrize("T", [1, 5, 8, 9, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("score,biased", FORMS)
def test_two_large_columns_that_cancel(g, ctx, T, dtype, score, biased):
    x, w, bias = router(T, 7168, 64, 30 + T, dtype)
    x[:, 0] = x[:, -1] = 256
    w[:, 0], w[:, -1] = 64, -64
    kw = forms(biased, bias * 0.01, score)
    check_route(route(g, ctx, x, w, 8, **kw), reference(x, w, 8, **kw))


@pytest.mark.parametrize("T", [1, 8, 128])
@pytest.mark.parametrize("offset", [30.0, 100.0, -300.0])
@pytest.mark.parametrize("score,biased", FORMS)
def test_rows_with_a_common_offset(g, ctx, T, offset, score, biased):
    for seed in range(3):
        x, w, bias = router(T, 7168, 256, 50 + seed)
        x = (x.float() + offset).bfloat16()
        w = (w.float() - w.float().mean(1, keepdim=True)).bfloat16()
        kw = forms(biased, bias * 0.01, score)
        check_route(route(g, ctx, x, w, 8, **kw), reference(x, w, 8, **kw))


@pytest.mark.parametrize("T,H,E", [(128, 16384, 1024), (8, 65536, 300), (70, 65536, 640)])
@pytest.mark.parametrize("score,biased", [(0, False), (1, True)])
def test_long_rows_and_many_experts(g, ctx, T, H, E, score, biased):
    x, w, bias = router(T, H, E, H + T)
    kw = forms(biased, bias * 0.01, score)
    check_route(route(g, ctx, x, w, 16, **kw), route_reference(x, w, 16, **kw))


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("scale", [1e-12, 1e-6, 1e6, 1e15])
def test_sizes_far_from_one(g, ctx, T, scale):
    """Rows and router far from 1 in opposite directions and in the same one."""
    x, w, _ = router(T, 1024, 64, 70, torch.float32)
    x, w = (x.float() * scale).bfloat16(), w / scale
    check_route(route(g, ctx, x, w, 8), route_reference(x, w, 8))
    ids, _ = route(g, ctx, x, w * scale, 8, renorm=False)
    l = x.double() @ (w * scale).double().T
    assert torch.equal(ids, torch.sort(l, dim=1, descending=True, stable=True).indices[:, :8].int())


@pytest.mark.parametrize("T", [1, 8, 40])
@pytest.mark.parametrize("biased", [False, True])
def test_saturated_sigmoids_with_a_bias(g, ctx, T, biased):
    """Half the sigmoids are 1 to 64 bits: the bias orders them, or equal ones take the lowest."""
    x, w, bias = router(T, 1024, 64, 80)
    x[:, 0], w[:, 0] = 1, -80
    w[1::2, 0] = 80
    kw = dict(bias=bias if biased else torch.zeros_like(bias), score=1)
    got = route(g, ctx, x, w, 8, **kw)
    check_route(got, route_reference(x, w, 8, **kw))
    if not biased:
        assert got[0][0].tolist() == list(range(1, 17, 2))


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("biased", [False, True])
def test_padded_rows_among_others(g, ctx, T, biased):
    """A row of zeros: every logit is 0, the bias alone or the lowest number decides."""
    x, w, bias = router(T, 1024, 96, 90)
    x[::3] = 0
    kw = dict(bias=bias if biased else None, score=1)
    check_route(route(g, ctx, x, w, 8, **kw), route_reference(x, w, 8, **kw))


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_router_row_that_is_not_finite(g, ctx, T, bad):
    """One expert's logits are infinite or NaN; the others keep their order."""
    x, w, _ = router(T, 1024, 64, 95)
    x[:, 7] = x[:, 7].abs() + 1
    w[11, 7] = bad
    ids, _ = route(g, ctx, x, w, 8)
    l = x.double() @ w.double().T
    l[:, 11] = bad if bad == bad else -float("inf")
    assert torch.equal(ids, torch.sort(l, dim=1, descending=True, stable=True).indices[:, :8].int())
