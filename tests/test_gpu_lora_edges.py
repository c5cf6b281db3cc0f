"""lora_apply and lora_apply_bwd on non-finite and extreme values, and what they refuse.  Formulas, inputs and
tolerances are those of the operators' own test file."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(os.path.dirname(os.path.abspath(__file__)), name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


lora = load("test_gpu_lora")


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


@pytest.mark.parametrize("T,r", [(24, 16), (900, 32), (700, 100)])
def test_columns_of_v_past_a_rank_are_zero_for_any_token(g, ctx, T, r):
    """Also for tokens with NaN or infinities, whose products with absent rows would be NaN."""
    d = lora.make(g, ctx, lora.mixed_ids(T, 4, 6), 4, r, 256, 384, seed=6)
    d["x"][::3, 5] = float("nan")
    d["x"][1::3, 7] = float("inf")
    _, v = lora.apply(g, ctx, d)
    at = d["offsets"].tolist()
    for a in range(4):
        k = int(d["ranks"][a])
        assert (v[at[a]:at[a + 1], k:] == 0).all(), a
        assert k == 0 or not torch.isfinite(v[at[a]:at[a + 1], :k]).all()


@pytest.mark.parametrize("T,r", [(24, 16), (900, 32), (700, 100)])
def test_an_infinite_scale_reaches_the_ranks_alone(g, ctx, T, r):
    """w is infinite at an adapter's ranks; past them, where zeros stand for its rows, it must not be 0 * inf."""
    d = lora.make(g, ctx, lora.mixed_ids(T, 4, 6), 4, r, 256, 384, seed=6)
    for k in ("A", "B", "dy"):
        d[k] = d[k].abs() + 0.01
    d["scales"][1:3] = float("inf")
    dx, _, _ = lora.apply_bwd(g, ctx, d, torch.zeros(T, r, device="cuda"))
    sick = (d["ids"] == 1) | (d["ids"] == 2)
    assert torch.isfinite(dx[~sick].float()).all() and (dx[sick] == float("inf")).all()


def alike(got, ref):
    """Infinities and NaN at the same places, the infinities of the same sign."""
    got, bad = got.double(), ~torch.isfinite(ref)
    return torch.equal(~torch.isfinite(got), bad) and torch.equal(got[bad].nan_to_num(0.0), ref[bad].nan_to_num(0.0))


@pytest.mark.parametrize("T,r", [(24, 16), (900, 32), (700, 128)])
def test_infinite_sums_stay_infinite(g, ctx, T, r):
    """An infinity of x makes v infinite, and out = y + s v B is infinite of v B's sign (factors of one sign, so no
    sum has infinities of both); one of dy does the same to w, dx and dA."""
    d = lora.make(g, ctx, lora.mixed_ids(T, 4, 6), 4, r, 256, 384, seed=6, ranks=None)
    d["A"], d["B"] = d["A"].abs() + 0.01, d["B"].abs() + 0.01
    d["x"][::5, 7] = float("inf")
    d["x"][1::5, 9] = -float("inf")
    d["dy"][:, 11] = d["dy"][:, 11].abs()
    out, v = lora.apply(g, ctx, d)
    at = d["offsets"].tolist()
    ref = d["y"].double()
    for a in range(4):
        rows = d["order"][at[a]:at[a + 1]].long()
        vr = d["x"][rows].double() @ d["A"][a].double().T
        assert alike(v[at[a]:at[a + 1]], vr)
        ref[rows] += float(d["scales"][a]) * vr @ d["B"][a].double()
    assert alike(out, ref) and ref.isinf().any() and not ref.isnan().any()
    d = lora.make(g, ctx, lora.mixed_ids(T, 4, 6), 4, r, 256, 384, seed=6, ranks=None)
    d["A"], d["B"], d["x"] = d["A"].abs() + 0.01, d["B"].abs() + 0.01, d["x"].abs() + 0.01
    _, v = lora.apply(g, ctx, d)
    d["dy"][::5, 7] = float("inf")
    dx, dA, _ = lora.apply_bwd(g, ctx, d, v)
    ref = d["dx0"].double()
    for a in range(4):
        rows = d["order"][at[a]:at[a + 1]].long()
        w = float(d["scales"][a]) * d["dy"][rows].double() @ d["B"][a].double().T
        ref[rows] += w @ d["A"][a].double()
        assert alike(dA[a], w.T @ d["x"][rows].double())
    assert alike(dx, ref) and ref.isinf().any() and not ref.isnan().any()


@pytest.mark.parametrize("T,r", [(24, 16), (900, 32)])
def test_v_above_the_largest_bf16(g, ctx, T, r):
    """v = 0x7F7F (the largest bf16) + 2^119 is finite in fp32 and rounds to infinity in bf16."""
    d = lora.make(g, ctx, np.zeros(T, np.int32), 1, r, 64, 128, seed=2, ranks=None)
    big = torch.tensor(0x7F7F, dtype=torch.int16).view(torch.bfloat16).item()
    d["A"].zero_()
    d["A"][0, :, :2] = 1.0
    d["x"].zero_()
    d["x"][:, 0], d["x"][:, 1] = big, 2.0 ** 119
    d["B"] *= 2.0 ** -12
    out, v = lora.apply(g, ctx, d)
    lora.check_apply(d, out, v)


@pytest.mark.parametrize("T,r,K,N", [(2000, 16, 2048, 512), (3000, 64, 512, 2048), (900, 128, 256, 7168)])
def test_dx_reads_the_v_of_its_own_call(g, ctx, T, r, K, N):
    """Two batches in turn through one context's scratch, nothing between the calls: dx, whose launch overlaps the
    end of the weight gradients', must not see the other batch's w."""
    batches = [lora.make(g, ctx, lora.mixed_ids(T, 5, s), 5, r, K, N, seed=s) for s in (1, 2)]
    kept = [lora.apply(g, ctx, d)[1] for d in batches]
    want = []
    for d, v in zip(batches, kept):
        want.append(lora.apply_bwd(g, ctx, d, v))
        lora.check_bwd(d, v, *want[-1])
    for _ in range(20):
        got = [lora.apply_bwd(g, ctx, d, v) for d, v in zip(batches, kept)]
        assert all(torch.equal(a, b) for x, y in zip(got, want) for a, b in zip(x, y))
    assert g.gemmar_status(ctx)[0] == 0


def test_gradients_over_their_inputs_are_refused(g, ctx):
    """dx is written while x and dy are read, dA and dB while A and B are."""
    d = lora.make(g, ctx, [0, 1, -1, 0], 2, 8, 128, 128, seed=1, ranks=None)
    d["A"], d["B"] = d["A"].contiguous(), d["B"].contiguous()
    _, v = lora.apply(g, ctx, d)

    def code(**kw):
        a = dict(dx=torch.empty_like(d["x"]), dA=torch.empty_like(d["A"]), dB=torch.empty_like(d["B"]), dx0=d["dx0"])
        a.update(kw)
        before = {k: d[k].clone() for k in ("x", "dy", "A", "B")}
        with pytest.raises(g.GemmarError) as e:
            g.lora_apply_bwd(ctx, d["x"], d["dy"], d["order"], d["offsets"], d["A"], d["B"], d["scales"], d["ranks"], v, **a)
        assert all(torch.equal(d[k], before[k]) for k in before)
        return e.value.code
    flat = torch.zeros(3 * 2 * 8 * 128, dtype=torch.bfloat16, device="cuda")
    for kw in ({"dx": d["x"]}, {"dx": d["dy"]}, {"dA": d["A"]}, {"dB": d["B"]}, {"dA": d["B"]}, {"dB": d["A"]},
               {"dA": flat[:2048].view(2, 8, 128), "dB": flat[1024:3072].view(2, 8, 128)}):
        assert code(**kw) == g.GEMMAR_ERR_ARG, list(kw)
    assert g.gemmar_status(ctx)[0] == 0


def test_gradients_between_the_columns_of_their_inputs(g, ctx):
    """x and dx as columns of one matrix share no element: not refused, and right."""
    T, K, N = 300, 128, 256
    d = lora.make(g, ctx, lora.mixed_ids(T, 3, 2), 3, 16, K, N, seed=4)
    _, v = lora.apply(g, ctx, d)
    want = lora.apply_bwd(g, ctx, d, v)
    both = torch.cat([d["x"], torch.full_like(d["x"], 7.0)], 1)
    dx, dA, dB = both[:, K:], torch.empty_like(d["A"]), torch.empty_like(d["B"])
    g.lora_apply_bwd(ctx, both[:, :K], d["dy"], d["order"], d["offsets"], d["A"], d["B"], d["scales"], d["ranks"], v, dx, dA, dB, dx0=d["dx0"])
    assert torch.equal(both[:, :K], d["x"]) and all(torch.equal(a, b) for a, b in zip((dx, dA, dB), want))
    with pytest.raises(g.GemmarError) as e:
        g.lora_apply_bwd(ctx, both[:, :K], d["dy"], d["order"], d["offsets"], d["A"], d["B"], d["scales"], d["ranks"], v,
                         both[:, K - 8:-8], dA, dB, dx0=d["dx0"])
    assert e.value.code == g.GEMMAR_ERR_ARG


@pytest.mark.parametrize("N,r,T", [(128, 128, 1024), (128, 65, 1024), (256, 128, 777), (128, 128, 1)])
def test_a_context_of_the_layer_s_rows_is_large_enough(g, N, r, T):
    c = g.gemmar_create(0, T, N, 128, 1, flags=g.GEMMAR_NO_SELF_TEST)
    try:
        d = lora.make(g, c, lora.mixed_ids(T, 3, 5), 3, r, 512, N, seed=3)
        out, v = lora.apply(g, c, d)
        lora.check_apply(d, out, v)
        lora.check_bwd(d, v, *lora.apply_bwd(g, c, d, v))
        assert g.gemmar_status(c)[0] == 0
    finally:
        c.close()


def test_few_tokens_an_adapter_need_no_scratch(g, ctx):
    """The forward pass in one launch: any context serves it."""
    d = lora.make(g, ctx, lora.mixed_ids(3000, 64, 5), 64, 16, 128, 256, seed=3)
    c = g.gemmar_create(0, 1, 128, 128, 1, flags=g.GEMMAR_NO_SELF_TEST)
    try:
        out, v = lora.apply(g, c, d)
        lora.check_apply(d, out, v)
    finally:
        c.close()


def few_of_many(T, R, active, seed):
    """Tokens of a few adapters, far apart among many resident ones, in runs."""
    rng = np.random.default_rng(seed)
    which = rng.choice(R, active, replace=False)
    ids = np.repeat(which[rng.integers(0, active, T // 50 + 1)], 50)[:T]
    ids[rng.random(T) < 0.05] = -1
    return ids.astype(np.int32)


@pytest.mark.parametrize("T,R,active,r", [(1, 1024, 1, 16), (40, 1024, 3, 64), (2048, 1024, 4, 16), (3000, 1024, 4, 64), (4096, 256, 1, 33),
                                          (4097, 1024, 4, 64), (6000, 1000, 2, 128)])
def test_few_active_adapters_of_many(g, ctx, T, R, active, r):
    d = lora.make(g, ctx, few_of_many(T, R, active, T), R, r, 256, 384, seed=T, ranks=None)
    out, v = lora.apply(g, ctx, d)
    lora.check_apply(d, out, v)
    lora.check_bwd(d, v, *lora.apply_bwd(g, ctx, d, v))
    assert g.gemmar_status(ctx)[0] == 0


@pytest.mark.parametrize("T,R,r,K,N", [(8191, 9, 64, 2048, 1032), (16384, 3, 16, 512, 776), (5000, 2, 128, 1024, 512)])
def test_many_tokens(g, ctx, T, R, r, K, N):
    """Adapters cut into several tiles each, of which the parts are joined, and tiles in several waves."""
    d = lora.make(g, ctx, lora.mixed_ids(T, R, T), R, r, K, N, seed=T)
    out, v = lora.apply(g, ctx, d)
    lora.check_apply(d, out, v)
    lora.check_bwd(d, v, *lora.apply_bwd(g, ctx, d, v))
    assert g.gemmar_status(ctx)[0] == 0
