"""Seeded random shapes, widths, ranks, plans, strides and modes of the residual and adapter operators,
against the 64-bit formulas of their own test files."""
import importlib.util
import os
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(HERE, name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


res, lora = load("test_gpu_residual"), load("test_gpu_lora")
DRAWS = int(os.environ.get("GEMMAR_FUZZ_DRAWS", "24"))


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def ctx(g):
    torch.cuda.set_device(0)
    c = g.gemmar_create(0, 8192, 7168, 2048, 1, flags=g.GEMMAR_NO_SELF_TEST, wait_timeout_ns=500_000_000)
    yield c
    c.close()


def log_int(rng, lo, hi):
    return min(hi, int(lo * (hi / lo) ** rng.random() + 0.5))


def strided(rng, t):
    """The tensor, or a view of a wider one (a 16-byte multiple from its start, another one's stride)."""
    if t is None or t.dim() != 2 or rng.random() < 0.5:
        return t
    unit = 16 // t.element_size()
    lead, tail = unit * rng.randrange(4), unit * rng.randrange(1, 5)
    wide = torch.full((t.shape[0], lead + t.shape[1] + tail), float("nan"), dtype=t.dtype, device="cuda")
    view = wide[:, lead:lead + t.shape[1]]
    view.copy_(t)
    return view


@pytest.mark.parametrize("seed", range(DRAWS))
def test_residual(g, ctx, seed):
    rng = random.Random(1000 + seed)
    M, N = log_int(rng, 1, 900), 8 * log_int(rng, 1, 2048)
    post, pre = rng.random() < 0.7, rng.random() < 0.8
    d = res.make(M, N, post, pre, rng.choice(["none", "row", "token"]), rng.random() < 0.5, rng.random() < 0.3, seed=seed)
    for k in ("y", "h", "gate", "dt", "du"):
        d[k] = strided(rng, d[k])
    if rng.random() < 0.2:
        d["dt"] = None
    alpha, beta, eps = rng.choice([1.0, 0.5, -0.25]), rng.choice([1.0, 0.125, -2.0]), rng.choice([1e-6, 1e-5])
    o = res.forward(g, ctx, d, alpha, beta, eps, q=pre and N % 128 == 0)
    res.check_forward(d, o, alpha, beta, eps)
    res.check_backward(d, o["rstd"], res.backward(g, ctx, d, o["rstd"], alpha, beta), alpha, beta)
    assert g.gemmar_status(ctx)[0] == 0


@pytest.mark.parametrize("seed", range(DRAWS))
def test_adapters(g, ctx, seed):
    rng = random.Random(2000 + seed)
    T, R, r = log_int(rng, 1, 3000), log_int(rng, 1, 200), log_int(rng, 1, 128)
    K, N = 8 * log_int(rng, 1, 300), 8 * log_int(rng, 1, 300)
    npr = np.random.default_rng(seed)
    if rng.random() < 0.5:
        ids = npr.integers(-1, R, T)
    else:   # runs, most adapters idle
        ids = np.repeat(npr.integers(-1, R, T // 50 + 1), 50)[:T]
    d = lora.make(g, ctx, ids.astype(np.int32), R, r, K, N, seed=seed, ranks=rng.choice(["mixed", None]))
    base, dx0 = rng.choice(["y", "y", None]), rng.choice(["dx0", "dx0", None])
    for k in ("x", "y", "dy"):
        d[k] = strided(rng, d[k])
    out, v = lora.apply(g, ctx, d, y=base)
    lora.check_apply(d, out, v, y=base)
    lora.check_bwd(d, v, *lora.apply_bwd(g, ctx, d, v, dx0=dx0), dx0=dx0)
    assert g.gemmar_status(ctx)[0] == 0
