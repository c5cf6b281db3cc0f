"""norm_gate_residual and its backward pass at sizes that give a CTA many rows: weights staged in shared memory, row
slots filled again, the gradients' sums over several rows and many parts.  Formulas, inputs and tolerances are those of
the operators' own test file; its bound on the sums over rows (160 additions in a chain) covers 131100 rows of 64
columns: 54 rows a CTA, 19 parts a group and the groups' tree."""
import importlib.util
import os
import random

import pytest
import torch

pytestmark = pytest.mark.gpu


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(os.path.dirname(os.path.abspath(__file__)), name + ".py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


res = load("test_gpu_residual")
DRAWS = int(os.environ.get("GEMMAR_FUZZ_DRAWS", "24"))


@pytest.fixture(scope="module")
def g():
    import block_scaled_fp8_gemm_gb300 as g
    return g


@pytest.fixture(scope="module")
def ctx(g):
    torch.cuda.set_device(0)
    c = g.gemmar_create(0, 4096, 16384, 128, 1, flags=g.GEMMAR_NO_SELF_TEST, wait_timeout_ns=500_000_000)
    yield c
    c.close()


def check(g, ctx, d, alpha, beta, eps=1e-5):
    M, N = d["y"].shape
    o = res.forward(g, ctx, d, alpha, beta, eps, q=d["w_pre"] is not None and N % 128 == 0)
    res.check_forward(d, o, alpha, beta, eps)
    if "q" in o:   # codes alone, as a serving step asks for them
        only = res.forward(g, ctx, d, alpha, beta, eps, u=False, q=True)
        assert all(torch.equal(only[k], o[k]) for k in only)
    b = res.backward(g, ctx, d, o["rstd"], alpha, beta)
    res.check_backward(d, o["rstd"], b, alpha, beta)
    assert g.gemmar_status(ctx)[0] == 0


@pytest.mark.parametrize("M,N", [(1531, 2056), (2000, 7168), (1300, 8200), (700, 16384), (16000, 264), (3001, 4096), (2500, 1024)])
@pytest.mark.parametrize("post,pre,gate,h32,y32", [(True, True, "row", False, False), (False, True, "none", True, False),
                                                   (True, True, "token", True, True), (True, False, "none", False, False),
                                                   (False, True, "token", False, False), (True, True, "none", True, False),
                                                   (False, False, "row", False, True)])
def test_many_rows_a_cta(g, ctx, M, N, post, pre, gate, h32, y32):
    check(g, ctx, res.make(M, N, post, pre, gate, h32, y32, seed=M + N), 0.75, 1.5)


@pytest.mark.parametrize("gate", ["row", "token"])
def test_very_many_narrow_rows(g, ctx, gate):
    check(g, ctx, res.make(131100, 64, True, True, gate, False, seed=2), 1.0, 1.0)


@pytest.mark.parametrize("seed", range(DRAWS))
def test_drawn_rows(g, ctx, seed):
    rng = random.Random(3000 + seed)
    N = 8 * round(2 ** rng.uniform(0, 11))
    M = min(round(2 ** rng.uniform(8, 13)), max(1, (1 << 24) // N))
    if rng.random() < 0.5:
        N = max(128, N // 128 * 128)
    d = res.make(M, N, rng.random() < 0.7, rng.random() < 0.8, rng.choice(["none", "row", "token"]), rng.random() < 0.5, rng.random() < 0.3, seed=seed)
    check(g, ctx, d, rng.choice([1.0, 0.5, -0.25]), rng.choice([1.0, 0.125, -2.0]))
