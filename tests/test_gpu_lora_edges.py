"""lora_apply and lora_apply_bwd on non-finite and extreme values, and what they refuse.  Formulas, inputs and
tolerances are those of the operators' own test file."""
import importlib.util
import os

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
