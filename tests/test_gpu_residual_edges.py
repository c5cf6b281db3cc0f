"""norm_gate_residual and its backward pass on non-finite values and extreme magnitudes.  Formulas, inputs
and tolerances are those of the operators' own test file."""
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


res = load("test_gpu_residual")


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


@pytest.mark.parametrize("M,N", [(5, 1032), (700, 256), (3, 16384)])
@pytest.mark.parametrize("gate", ["none", "row", "token"])
def test_without_a_pre_norm_no_gradient_depends_on_the_stream(g, ctx, M, N, gate):
    """d = dt then, so h's infinities, NaN and sums that overflow must not reach any gradient."""
    d = res.make(M, N, True, False, gate, True, seed=M)
    o = res.forward(g, ctx, d)
    clean = res.backward(g, ctx, d, o["rstd"])
    res.check_backward(d, o["rstd"], clean, 1.0, 1.0)
    for row, value in ((0, float("inf")), (1, float("nan")), (2, 3e38)):
        d["h"][row, 1::2] = value
    sick = res.backward(g, ctx, d, o["rstd"])
    for k in clean:
        assert torch.equal(sick[k], clean[k]), k


@pytest.mark.parametrize("N", [512, 8200])
@pytest.mark.parametrize("post,gate", [(False, "none"), (True, "row"), (True, "token")])
@pytest.mark.parametrize("size", [1e16, 1e15, 1e13, 1e-12, 1e-14])
def test_gradients_of_rows_of_any_size(g, ctx, N, post, gate, size):
    """The pre norm takes a row's size out, so its gradient's terms stay comparable whatever it is."""
    d = res.make(6, N, post, True, gate, True, y32=True, seed=7)
    beta = size if post else 1.0   # a post norm takes y's size out
    d["h"] *= size
    if not post:
        d["y"] *= size
    d["dt"] /= size                # of du's gradient's size, which goes with 1 / size
    o = res.forward(g, ctx, d, 0.75, beta, 0.0)
    res.check_forward(d, o, 0.75, beta, 0.0)
    b = res.backward(g, ctx, d, o["rstd"], 0.75, beta)
    res.check_backward(d, o["rstd"], b, 0.75, beta)


@pytest.mark.parametrize("M,N", [(3, 1032), (3000, 1032), (3, 4104), (1000, 4104)])
@pytest.mark.parametrize("h32", [False, True])
@pytest.mark.parametrize("which", ["w_post", "gate", "w_pre"])
def test_an_infinite_weight_stays_in_its_column(g, ctx, M, N, h32, which):
    """Of the first column, whose weight is also at hand where a row's last threads have no column: t is infinite
    there alone, its square makes r2 zero, and 0 is what the other columns' x is.  An infinite w_pre makes only
    its own column of x infinite."""
    d = res.make(M, N, which == "w_post", True, "row" if which == "gate" else "none", h32, seed=M)
    d["y"][:, 0] = 1.0
    clean = res.forward(g, ctx, d)
    d[which][0] = float("inf")
    o = res.forward(g, ctx, d)
    assert torch.equal(o["t"][:, 1:], clean["t"][:, 1:]) and torch.equal(o["rstd"][:, 0], clean["rstd"][:, 0])
    if which == "w_pre":
        assert torch.equal(o["rstd"], clean["rstd"]) and torch.equal(o["u"][:, 1:], clean["u"][:, 1:])
        zero = d["h"][:, 0] + d["y"][:, 0] == 0   # 0 * inf
        assert torch.equal(o["u"][:, 0].isnan(), zero) and torch.equal(o["u"][:, 0].isinf(), ~zero)
    else:
        assert o["t"][:, 0].isinf().all() and (o["rstd"][:, 1] == 0).all()
        assert (o["u"][:, 1:] == 0).all() and o["u"][:, 0].isnan().all()
