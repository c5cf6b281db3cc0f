"""Slopes and values in the backward pass, relative to their own size: in both tails, where they vanish, too."""
import math

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
    c = g.gemmar_create(0, 1024, 2048, 256, 1, flags=g.GEMMAR_NO_SELF_TEST)
    yield c
    assert g.gemmar_status(c)[0] == 0
    c.close()


def slope(act, z):
    """act'(z) in fp64, and the sizes of its two terms: the factor, and z times the factor's slope."""
    if act == "silu":
        s, d = torch.sigmoid(z), torch.sigmoid(z) * torch.sigmoid(-z)
    elif act == "gelu":
        s, d = 0.5 * torch.erfc(-z / math.sqrt(2)), torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        u = c * (z + 0.044715 * z ** 3)
        s, d = torch.sigmoid(u), torch.sigmoid(u) * torch.sigmoid(-u) * c * (1 + 3 * 0.044715 * z ** 2)
    else:
        s = torch.ones_like(z) if act == "none" else (z > 0).double()
        d = torch.zeros_like(z)
    return s + z * d, s + (z * d).abs()


def roundings(act, z):
    """Roundings of 2^-23 in the factor and in its slope: a dozen for the operations, and those of the exponential's argument
    relative to its size: |z|, z^2 / 2, or 1.6 |z| + 0.0714 |z|^3 with the three of its own products."""
    a = z.abs()
    return 12 + {"silu": 2 * a, "gelu": 2 * a ** 2, "gelu_tanh": 6 * a + 0.25 * a ** 3}.get(act, 0 * a)


VANISHED = 2.0 ** -116   # below 2^-126 a factor is 0: times |z| (1 + slope of the exponent), at most 1000 here


def close(got, ref, size, act, z, what):
    # past 2^-1 of its size the bound of a first-order error says nothing: there the factor has vanished
    err = (roundings(act, z) * 2.0 ** -23).clamp(max=0.5) * size + VANISHED
    ff.within(got, ref, err + ff.BF16 * (ref.abs() + err), what)


@pytest.mark.parametrize("act", ff.ACTS)
@pytest.mark.parametrize("far", [1.0, 3.0, 12.0, 100.0])
def test_both_tails(g, ctx, act, far):
    M, N = 16, 512
    z = torch.linspace(-far, far, M * N, device="cuda").view(M, N).bfloat16()
    dout = torch.full((M, N), -3.0, device="cuda")
    zd = z.double()
    want, size = slope(act, zd)
    dz = torch.empty_like(z)
    g.gemm_blockscale_act_bwd(ctx, dout, z, dz, act=ff.ACTS.index(act))
    close(dz, -3 * want, 3 * size, act, zd, "slope")
    both = torch.cat([z, torch.ones_like(z)], 1)
    dz = torch.empty_like(both)
    g.gemm_blockscale_act_bwd(ctx, dout, both, dz, act=ff.ACTS.index(act), gated=True)
    torch.cuda.synchronize()
    close(dz[:, :N], -3 * want, 3 * size, act, zd, "slope of the gate")
    value = ff.value(act, zd)
    close(dz[:, N:], -3 * value, 3 * value.abs(), act, zd, "value")
