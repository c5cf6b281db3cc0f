"""What the feed-forward entry points refuse, before anything reaches the GPU (CPU only)."""
import ctypes
import os
import re
import types

import pytest
import torch

import block_scaled_fp8_gemm_gb300 as g

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gemmar.h")
NAMES = ("gemm_blockscale_act", "gemm_blockscale_act_bwd", "moe_route", "moe_apply")
CTX = types.SimpleNamespace(handle=ctypes.c_void_p(None))
M, N, K, T, H, INNER, E, KC = 4, 256, 384, 6, 256, 128, 5, 2


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


f32 = lambda *shape: torch.zeros(shape)

CALLS = {
    "gemm_blockscale_act": lambda: dict(A=u8(M, K), sa=f32(M, K // 128), B=u8(2 * N, K), sb=f32(2 * N // 128, K // 128), C=bf(M, N), gated=True,
                                        bias=f32(2 * N), residual=f32(M, N), q=u8(M, N), scales=f32(M, N // 128), z=bf(M, 2 * N)),
    "gemm_blockscale_act_bwd": lambda: dict(dout=bf(M, N), z=bf(M, N), dz=bf(M, N), dbias=f32(N), q=u8(M, N), scales=f32(M, N // 128)),
    "moe_route": lambda: dict(x=bf(T, H), router=f32(E, H), ids=i32(T, KC), weights=f32(T, KC), bias=f32(E)),
    "moe_apply": lambda: dict(q=u8(T, H), sx=f32(T, H // 128), ids=i32(T, KC), weights=f32(T, KC), w13=u8(E, 2 * INNER, H),
                              s13=f32(E, 2 * INNER // 128, H // 128), w2=u8(E, H, INNER), s2=f32(E, H // 128, INNER // 128), out=bf(T, H),
                              place=i32(9), y=bf(T, H)),
}
ARGS = [(name, arg) for name, make in CALLS.items() for arg, t in make().items() if isinstance(t, torch.Tensor)]


def call(name, **changed):
    getattr(g, name)(CTX, **{**CALLS[name](), **changed}, stream=0)


def test_null_context_is_an_argument_error():
    for name in NAMES:
        args = [a(0) if a is not ctypes.c_void_p else None for a in g._SIGS[name][1]]
        assert getattr(g._lib, name)(*args) == g.GEMMAR_ERR_ARG, name


def test_signatures_have_the_header_s_arguments():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    kinds = {"float": ctypes.c_float, "int64_t": ctypes.c_int64, "int": ctypes.c_int}
    for name in NAMES:
        params = re.search(r"\bint %s\((.*?)\);" % name, text, flags=re.S).group(1).split(",")
        assert g._SIGS[name][1] == [ctypes.c_void_p if "*" in p else kinds[p.split()[0]] for p in params], name


def test_limits_match_the_header():
    for name in ("GEMMAR_MOE_MAX_TOKENS", "GEMMAR_MOE_MAX_EXPERTS", "GEMMAR_MOE_MAX_CHOSEN"):
        assert getattr(g, name) == int(re.search(r"#define %s (\d+)" % name, open(HEADER).read()).group(1))


@pytest.mark.parametrize("name", NAMES)
def test_tensors_on_the_host(name):
    with pytest.raises(ValueError, match="must live on a CUDA device"):
        call(name)


@pytest.mark.parametrize("name,arg", ARGS)
@pytest.mark.parametrize("kind", ["number", "complex", "scalar"])
def test_a_tensor_that_does_not_fit(name, arg, kind):
    t = CALLS[name]()[arg]
    bad = {"number": 3, "complex": torch.zeros(t.shape, dtype=torch.complex64), "scalar": torch.zeros((), dtype=t.dtype)}[kind]
    with pytest.raises((TypeError, ValueError)):
        call(name, **{arg: bad})


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_that_only_the_binding_refuses(name, monkeypatch):
    monkeypatch.setattr(g, "_operators", types.SimpleNamespace(**{name: lambda *a: -1}))
    monkeypatch.setattr(g, "_explain_" + name, lambda *a: None)
    with pytest.raises(ValueError, match=name + ": an argument does not fit"):
        call(name)


@pytest.mark.parametrize("name,arg", [("gemm_blockscale_act", "act"), ("gemm_blockscale_act_bwd", "act"), ("moe_route", "score"), ("moe_apply", "act")])
@pytest.mark.parametrize("bad", ["silu", 1 << 40])
def test_a_choice_that_is_no_number(name, arg, bad):
    with pytest.raises((TypeError, ValueError, OverflowError)):
        call(name, **{arg: bad})


def test_an_odd_number_of_gated_rows():
    with pytest.raises(ValueError, match="even number of rows"):
        call("gemm_blockscale_act", B=u8(2 * N + 1, K))


def test_a_factor_that_is_no_number():
    with pytest.raises((TypeError, ValueError)):
        call("moe_route", factor="one")


def test_destroyed_context():
    for name in NAMES:
        with pytest.raises(ValueError, match="destroyed"):
            getattr(g, name)(g.Context(None, 0), **CALLS[name](), stream=0)
