"""What the operators' binding says to arguments that do not fit, before any of them reaches the library."""
import ctypes

import pytest
import torch

import block_scaled_fp8_gemm_gb300 as g

M, N, T, K, R, R_MAX = 4, 256, 6, 64, 3, 8


class _Handle:
    handle = ctypes.c_void_p(None)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


CALLS = {
    "norm_gate_residual": lambda: dict(y=bf(M, N), h=bf(M, N), w_pre=f32(N), t=bf(M, N), w_post=f32(N), gate=bf(N),
                                       u=bf(M, N), q=torch.zeros(M, N, dtype=torch.uint8), scales=f32(M, N // 128),
                                       rstd=f32(M, 2)),
    "norm_gate_residual_bwd": lambda: dict(y=bf(M, N), h=bf(M, N), rstd=f32(M, 2), dt=bf(M, N), dy=bf(M, N), dh=bf(M, N),
                                           w_post=f32(N), w_pre=f32(N), gate=bf(N), du=bf(M, N), dw_post=f32(N),
                                           dw_pre=f32(N), dgate=f32(N)),
    "lora_apply": lambda: dict(x=bf(T, K), order=i32(T), offsets=i32(R + 1), A=bf(R, R_MAX, K), B=bf(R, R_MAX, N),
                               scales=f32(R), ranks=i32(R), out=bf(T, N), y=bf(T, N), v=f32(T, R_MAX)),
    "lora_apply_bwd": lambda: dict(x=bf(T, K), dy=bf(T, N), order=i32(T), offsets=i32(R + 1), A=bf(R, R_MAX, K),
                                   B=bf(R, R_MAX, N), scales=f32(R), ranks=i32(R), v=f32(T, R_MAX), dx=bf(T, K),
                                   dA=bf(R, R_MAX, K), dB=bf(R, R_MAX, N), dx0=bf(T, K)),
}
ARGS = [(name, arg) for name, make in CALLS.items() for arg in make()]


def call(name, **changed):
    getattr(g, name)(_Handle(), **{**CALLS[name](), **changed}, stream=0)


@pytest.mark.parametrize("name", CALLS)
def test_tensors_on_the_host(name):
    with pytest.raises(ValueError, match="must live on a CUDA device"):
        call(name)


@pytest.mark.parametrize("name,arg", ARGS)
def test_no_tensor(name, arg):
    with pytest.raises((TypeError, ValueError)):
        call(name, **{arg: 3})


@pytest.mark.parametrize("name,arg", ARGS)
def test_complex_tensor(name, arg):
    shape = CALLS[name]()[arg].shape
    with pytest.raises((TypeError, ValueError)):
        call(name, **{arg: torch.zeros(shape, dtype=torch.complex64)})


@pytest.mark.parametrize("name,arg", ARGS)
def test_scalar_tensor(name, arg):
    with pytest.raises((TypeError, ValueError)):
        call(name, **{arg: torch.zeros((), dtype=CALLS[name]()[arg].dtype)})


@pytest.mark.parametrize("name,first", [("norm_gate_residual", "y"), ("norm_gate_residual_bwd", "h"), ("lora_apply", "A"),
                                        ("lora_apply_bwd", "x")])
def test_names_the_argument(name, first):
    with pytest.raises(TypeError, match=f"{first} must be a torch.Tensor"):
        call(name, **{first: None})


@pytest.mark.parametrize("name", ["norm_gate_residual", "norm_gate_residual_bwd"])
@pytest.mark.parametrize("arg", ["alpha", "beta"])
def test_factor_that_is_no_number(name, arg):
    with pytest.raises((TypeError, ValueError)):
        call(name, **{arg: "one"})


def test_destroyed_context():
    ctx = g.Context(None, 0)
    with pytest.raises(ValueError, match="destroyed"):
        g.lora_apply(ctx, **CALLS["lora_apply"](), stream=0)
