"""Refusals of the operators' Python entry points: each has a reason and the argument's name (CPU only)."""
import ctypes
import types

import pytest
import torch

import block_scaled_fp8_gemm_gb300 as g

CTX = types.SimpleNamespace(handle=ctypes.c_void_p(None))
ARGS = {"norm_gate_residual": 4, "norm_gate_residual_bwd": 6, "lora_apply": 8, "lora_apply_bwd": 12}


@pytest.mark.parametrize("name", ARGS)
def test_a_tensor_that_only_the_binding_refuses(name, monkeypatch):
    """Should the two sets of checks drift apart, the caller still reads an error and not a status of -1."""
    monkeypatch.setattr(g, "_operators", types.SimpleNamespace(**{name: lambda *a: -1}))
    monkeypatch.setattr(g, "_explain_" + name, lambda *a: None)
    with pytest.raises(ValueError, match=name + ": an argument does not fit"):
        getattr(g, name)(CTX, *[None] * ARGS[name], stream=0)


def test_codes_that_are_no_tensor():
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        g._codes(3, (4, 128), "q")


@pytest.mark.parametrize("ids,offsets,error,text", [(None, torch.zeros(3), TypeError, "adapter_ids must be a torch.Tensor"),
                                                    (torch.zeros(4), 3, TypeError, "offsets must be a torch.Tensor"),
                                                    (torch.zeros(2, 2), torch.zeros(3), ValueError, "adapter_ids must have 1 dimensions")])
def test_a_plan_of_no_tensors(ids, offsets, error, text):
    with pytest.raises(error, match=text):
        g.lora_plan(CTX, ids, torch.zeros(4, dtype=torch.int32), offsets, stream=0)


@pytest.mark.parametrize("name", ["norm_gate_residual", "norm_gate_residual_bwd"])
@pytest.mark.parametrize("arg", ["y", "h"])
def test_a_type_that_is_neither_bf16_nor_fp32(name, arg):
    kinds = {"y": torch.bfloat16, "h": torch.bfloat16, arg: torch.float16}
    y, h = (torch.zeros(4, 256, dtype=kinds[k]) for k in "yh")
    with pytest.raises(TypeError, match=f"{arg} must be bfloat16 or float32"):
        getattr(g, name)(CTX, y, h, *[None] * (ARGS[name] - 2), stream=0)
