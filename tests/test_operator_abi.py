"""The residual and adapter entry points refuse a null context before they touch the GPU, and the
library's limits are the header's (CPU only)."""
import ctypes
import os
import re

import block_scaled_fp8_gemm_gb300 as g

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "gemmar.h")
NAMES = ("norm_gate_residual", "norm_gate_residual_bwd", "lora_plan", "lora_apply", "lora_apply_bwd")


def test_null_context_is_an_argument_error():
    for name in NAMES:
        args = [a(0) if a is not ctypes.c_void_p else None for a in g._SIGS[name][1]]
        assert getattr(g._lib, name)(*args) == g.GEMMAR_ERR_ARG, name


def test_signatures_have_the_header_s_arguments():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    kinds = {"float": ctypes.c_float, "int64_t": ctypes.c_int64, "int": ctypes.c_int}
    for name in NAMES:
        params = re.search(r"\bint %s\((.*?)\);" % name, text, flags=re.S).group(1).split(",")
        want = [ctypes.c_void_p if "*" in p else kinds[p.split()[0]] for p in params]
        assert g._SIGS[name][1] == want, name


def test_limits_match_the_header():
    for name in ("GEMMAR_NORM_MAX_N", "GEMMAR_LORA_MAX_ADAPTERS", "GEMMAR_LORA_MAX_RANK"):
        value = re.search(r"#define %s (\d+)" % name, open(HEADER).read()).group(1)
        assert getattr(g, name) == int(value)
