"""block_scaled_fp8_gemm_gb300 -- Python binding of libgemmar (include/gemmar.h).

The wo_b path of a DeepSeek-style attention block on one GB300: block-scaled
e4m3 GEMMs per K-slice (tcgen05 MMA, TMEM accumulators, TMA-fed shared
stages), the fixed-order fp32 band reduce to bf16, the per-row e4m3 "fp8 wire"
codec, and the mxfp8 variant on the native block-scaled MMA.

Every function here has the name of the C entry point it calls and only
marshals arguments: torch tensors supply device memory, torch streams supply
the CUDA stream, and all arithmetic runs in the library's CUDA kernels.  The
library is required: importing this package raises if ``libgemmar.so`` has not
been built (``python -c "import __graft_entry__ as g; g.build()"``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgemmar.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"libgemmar.so not found at {LIB_PATH}; build it first with "
        "block_scaled_fp8_gemm_gb300.build.build() (there is no fallback path)")

_lib = ctypes.CDLL(LIB_PATH)


class _NoBinding:
    """Stands for the operators' binding where it cannot be used: the GEMMs and codecs work without it, its own
    entry points say why not."""

    def __init__(self, why: str):
        self._why = why

    def __getattr__(self, name: str):
        raise ImportError(f"{name}: {self._why}; build it with block_scaled_fp8_gemm_gb300.build.build() (there is no fallback path)")


def _binding():
    path = os.path.join(_HERE, "_operators.so")
    if not os.path.exists(path):
        return _NoBinding(f"_operators.so not found at {path}")
    try:
        from . import _operators   # needs torch loaded
    except ImportError as e:
        return _NoBinding(f"{path} does not load ({e})")
    # it reads tensors through torch's own layout of them
    built = getattr(_operators, "torch_version", "of another version")
    if built != str(torch.__version__):
        return _NoBinding(f"{path} was built against torch {built}, this is {torch.__version__}")
    return _operators


_operators = _binding()

# ---- constants (mirror include/gemmar.h) -------------------------------------
GEMMAR_OK = 0
GEMMAR_ERR_ARG = 1
GEMMAR_ERR_SHAPE = 2
GEMMAR_ERR_ALIGN = 3
GEMMAR_ERR_WORKSPACE = 4
GEMMAR_ERR_CUDA = 5
GEMMAR_ERR_TIMEOUT = 6
GEMMAR_ERR_DISABLED = 7
GEMMAR_ERR_DEVICE = 8
STATUS_NAMES = {0: "OK", 1: "ERR_ARG", 2: "ERR_SHAPE", 3: "ERR_ALIGN", 4: "ERR_WORKSPACE",
                5: "ERR_CUDA", 6: "ERR_TIMEOUT", 7: "ERR_DISABLED", 8: "ERR_DEVICE"}

GEMMAR_DTYPE_F32 = 0
GEMMAR_DTYPE_BF16 = 1
GEMMAR_SCALE_BLOCK128 = 0
GEMMAR_SCALE_MX32 = 1
GEMMAR_SCALE_PTPC = 2
GEMMAR_FP8_WIRE = 1 << 0
GEMMAR_DEBUG_CANARY = 1 << 1
GEMMAR_FAULT_SKIP_BAND = 1 << 2
GEMMAR_NO_SELF_TEST = 1 << 3
GEMMAR_FUSE_SLICES = 1 << 4
GEMMAR_CTA_PAIR = 1 << 5
GEMMAR_FUSE_ONCHIP = 1 << 6
GEMMAR_SERIAL_REDUCE = 1 << 7
GEMMAR_FUSE_QUANTIZE = 1 << 8
GEMMAR_MAX_P = 8
GEMMAR_NOALLOC_MAX_PARTIALS = 8 * 1024 * 1024
GEMMAR_NORM_MAX_N = 16384
GEMMAR_LORA_MAX_ADAPTERS = 1024
GEMMAR_LORA_MAX_RANK = 128
GEMMAR_ACT_NONE = 0
GEMMAR_ACT_RELU = 1
GEMMAR_ACT_SILU = 2
GEMMAR_ACT_GELU = 3
GEMMAR_ACT_GELU_TANH = 4
GEMMAR_SCORE_SOFTMAX = 0
GEMMAR_SCORE_SIGMOID = 1
GEMMAR_MOE_MAX_TOKENS = 128
GEMMAR_MOE_MAX_EXPERTS = 1024
GEMMAR_MOE_MAX_CHOSEN = 16

# ---- signatures ----------------------------------------------------------------
_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_U32 = ctypes.c_uint32
_F = ctypes.c_float
_PP = ctypes.POINTER(ctypes.c_void_p)

_SIGS = {
    "gemmar_supports": (_I, [_I, _I64, _I64, _I64, _I, _I]),
    "gemmar_create": (_I, [ctypes.POINTER(_P), _I, _I64, _I64, _I64, _I, _U32, _I64]),
    "gemmar_destroy": (_I, [_P]),
    "gemmar_status": (_I, [_P, ctypes.POINTER(_I)]),
    "gemmar_workspace_bytes": (_I64, [_P]),
    "gemmar_set_phase_timing": (_I, [_P, _I]),
    "gemmar_phase_times": (_I, [_P, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(_I)]),
    "gemmar_overlap_stats": (_I, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "gemm_blockscale_fp8": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P]),
    "gemm_mxfp8": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P]),
    "gemm_ptpc_fp8": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _I64, _P]),
    "band_reduce": (_I, [_P, _P, _I, _I64, _I64, _I, _P, _P]),
    "rowquant_e4m3": (_I, [_P, _P, _I, _I64, _I64, _P, _P, _P]),
    "rowdequant_e4m3": (_I, [_P, _P, _P, _I64, _I64, _P, _P]),
    "quant_blockscale_e4m3": (_I, [_P, _P, _I, _I64, _I64, _I, _P, _P, _P]),
    "quant_mx_e4m3": (_I, [_P, _P, _I, _I64, _I64, _P, _P, _P]),
    "fused_gemm_reduce": (_I, [_P, _I, _PP, _PP, _PP, _PP, _I, _I64, _I64, _I64, _I, _U32, _P, _P]),
    "fused_gemm_reduce_noalloc": (_I, [_I, _PP, _PP, _PP, _PP, _I64, _I64, _I64, _I, _P, _P]),
    "fused_gemm_reduce_noalloc_status": (_I, [ctypes.POINTER(_I)]),
    "norm_gate_residual": (_I, [_P, _P, _I, _I64, _P, _I, _I64, _P, _P, _P, _I64, _F, _F, _F, _I64, _I64,
                                _P, _P, _P, _P, _P, _P]),
    "norm_gate_residual_bwd": (_I, [_P, _P, _I, _I64, _P, _I, _I64, _P, _P, _P, _P, _I64, _F, _F, _I64, _I64,
                                    _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P]),
    "lora_plan": (_I, [_P, _P, _I64, _I, _P, _P, _P]),
    "lora_apply": (_I, [_P, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P, _I64, _P, _I64, _P, _P]),
    "lora_apply_bwd": (_I, [_P, _P, _I64, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I,
                            _P, _I64, _P, _I64, _P, _P, _P]),
    "gemm_blockscale_act": (_I, [_P, _P, _P, _P, _P, _I, _I, _P, _P, _I, _I64, _I64, _I64, _I64, _P, _I, _I64, _P, _P, _P, _P]),
    "gemm_blockscale_act_bwd": (_I, [_P, _P, _I, _I64, _P, _I, _I, _I64, _I64, _P, _P, _P, _P, _P]),
    "moe_route": (_I, [_P, _P, _I64, _P, _I, _P, _I64, _I64, _I, _I, _I, _I, _F, _P, _P, _P]),
    "moe_apply": (_I, [_P, _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _I, _I64, _I64, _I64, _I, _I, _P, _I64, _P, _I64, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)

if not isinstance(_operators, _NoBinding):
    _operators.bind(*(ctypes.cast(getattr(_lib, n), _P).value for n in
                      ("norm_gate_residual", "norm_gate_residual_bwd", "lora_apply", "lora_apply_bwd", "gemm_blockscale_act",
                       "gemm_blockscale_act_bwd", "moe_route", "moe_apply")))


class GemmarError(RuntimeError):
    def __init__(self, code: int, where: str, detail: int = 0):
        self.code = code
        self.detail = detail
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} (code {code}, detail {detail})")


def _check(code: int, where: str):
    if code != GEMMAR_OK:
        raise GemmarError(code, where)


def _ptr(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _u8(t: torch.Tensor, name: str) -> int:
    if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
        raise TypeError(f"{name} must be uint8 codes (or float8_e4m3fn), got {t.dtype}")
    return _ptr(t, name)


def _f32(t: torch.Tensor, name: str) -> int:
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    return _ptr(t, name)


def _bf16(t: torch.Tensor, name: str) -> int:
    if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    return _ptr(t, name)


def _stream(stream) -> int:
    if stream is None:
        # the raw handle: building a torch.cuda.Stream for it takes 3 us a call
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


class Context:
    """Owns one gemmar_ctx (its workspace and status word)."""

    def __init__(self, handle: int, device: int):
        self._h = ctypes.c_void_p(handle)
        self.device = device

    @property
    def handle(self) -> ctypes.c_void_p:
        if self._h.value is None:
            raise ValueError("context already destroyed")
        return self._h

    def close(self):
        if self._h:
            with torch.cuda.device(self.device):
                gemmar_destroy(self)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---- entry points ------------------------------------------------------------------

def gemmar_supports(P: int, M: int, N: int, K: int, bands: int = 0,
                    scale_kind: int = GEMMAR_SCALE_BLOCK128) -> int:
    return int(_lib.gemmar_supports(P, M, N, K, bands if bands else P, scale_kind))


def gemmar_create(device: int, max_M: int, N: int, K: int, max_P: int, flags: int = 0,
                  wait_timeout_ns: int = 0) -> Context:
    h = ctypes.c_void_p()
    with torch.cuda.device(device):
        _check(_lib.gemmar_create(ctypes.byref(h), device, max_M, N, K, max_P, flags, wait_timeout_ns),
               "gemmar_create")
    return Context(h.value, device)


def gemmar_destroy(ctx: Context) -> None:
    h = ctx._h
    ctx._h = ctypes.c_void_p()
    if h:
        _check(_lib.gemmar_destroy(h), "gemmar_destroy")


def gemmar_status(ctx: Context):
    """(code, detail) of the device status word; call after the work completed."""
    d = ctypes.c_int(0)
    code = int(_lib.gemmar_status(ctx.handle, ctypes.byref(d)))
    return code, int(d.value)


def gemmar_workspace_bytes(ctx: Context) -> int:
    return int(_lib.gemmar_workspace_bytes(ctx.handle))


GEMMAR_NUM_PHASES = 4
PHASE_NAMES = ("gemm", "reduce", "quantize", "dequantize")


def gemmar_set_phase_timing(ctx: Context, enable: bool = True) -> None:
    _check(_lib.gemmar_set_phase_timing(ctx.handle, 1 if enable else 0), "gemmar_set_phase_timing")


def gemmar_phase_times(ctx: Context):
    """(dict phase -> summed ms, number of recorded calls); clears the record."""
    ms = (ctypes.c_float * GEMMAR_NUM_PHASES)()
    calls = ctypes.c_int(0)
    _check(_lib.gemmar_phase_times(ctx.handle, ms, ctypes.byref(calls)), "gemmar_phase_times")
    return {PHASE_NAMES[i]: float(ms[i]) for i in range(GEMMAR_NUM_PHASES)}, int(calls.value)


def gemmar_overlap_stats(ctx: Context):
    """(blocks summed by the GEMM kernel while it ran, all 32 x 32 output blocks)
    of the last fused band-path call; call after its work completed."""
    ov = ctypes.c_int64(0)
    tot = ctypes.c_int64(0)
    _check(_lib.gemmar_overlap_stats(ctx.handle, ctypes.byref(ov), ctypes.byref(tot)), "gemmar_overlap_stats")
    return int(ov.value), int(tot.value)


def _cdtype(C: torch.Tensor) -> int:
    if C.dtype == torch.float32:
        return GEMMAR_DTYPE_F32
    if C.dtype == torch.bfloat16:
        return GEMMAR_DTYPE_BF16
    raise TypeError(f"C must be float32 or bfloat16, got {C.dtype}")


def gemm_blockscale_fp8(ctx: Context, A, sa, B, sb, C, stream=None) -> None:
    M, K = A.shape
    N = B.shape[0]
    _check(_lib.gemm_blockscale_fp8(ctx.handle, _u8(A, "A"), _f32(sa, "sa"), _u8(B, "B"), _f32(sb, "sb"),
                                    _ptr(C, "C"), _cdtype(C), M, N, K, _stream(stream)),
           "gemm_blockscale_fp8")


def gemm_ptpc_fp8(ctx: Context, A, sa, B, sb, C, stream=None) -> None:
    """C = (sa[m]*sb[n]) * A @ B^T with per-token sa [M] and per-channel sb [N] (fp32)."""
    M, K = A.shape
    N = B.shape[0]
    _check(_lib.gemm_ptpc_fp8(ctx.handle, _u8(A, "A"), _f32(sa, "sa"), _u8(B, "B"), _f32(sb, "sb"),
                              _ptr(C, "C"), _cdtype(C), M, N, K, _stream(stream)),
           "gemm_ptpc_fp8")


def gemm_mxfp8(ctx: Context, A, ea, B, eb, C, stream=None) -> None:
    M, K = A.shape
    N = B.shape[0]
    _check(_lib.gemm_mxfp8(ctx.handle, _u8(A, "A"), _u8(ea, "ea"), _u8(B, "B"), _u8(eb, "eb"),
                           _ptr(C, "C"), _cdtype(C), M, N, K, _stream(stream)),
           "gemm_mxfp8")


def band_reduce(ctx: Context, W, P: int, M: int, N: int, bands: int, out, stream=None) -> None:
    _check(_lib.band_reduce(ctx.handle, _f32(W, "W"), P, M, N, bands, _bf16(out, "out"), _stream(stream)),
           "band_reduce")


def _xdtype(x, name: str = "x") -> int:
    if x.dtype is torch.bfloat16:
        return GEMMAR_DTYPE_BF16
    if x.dtype is torch.float32:
        return GEMMAR_DTYPE_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {x.dtype}")


def rowquant_e4m3(ctx: Context, x, q, row_scale, stream=None) -> None:
    M, N = x.shape
    _check(_lib.rowquant_e4m3(ctx.handle, _ptr(x, "x"), _xdtype(x), M, N, _u8(q, "q"),
                              _f32(row_scale, "row_scale"), _stream(stream)),
           "rowquant_e4m3")


def rowdequant_e4m3(ctx: Context, q, row_scale, y, stream=None) -> None:
    M, N = q.shape
    _check(_lib.rowdequant_e4m3(ctx.handle, _u8(q, "q"), _f32(row_scale, "row_scale"), M, N, _bf16(y, "y"),
                                _stream(stream)),
           "rowdequant_e4m3")


def quant_blockscale_e4m3(ctx: Context, x, group_rows: int, q, scales, stream=None) -> None:
    """Blockscale quantiser of a bf16 or fp32 [R, C] matrix (group_rows 1 or 128)."""
    R, C = x.shape
    _check(_lib.quant_blockscale_e4m3(ctx.handle, _ptr(x, "x"), _xdtype(x), R, C, group_rows, _u8(q, "q"),
                                      _f32(scales, "scales"), _stream(stream)),
           "quant_blockscale_e4m3")


def quant_mx_e4m3(ctx: Context, x, q, e8m0, stream=None) -> None:
    """mxfp8 quantiser (ue8m0 per 1x32) of a bf16 or fp32 [R, C] matrix."""
    R, C = x.shape
    _check(_lib.quant_mx_e4m3(ctx.handle, _ptr(x, "x"), _xdtype(x), R, C, _u8(q, "q"), _u8(e8m0, "e8m0"),
                              _stream(stream)),
           "quant_mx_e4m3")


def fused_gemm_reduce(ctx: Context, A: Sequence, sa: Sequence, B: Sequence, sb: Sequence, out,
                      scale_kind: int = GEMMAR_SCALE_BLOCK128, bands: int = 0, flags: int = 0,
                      stream=None) -> None:
    P = len(A)
    if not (len(sa) == len(B) == len(sb) == P):
        raise ValueError("A, sa, B, sb must have one entry per slice")
    M, K = A[0].shape
    N = B[0].shape[0]
    sc = _u8 if scale_kind == GEMMAR_SCALE_MX32 else _f32
    arr = lambda ptrs: (ctypes.c_void_p * P)(*ptrs)
    pa = arr([_u8(a, "A[p]") for a in A])
    pb = arr([_u8(b, "B[p]") for b in B])
    psa = arr([sc(s, "sa[p]") for s in sa])
    psb = arr([sc(s, "sb[p]") for s in sb])
    cast = lambda x: ctypes.cast(x, _PP)
    _check(_lib.fused_gemm_reduce(ctx.handle, P, cast(pa), cast(psa), cast(pb), cast(psb), scale_kind,
                                  M, N, K, bands, flags, _bf16(out, "out"), _stream(stream)),
           "fused_gemm_reduce")


def fused_gemm_reduce_noalloc(A: Sequence, sa: Sequence, B: Sequence, sb: Sequence, out, bands: int = 0,
                              stream=None) -> None:
    """Blockscale fused GEMM + band reduce that allocates no device memory
    (its scratch is fixed-size library memory, at most
    GEMMAR_NOALLOC_MAX_PARTIALS fp32 partials).  For callers that cannot call
    cudaMalloc, e.g. engines owning all device memory in a pool of their own."""
    P = len(A)
    if not (len(sa) == len(B) == len(sb) == P):
        raise ValueError("A, sa, B, sb must have one entry per slice")
    M, K = A[0].shape
    N = B[0].shape[0]
    arr = lambda ptrs: ctypes.cast((ctypes.c_void_p * P)(*ptrs), _PP)
    _check(_lib.fused_gemm_reduce_noalloc(P, arr([_u8(a, "A[p]") for a in A]), arr([_f32(s, "sa[p]") for s in sa]),
                                          arr([_u8(b, "B[p]") for b in B]), arr([_f32(s, "sb[p]") for s in sb]),
                                          M, N, K, bands, _bf16(out, "out"), _stream(stream)),
           "fused_gemm_reduce_noalloc")


def fused_gemm_reduce_noalloc_status():
    """(code, detail) of the last fused_gemm_reduce_noalloc call on the current
    device; call after its work has completed (code 0: every wait finished)."""
    d = ctypes.c_int(0)
    code = int(_lib.fused_gemm_reduce_noalloc_status(ctypes.byref(d)))
    return code, int(d.value)


# ---- the residual stream after wo_b, and adapters beside it --------------------------

# A decode step is a few microseconds of device time, so csrc/binding.cpp reads the tensors
# of these entry points and calls the library.  Where it finds one that does not fit, it
# answers -1 and the checks here say which and why.

def _refuse(t, shape, name: str, dtype, rows: bool):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must have contiguous rows" if rows else f"{name} must be contiguous")


def _dense(t, shape, name: str, dtype):
    """Pointer of a contiguous tensor of that shape and type; None stays None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, shape, name, dtype, False)


def _rows(t, shape, name: str, dtype=None):
    """(pointer, row stride) of a [rows, cols] matrix with contiguous rows, which may be a view."""
    try:
        if (dtype is None or t.dtype is dtype) and t.shape == shape and t.is_cuda:
            row, col = t.stride()
            if col == 1 or shape[1] == 1:
                return t.data_ptr(), row if shape[0] > 1 else shape[1]
    except AttributeError:
        pass
    _refuse(t, shape, name, dtype, True)


def _gate(gate, M: int, N: int):
    """(pointer, row stride) of a gate: [N] (stride 0) or [M, N]."""
    if gate is None:
        return None, 0
    if getattr(gate, "ndim", 2) == 1:
        return _dense(gate, (N,), "gate", torch.bfloat16), 0
    ptr, stride = _rows(gate, (M, N), "gate", torch.bfloat16)
    if stride == 0:
        raise ValueError("gate: pass one row for all rows as a tensor of shape [N]")
    return ptr, stride


def _codes(q, shape, name: str):
    if q is None:
        return None
    return _dense(q, shape, name, torch.uint8 if getattr(q, "dtype", None) is torch.uint8 else torch.float8_e4m3fn)


def _dims(t, name: str, dim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    return t.shape


def _explain_norm_gate_residual(y, h, w_pre, t, w_post, gate, u, q, scales, rstd):
    shape = M, N = _dims(y, "y", 2)
    _dims(h, "h", 2)
    f32, bf16 = torch.float32, torch.bfloat16
    _xdtype(y, "y"), _xdtype(h, "h")
    _rows(y, shape, "y")
    _rows(h, shape, "h")
    _gate(gate, M, N)
    for x, s, name, dtype in ((w_post, (N,), "w_post", f32), (w_pre, (N,), "w_pre", f32), (t, shape, "t", h.dtype),
                              (u, shape, "u", bf16), (scales, (M, N // 128), "scales", f32), (rstd, (M, 2), "rstd", f32)):
        _dense(x, s, name, dtype)
    _codes(q, shape, "q")


def _explain_norm_gate_residual_bwd(y, h, rstd, dt, dy, dh, w_post, w_pre, gate, du, dw_post, dw_pre, dgate):
    shape = M, N = _dims(y, "y", 2)
    _dims(h, "h", 2)
    f32, bf16 = torch.float32, torch.bfloat16
    _xdtype(y, "y"), _xdtype(h, "h")
    _rows(y, shape, "y")
    _rows(h, shape, "h")
    row = _gate(gate, M, N)[1] == 0
    if dt is not None:
        _rows(dt, shape, "dt", h.dtype)
    if du is not None:
        _rows(du, shape, "du", bf16)
    for x, s, name, dtype in ((rstd, (M, 2), "rstd", f32), (dy, shape, "dy", y.dtype), (dh, shape, "dh", h.dtype),
                              (w_post, (N,), "w_post", f32), (w_pre, (N,), "w_pre", f32), (dw_post, (N,), "dw_post", f32),
                              (dw_pre, (N,), "dw_pre", f32), (dgate, (N,) if row else shape, "dgate", f32 if row else bf16)):
        _dense(x, s, name, dtype)


def _explain_lora_operands(x, order, offsets, A, B, scales, ranks):
    T, K = _dims(x, "x", 2)
    R, r, _ = _dims(A, "A", 3)
    N = _dims(B, "B", 3)[2]
    i32, bf16 = torch.int32, torch.bfloat16
    _rows(x, (T, K), "x", bf16)
    for t, s, name, dtype in ((order, (T,), "order", i32), (offsets, (R + 1,), "offsets", i32), (A, (R, r, K), "A", bf16),
                              (B, (R, r, N), "B", bf16), (scales, (R,), "scales", torch.float32), (ranks, (R,), "ranks", i32)):
        _dense(t, s, name, dtype)
    return T, K, N, R, r


def _explain_lora_apply(x, order, offsets, A, B, scales, ranks, out, y, v):
    T, K, N, R, r = _explain_lora_operands(x, order, offsets, A, B, scales, ranks)
    _rows(out, (T, N), "out", torch.bfloat16)
    if y is not None:
        _rows(y, (T, N), "y", torch.bfloat16)
    _dense(v, (T, r), "v", torch.float32)


def _explain_lora_apply_bwd(x, order, offsets, A, B, scales, ranks, dy, v, dx, dA, dB, dx0):
    T, K, N, R, r = _explain_lora_operands(x, order, offsets, A, B, scales, ranks)
    bf16 = torch.bfloat16
    _rows(dy, (T, N), "dy", bf16)
    _rows(dx, (T, K), "dx", bf16)
    if dx0 is not None:
        _rows(dx0, (T, K), "dx0", bf16)
    for t, s, name, dtype in ((v, (T, r), "v", torch.float32), (dA, (R, r, K), "dA", bf16), (dB, (R, r, N), "dB", bf16)):
        _dense(t, s, name, dtype)


def _explain_gemm_blockscale_act(A, sa, B, sb, C, act, gated, bias, residual, q, scales, z):
    M, K = _dims(A, "A", 2)
    P = _dims(B, "B", 2)[0]
    if gated and P % 2:
        raise ValueError("B must have an even number of rows where the activation is gated")
    N = P // 2 if gated else P
    f32 = torch.float32
    for t, s, name in ((A, (M, K), "A"), (B, (P, K), "B"), (q, (M, N), "q")):
        _codes(t, s, name)
    for t, s, name, dtype in ((sa, (M, K // 128), "sa", f32), (sb, (P // 128, K // 128), "sb", f32), (bias, (P,), "bias", f32),
                              (scales, (M, N // 128), "scales", f32), (z, (M, P), "z", torch.bfloat16)):
        _dense(t, s, name, dtype)
    for t, name in ((C, "C"), (residual, "residual")):
        if t is not None:
            _dims(t, name, 2)
            _xdtype(t, name)
            _rows(t, (M, N), name)


def _explain_gemm_blockscale_act_bwd(dout, z, dz, act, gated, dbias, q, scales):
    M, N = _dims(dout, "dout", 2)
    P = 2 * N if gated else N
    _xdtype(dout, "dout")
    _rows(dout, (M, N), "dout")
    for t, s, name, dtype in ((z, (M, P), "z", torch.bfloat16), (dz, (M, P), "dz", torch.bfloat16), (dbias, (P,), "dbias", torch.float32),
                              (scales, (M, P // 128), "scales", torch.float32)):
        _dense(t, s, name, dtype)
    _codes(q, (M, P), "q")


def _explain_moe_route(x, router, ids, weights, bias):
    T, H = _dims(x, "x", 2)
    E = _dims(router, "router", 2)[0]
    k = _dims(ids, "ids", 2)[1]
    _xdtype(router, "router")
    _rows(x, (T, H), "x", torch.bfloat16)
    for t, s, name, dtype in ((router, (E, H), "router", router.dtype), (ids, (T, k), "ids", torch.int32), (weights, (T, k), "weights", torch.float32),
                              (bias, (E,), "bias", torch.float32)):
        _dense(t, s, name, dtype)


def _explain_moe_apply(q, sx, ids, weights, w13, s13, w2, s2, out, place, y):
    T, H = _dims(q, "q", 2)
    k = _dims(ids, "ids", 2)[1]
    E, _, inner = _dims(w2, "w2", 3)
    f32, i32 = torch.float32, torch.int32
    for t, s, name in ((q, (T, H), "q"), (w13, (E, 2 * inner, H), "w13"), (w2, (E, H, inner), "w2")):
        _codes(t, s, name)
    for t, s, name, dtype in ((sx, (T, H // 128), "sx", f32), (ids, (T, k), "ids", i32), (weights, (T, k), "weights", f32),
                              (s13, (E, 2 * inner // 128, H // 128), "s13", f32), (s2, (E, H // 128, inner // 128), "s2", f32)):
        _dense(t, s, name, dtype)
    if place is not None:
        _dense(place, _dims(place, "place", 1), "place", i32)
    _rows(out, (T, H), "out", torch.bfloat16)
    if y is not None:
        _rows(y, (T, H), "y", torch.bfloat16)


def norm_gate_residual(ctx: Context, y, h, w_pre, t, w_post=None, gate=None, alpha: float = 1.0, beta: float = 1.0,
                       eps: float = 1e-6, u=None, q=None, scales=None, rstd=None, stream=None) -> None:
    """t = alpha*h + beta*gate*norm(y)*w_post and the next block's input norm(t)*w_pre, as bf16 rows u
    and/or e4m3 codes q with fp32 scales per 1x128 (gemm_blockscale_fp8's A operand).  w_post None: no
    post norm; w_pre None: t only; gate bf16 [N] or [M, N]; rstd fp32 [M, 2] for the backward pass."""
    rc = _operators.norm_gate_residual(ctx.handle.value, y, h, w_pre, t, w_post, gate, alpha, beta, eps, u, q,
                                       scales, rstd, _stream(stream))
    if rc < 0:
        _explain_norm_gate_residual(y, h, w_pre, t, w_post, gate, u, q, scales, rstd)
        raise ValueError("norm_gate_residual: an argument does not fit")
    if rc:
        _check(rc, "norm_gate_residual")


def norm_gate_residual_bwd(ctx: Context, y, h, rstd, dt, dy, dh, w_post=None, w_pre=None, gate=None,
                           alpha: float = 1.0, beta: float = 1.0, du=None, dw_post=None, dw_pre=None, dgate=None,
                           stream=None) -> None:
    """Gradients of norm_gate_residual from dt (of t; None: zero) and du (of the normed rows), given its
    inputs and rstd.  dw_post, dw_pre fp32 [N]; dgate fp32 [N] for a gate row, bf16 [M, N] per token."""
    rc = _operators.norm_gate_residual_bwd(ctx.handle.value, y, h, rstd, dt, dy, dh, w_post, w_pre, gate, alpha, beta, du,
                                           dw_post, dw_pre, dgate, _stream(stream))
    if rc < 0:
        _explain_norm_gate_residual_bwd(y, h, rstd, dt, dy, dh, w_post, w_pre, gate, du, dw_post, dw_pre, dgate)
        raise ValueError("norm_gate_residual_bwd: an argument does not fit")
    if rc:
        _check(rc, "norm_gate_residual_bwd")


def lora_plan(ctx: Context, adapter_ids, order, offsets, stream=None) -> None:
    """Sort a batch's tokens by adapter: order int32 [T] and offsets int32 [R+1] from adapter_ids int32 [T]
    (an id outside [0, R) is a token without one).  One plan serves every layer of the batch."""
    T, R = _dims(adapter_ids, "adapter_ids", 1)[0], _dims(offsets, "offsets", 1)[0] - 1
    i32 = torch.int32
    _check(_lib.lora_plan(ctx.handle, _dense(adapter_ids, (T,), "adapter_ids", i32), T, R,
                          _dense(order, (T,), "order", i32), _dense(offsets, (R + 1,), "offsets", i32),
                          _stream(stream)),
           "lora_plan")


def lora_apply(ctx: Context, x, order, offsets, A, B, scales, ranks, out, y=None, v=None, stream=None) -> None:
    """out = y + the tokens' adapters applied to x: scales[a] * (x[t] A[a]^T) B[a], A [R, r, K] and B [R, r, N]
    bf16, ranks int32 [R] or None.  y None: zero; y may be out.  v fp32 [T, r]: kept for the backward pass."""
    rc = _operators.lora_apply(ctx.handle.value, x, order, offsets, A, B, scales, ranks, out, y, v, _stream(stream))
    if rc < 0:
        _explain_lora_apply(x, order, offsets, A, B, scales, ranks, out, y, v)
        raise ValueError("lora_apply: an argument does not fit")
    if rc:
        _check(rc, "lora_apply")


def lora_apply_bwd(ctx: Context, x, dy, order, offsets, A, B, scales, ranks, v, dx, dA, dB, dx0=None,
                   stream=None) -> None:
    """Gradients of lora_apply: dx = dx0 + the adapters' part (dx0 None: zero; may be dx), dA and dB of A's
    and B's shapes, from dy, the forward pass's x and its v."""
    rc = _operators.lora_apply_bwd(ctx.handle.value, x, order, offsets, A, B, scales, ranks, dy, v, dx, dA, dB, dx0,
                                   _stream(stream))
    if rc < 0:
        _explain_lora_apply_bwd(x, order, offsets, A, B, scales, ranks, dy, v, dx, dA, dB, dx0)
        raise ValueError("lora_apply_bwd: an argument does not fit")
    if rc:
        _check(rc, "lora_apply_bwd")


# ---- the feed-forward half -------------------------------------------------------------

def gemm_blockscale_act(ctx: Context, A, sa, B, sb, C, act: int = GEMMAR_ACT_NONE, gated: bool = False, bias=None,
                        residual=None, q=None, scales=None, z=None, stream=None) -> None:
    """out = residual + act(z), z = A B^T + bias of block-scaled e4m3 codes; gated: B holds 2N rows and out =
    residual + act(z[:, :N]) * z[:, N:].  out goes to C (bf16 or fp32, may be a view, may be residual itself;
    None: left out) and/or to e4m3 codes q with scales [M, N/128]; z bf16 is kept for the backward pass."""
    rc = _operators.gemm_blockscale_act(ctx.handle.value, A, sa, B, sb, C, act, gated, bias, residual, q, scales, z,
                                        _stream(stream))
    if rc < 0:
        _explain_gemm_blockscale_act(A, sa, B, sb, C, act, gated, bias, residual, q, scales, z)
        raise ValueError("gemm_blockscale_act: an argument does not fit")
    if rc:
        _check(rc, "gemm_blockscale_act")


def gemm_blockscale_act_bwd(ctx: Context, dout, z, dz, act: int = GEMMAR_ACT_NONE, gated: bool = False, dbias=None,
                            q=None, scales=None, stream=None) -> None:
    """dz = the gradient of z from dout, as bf16 rows (None: left out) and/or e4m3 codes q with 1x128 scales;
    dbias fp32 [N or 2N] its sums over the rows.  A's gradient is gemm_blockscale_fp8 of those codes with B's
    codes and scales transposed; residual's is dout."""
    rc = _operators.gemm_blockscale_act_bwd(ctx.handle.value, dout, z, dz, act, gated, dbias, q, scales, _stream(stream))
    if rc < 0:
        _explain_gemm_blockscale_act_bwd(dout, z, dz, act, gated, dbias, q, scales)
        raise ValueError("gemm_blockscale_act_bwd: an argument does not fit")
    if rc:
        _check(rc, "gemm_blockscale_act_bwd")


def moe_route(ctx: Context, x, router, ids, weights, bias=None, score: int = GEMMAR_SCORE_SOFTMAX, renorm: bool = True,
              factor: float = 1.0, stream=None) -> None:
    """Each token's k experts: ids int32 [T, k] of the largest softmax or sigmoid scores of x router^T (+ bias, for
    the choice alone) and their weights fp32 [T, k], over their sum where renorm, times factor."""
    rc = _operators.moe_route(ctx.handle.value, x, router, ids, weights, bias, score, renorm, factor, _stream(stream))
    if rc < 0:
        _explain_moe_route(x, router, ids, weights, bias)
        raise ValueError("moe_route: an argument does not fit")
    if rc:
        _check(rc, "moe_route")


def moe_apply(ctx: Context, q, sx, ids, weights, w13, s13, w2, s2, out, act: int = GEMMAR_ACT_SILU, place=None, y=None,
              stream=None) -> None:
    """out = y + each token's experts applied to its codes q, sx: weights * w2[e] (act(gate) * up) with gate and up the
    halves of w13[e].  ids outside the experts add nothing; place int32 maps the router's numbers to rows of w13 and
    w2 (-1: held elsewhere).  y None: zero; y may be out."""
    rc = _operators.moe_apply(ctx.handle.value, q, sx, ids, weights, w13, s13, w2, s2, out, act, place, y, _stream(stream))
    if rc < 0:
        _explain_moe_apply(q, sx, ids, weights, w13, s13, w2, s2, out, place, y)
        raise ValueError("moe_apply: an argument does not fit")
    if rc:
        _check(rc, "moe_apply")
