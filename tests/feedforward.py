"""Operands, definitions in 64 bits and derived tolerances of the feed-forward operators' tests."""
import math

import torch

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
BF16, E4M3 = 2.0 ** -8, 2.0 ** -4   # half a step, relative


def codes_1x128(x):
    """e4m3 codes (uint8) and scales per row and 128 columns; a zero group has scale 0."""
    g = x.float().view(x.shape[0], -1, 128)
    s = g.abs().amax(2) / 448
    q = torch.where(s[..., None] > 0, g / s[..., None], torch.zeros_like(g))
    return q.view(x.shape).to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), s.contiguous()


def codes_128x128(w):
    b = w.float().view(w.shape[0] // 128, 128, w.shape[1] // 128, 128)
    s = b.abs().amax((1, 3)) / 448
    q = torch.where(s[:, None, :, None] > 0, b / s[:, None, :, None], torch.zeros_like(b))
    return q.view(w.shape).to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), s.contiguous()


def values(q, s):
    """fp64 values of codes; s [rows, K/128] or [rows/128, K/128]."""
    per = q.shape[0] // s.shape[0]
    return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(per, 0).repeat_interleave(128, 1)


def value(act, z):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "gelu_tanh":
        # (1 + tanh u) / 2 as the sigmoid of 2 u: the first form cancels to 0 for z below -7 even in 64 bits
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return z


def product(A, sa, B, sb):
    """z = A B^T in fp64 and a bound on an fp32 evaluation's error: per 128 of K one accumulation of the
    MMA (four steps of 32, each with at most 8 roundings of 2^-23), the product of two scales and a
    multiply-add, then one addition per block of K; every term relative to the sum of the terms' sizes."""
    a, b = values(A, sa), values(B, sb)
    sizes = a.abs() @ b.abs().T
    return a @ b.T, (8 + 4 + A.shape[1] // 128) * 2.0 ** -23 * sizes


def value_error(act, z, dz):
    """Bound on the error of act(z) in fp32 where z is off by dz: slopes are at most 1.13; the functions'
    factor in [0, 1] is off by (8 + z^2 + 0.15 |z|^3) 2^-23 relative, which the rounding of its
    argument gives for the steepest of the five."""
    a = value(act, z).abs()
    return 1.13 * dz + a * (8 + z.abs() ** 2 + 0.15 * z.abs() ** 3).clamp(max=2.0 ** 12) * 2.0 ** -23


def act_reference(A, sa, B, sb, act, gated, bias=None, residual=None):
    """(out, its fp32 error bound, z, its bound)."""
    z, ez = product(A, sa, B, sb)
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0 ** -24 * z.abs()
    if gated:
        zg, zu = z.chunk(2, 1)
        eg, eu = ez.chunk(2, 1)
        a = value(act, zg) * zu
        err = value_error(act, zg, eg) * (zu.abs() + eu) + value(act, zg).abs() * eu + 2.0 ** -24 * a.abs()
    else:
        a, err = value(act, z), value_error(act, z, ez)
    if residual is not None:
        a = a + residual.double()
        err = err + 2.0 ** -24 * a.abs()
    return a, err, z, ez


def within(got, ref, bound, what=""):
    got, ref = got.double(), ref.double()
    assert torch.isfinite(got).all(), what
    bad = (got - ref).abs() > bound
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got - ref).abs() / bound.clamp(min=1e-300)).max():.2f} of the bound"


def codes_within(q, s, ref, err, what=""):
    """Codes and scales of the fp32 value of ref, which is off by err: the scale is the group's largest
    over 448; a code stands for its value to half a step, 2^-4 of it or 2^-10 of a scale."""
    top = ref.abs().view(*s.shape, 128).amax(2)
    terr = err.view(*s.shape, 128).amax(2)
    within(s, top / 448, terr / 448 + 2.0 ** -23 * top / 448, what + " scales")
    got = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)
    step = torch.maximum(E4M3 * (ref.abs() + err), 2.0 ** -10 * s.double().repeat_interleave(128, 1))
    # near the largest value the scale's own error can push it past 448, where codes saturate
    within(got, ref, 1.001 * err + 1.0001 * step + terr.repeat_interleave(128, 1), what + " codes")
