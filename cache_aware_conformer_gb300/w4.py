"""Weights at 4 bits for cac_op_gemm_w4: W[n][k] = scale[n][k / group] *
(code[n][k] - zero[n][k / group]), two codes to a byte, the even k in the low half.

Rounding to nearest by the range of each group: a compression tool for users of the
library, not an optimal quantiser; codes from any other method go through the same
entry point.  Plain torch, on any device.
"""
from __future__ import annotations

import torch

GROUPS = (32, 64, 128)


def quantize(w, group: int = 64, zeros: bool = False):
    """(packed uint8 [N, K/2], scale bf16 [N, K/group], zero uint8 [N, K/group] or None) of w [N, K].  Without zeros the
    codes lie around 8 and the scale is the group's largest value / 7; with them the group's range, 0 included, is spread
    over the 16 codes.  The codes are those nearest under the scale as it is rounded to bf16."""
    N, K = w.shape
    if group not in GROUPS or K % group:
        raise ValueError(f"group: one of {GROUPS} that divides {K}")
    x = w.float().view(N, K // group, group)
    if not bool(torch.isfinite(x).all()):
        raise ValueError("weights have to be finite")
    if zeros:
        lo, hi = x.amin(-1).clamp_max(0), x.amax(-1).clamp_min(0)
        scale = ((hi - lo) / 15).to(torch.bfloat16)
        at = torch.where(scale > 0, scale.float(), 1.0)
        zero = torch.round(-lo / at).clamp(0, 15)
    else:
        scale = (x.abs().amax(-1) / 7).to(torch.bfloat16)
        at = torch.where(scale > 0, scale.float(), 1.0)
        zero = torch.full_like(at, 8.0)
    code = torch.round(x / at[..., None] + zero[..., None]).clamp(0, 15).to(torch.uint8).view(N, K)
    return pack(code), scale, zero.to(torch.uint8) if zeros else None


def pack(code):
    """uint8 codes 0 .. 15 [N, K] as bytes [N, K/2]."""
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def unpack(packed):
    """The codes [N, K] of packed bytes."""
    return torch.stack([packed & 15, packed >> 4], -1).view(packed.size(0), -1)


def dequantize(packed, scale, zero=None):
    """The weights that the codes stand for, fp64 [N, K]."""
    code = unpack(packed).double().view(*scale.shape, -1)
    return ((code - (8.0 if zero is None else zero.double()[..., None])) * scale.double()[..., None]).view(packed.size(0), -1)
