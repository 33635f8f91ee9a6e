"""Plain 64-bit forms of the paged cache's operators, for the tests: the 4-bit code, the rotation, the page map, and
attention over gathered values.  Nothing here uses the library."""
from __future__ import annotations

import math

import numpy as np
import torch

F16_MAX = 65504.0
E4M3_MAX = 448.0


def encode_int4(x: torch.Tensor):
    """Codes uint8 [..., D/2] and fp16 (scale, zero) [..., 2] of x [..., D], each step in fp32 as the header states it."""
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=F16_MAX, neginf=-F16_MAX).clamp(-F16_MAX, F16_MAX)
    zero = x.amin(-1, keepdim=True).half()
    step = ((x.amax(-1, keepdim=True) - zero.float()) * np.float32(1.0 / 15.0)).clamp(min=0).half()
    inv = torch.where(step > 0, 1.0 / step.float(), torch.zeros_like(step.float()))
    u = ((x - zero.float()) * inv).round().clamp(0, 15).to(torch.uint8)
    return pack_int4(u), torch.cat([step, zero], -1)


def pack_int4(u: torch.Tensor) -> torch.Tensor:
    return u[..., 0::2] | (u[..., 1::2] << 4)


def unpack_int4(b: torch.Tensor) -> torch.Tensor:
    return torch.stack([b & 15, b >> 4], -1).flatten(-2)


def value_int4(codes, params):
    """64-bit values of codes [..., D/2] with params [..., 2] (scale, zero)."""
    p = params.double()
    return unpack_int4(codes).double() * p[..., 0:1] + p[..., 1:2]


def values(kind, codes, params=None, scale=1.0):
    if kind == "int4":
        return value_int4(codes, params)
    if kind == "fp8":
        return codes.view(torch.float8_e4m3fn).double() * scale
    if kind == "int8":
        return codes.double() * scale
    return codes.double()


def encode(kind, x, scale=1.0):
    """Codes of fp32 x as the append states them (None params except for int4)."""
    if kind == "bf16":
        return x.to(torch.bfloat16), None
    if kind == "int4":
        return encode_int4(x)
    y = x * float(np.float32(1.0) / np.float32(scale))
    if kind == "fp8":
        return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8), None
    return torch.nan_to_num(y, nan=0.0).round().clamp(-127, 127).to(torch.int8), None


def rotate(x: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor, rot: int, interleaved: bool) -> torch.Tensor:
    """x [T, H, D] with cos, sin [T, rot/2], in x's own precision, one rounding an operation."""
    y = x.clone()
    half = torch.arange(rot // 2)
    i, j = (2 * half, 2 * half + 1) if interleaved else (half, half + rot // 2)
    c, s = cos[:, None].to(x.dtype), sin[:, None].to(x.dtype)
    a, b = x[..., i], x[..., j]
    y[..., i] = a * c - b * s
    y[..., j] = b * c + a * s
    return y


def rope_table(max_pos: int, rot: int, base=10000.0) -> torch.Tensor:
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], -1).float()


def slots(page_table_row, page_size: int, positions):
    p = torch.as_tensor(positions, dtype=torch.int64)
    return page_table_row.long()[p // page_size] * page_size + p % page_size


def attend(q, k, v, n_visible):
    """64-bit softmax attention of q [Hq, D] over the first n_visible of k, v [n, Hkv, D] (double); scale 1/sqrt(D).
    Returns (out [Hq, D], lse [Hq])."""
    Hq, D = q.shape
    Hkv = k.shape[1]
    if n_visible <= 0:
        return torch.zeros(Hq, D, dtype=torch.float64), torch.full((Hq,), -math.inf, dtype=torch.float64)
    k, v = k[:n_visible], v[:n_visible]
    x = torch.einsum("hgd,thd->hgt", q.double().view(Hkv, Hq // Hkv, D), k) / math.sqrt(D)
    return (torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v).reshape(Hq, D), torch.logsumexp(x, -1).reshape(Hq))


def int4_bounds(q, params, D):
    """(score error, range of V) bounds of the 4-bit decode for query rows q [..., D] and a request's params [n, Hkv, 4].

    The kernel's only roundings of a score are fp32 additions and products: a dot product of D terms of at most
    |q_d| 15 ks, its scale, and the zero's term |kz| sum|q|, each within 2^-23 of the sum of magnitudes (a tensor
    core may truncate where fp32 rounds): |error| <= (D + 8) 2^-23 (15 ks + |kz|) sum|q| / sqrt(D).  The weights of
    V are rounded to fp16, 2^-11 each, on codes worth at most 15 vs."""
    p = params.double().reshape(-1, 4)
    if p.numel() == 0:
        return 0.0, 0.0, 0.0
    k_mag = float((15 * p[:, 0] + p[:, 1].abs()).max())
    v_range = float((15 * p[:, 2]).max())
    v_mag = float((15 * p[:, 2] + p[:, 3].abs()).max())
    return (D + 8) * 2.0 ** -23 * k_mag * float(q.double().abs().sum(-1).max()) / math.sqrt(D), v_range, v_mag
