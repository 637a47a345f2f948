"""The quantised cache's definition in 64 bits, for the tests (CPU tensors)."""
from __future__ import annotations

import torch

from axes_refs import half_of

QMAX = {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}


def grid(v: torch.Tensor, fmt: str) -> torch.Tensor:
    """fp64 values rounded to the format's nearest, ties to even."""
    q = QMAX[fmt]
    if fmt != "e4m3":
        return torch.round(v).clamp(-q, q)
    e = torch.clamp(torch.frexp(v)[1] - 1, min=-6)
    unit = torch.ldexp(torch.ones_like(v), e - 3)
    return (torch.round(v / unit) * unit).clamp(-q, q)


def encode(z: torch.Tensor, fmt: str, group: int):
    """(codes, scales) of fp32 rows z (..., D) as fp64 values: the quotient of
    two fp32 numbers lies at least 2^-33 of its size away from a midpoint that
    it does not equal (both have 24 bits, a midpoint 8), so its fp64 rounding
    falls on the right side."""
    z = z.double()
    g = z.unflatten(-1, (-1, group))
    m = torch.where(torch.isfinite(g), g.abs(), torch.zeros_like(g)).amax(-1)
    s = torch.where(m > 0, (m / QMAX[fmt]).float().double().clamp(min=2.0 ** -100), torch.ones_like(m))
    c = grid(torch.minimum(torch.maximum(g, -m[..., None]), m[..., None]) / s[..., None], fmt)
    nan = torch.isnan(g)
    c = torch.where(nan, torch.full_like(c, float("nan") if fmt == "e4m3" else 0.0), c)
    return c.flatten(-2), s


def decode_codes(data: torch.Tensor) -> torch.Tensor:
    """The codes a cache tensor holds, as fp64."""
    data = data.cpu()
    if data.dtype != torch.uint8:
        return data.float().double()
    w = data.to(torch.int64)
    both = torch.stack([w & 15, w >> 4], dim=-1).flatten(-2)
    return torch.where(both > 7, both - 16, both).double()


def rotate32(x: torch.Tensor, cos, sin, mode, sl) -> torch.Tensor:
    """x (B, S, N, D) as fp32 with its slice rotated in fp32, every product and
    sum rounded (what the operation defines for the cache); cos and sin fp64
    tables (Bp, S, 1, pairs)."""
    s, e = sl
    y = x.float().clone()
    if e == s:
        return y
    h = half_of(mode, e - s)
    j = torch.arange(e - s)
    first = (j // h) % 2 == 0
    other = torch.where(first, j + h, j - h)
    pair = j // (2 * h) * h + j % h
    c, sn = cos.float()[..., pair], sin.float()[..., pair]
    z = x.float()[..., s:e]
    t = z[..., other] * sn
    y[..., s:e] = z * c + torch.where(first, -t, t)
    return y
