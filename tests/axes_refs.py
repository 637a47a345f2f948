"""The rotation from positions on several axes, in 64 bits, for the tests.

Angles, cos and sin are evaluated in fp64 and rounded once to the table's type
(through an fp64 grid, not through fp32), as the operation defines them; the
rotation itself then stays in fp64.
"""
from __future__ import annotations

import torch

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BITS = {"f32": (24, -126), "f16": (11, -14), "bf16": (8, -126)}


def round_to(v: torch.Tensor, dtype: str) -> torch.Tensor:
    """fp64 values rounded to nearest even in `dtype`, still fp64."""
    p, emin = BITS[dtype]
    e = torch.clamp(torch.frexp(v)[1], min=emin + 1)
    unit = torch.ldexp(torch.ones_like(v), e - p)
    return torch.round(v / unit) * unit


def half_of(mode, L: int) -> int:
    return 1 if mode == "interleave" else L // 2 if mode == "rotate_half" else L // int(mode)


def pair_tables(positions, inv_freq, pair_axes, table: str):
    """(cos, sin), each (Bp, S, 1, pairs) fp64 values of the table's type.
    positions (A, Bp, S), inv_freq (pairs), any device; computed on the CPU."""
    pos = positions.cpu()[torch.tensor(pair_axes, dtype=torch.long)].permute(1, 2, 0).double()
    th = pos * inv_freq.cpu()
    return round_to(torch.cos(th), table)[:, :, None], round_to(torch.sin(th), table)[:, :, None]


def rotate64(x: torch.Tensor, cos, sin, mode, sl, back: bool = False):
    """x fp64 (B, S, N, D) with its slice rotated, and the size of the terms,
    |x_j c| + |x_p s| (0 outside the slice)."""
    s, e = sl
    L = e - s
    y, size = x.clone(), torch.zeros_like(x)
    if L == 0:
        return y, size
    h = half_of(mode, L)
    j = torch.arange(L)
    first = (j // h) % 2 == 0
    other = torch.where(first, j + h, j - h)
    pair = j // (2 * h) * h + j % h
    c, sn = cos[..., pair], sin[..., pair]
    sign = torch.where(first, -1.0, 1.0).double() * (-1.0 if back else 1.0)
    z = x[..., s:e]
    a, b = z * c, z[..., other] * sn
    y[..., s:e] = a + sign * b
    size[..., s:e] = a.abs() + b.abs()
    return y, size


def bound(want, size, dtype: str):
    """How far a result may lie from the fp64 one: the two products and the
    sum round to fp32, at most 2^-24 of the terms' size each (4 for the
    second-order parts), then one rounding to the storage type, half a unit in
    the last place (eps/2 of the value, or half the least subnormal)."""
    arith = 4 * 2.0 ** -24 * size + 2.0 ** -149
    if dtype == "f32":
        return arith
    p, emin = BITS[dtype]
    return arith + 2.0 ** -p * (want.abs() + arith) + 2.0 ** (emin - p)


def check(got, want, size, x, sl, dtype: str, what: str):
    """got (storage) against want (fp64): within the bound on the slice, and
    outside it the bytes of x."""
    s, e = sl
    got, x = got.detach().cpu(), x.detach().cpu()
    for part in (slice(0, s), slice(e, None)):
        assert torch.equal(got[..., part].contiguous().view(torch.uint8), x[..., part].contiguous().view(torch.uint8)), \
            f"{what}: lanes outside the slice changed"
    err = (got.double() - want).abs()[..., s:e]
    lim = bound(want, size, dtype)[..., s:e]
    assert bool((err <= lim).all()), f"{what}: {int((err > lim).sum())} lanes off, worst {float((err / lim).max()):.3g} of the bound"
