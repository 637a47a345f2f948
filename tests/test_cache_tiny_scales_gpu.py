"""Codes of groups whose scale lies just above the least one, 2^-100: where the
exact quotient is next to a midpoint, its residual is an fp32 subnormal."""
import pytest
import torch

import transformer_positional_encoding_amd as rp
from cache_refs import QMAX
from test_cache_gpu import expect_written, make_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [128, 36])
@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
def test_quotients_next_to_midpoints_at_the_least_scales(fmt, D):
    """Values next to every midpoint times the scale, for scales one unit and
    a few above 2^-100 and up to 2^-92, on the vector and the general kernel."""
    q = QMAX[fmt]
    if fmt == "e4m3":
        v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
        mids = (v[1:] + v[:-1]) / 2
    else:
        mids = torch.arange(0, int(q)).double() + 0.5
    rows = []
    for k in [1, 2, 3, 7, 1001, 2 ** 22 + 1, 2 ** 23 - 1] + [2 ** 23 * (2 ** i - 1) + 5 * 2 ** i for i in range(1, 8)]:
        # the scale of a group is its largest magnitude / q rounded to fp32
        m = torch.tensor(q * 2.0 ** -100 * (1 + k * 2.0 ** -23), dtype=torch.float64).float()
        s = (m.double() / q).float().double()
        t = (mids * s).float()
        vals = torch.cat([torch.nextafter(t, torch.zeros_like(t)), t, torch.nextafter(t, t * 2)])
        vals = torch.cat([vals, -vals])
        full = torch.zeros(-(-len(vals) // (D - 1)) * (D - 1))
        full[:len(vals)] = vals
        rows.append(torch.cat([m.expand(len(full) // (D - 1), 1), full.view(-1, D - 1)], 1))
    rows = torch.cat(rows)[None, :, None]
    assert float(rows.abs().max()) < 2.0 ** -80
    n = rows.shape[1]
    c = make_cache(n, 1, 1, D, fmt, D, "f32")
    slots = torch.arange(n)[None]
    rp.rope_cache_write(rows.cuda(), None, c, None, slots.cuda())
    expect_written(c, slots, rows, fmt, D, "f32", "least scales")
