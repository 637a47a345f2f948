"""Reads of tokens whose width decides between the read's two vector kernels, on
both sides of each border, turned and not, against the definition."""
import pytest
import torch

import transformer_positional_encoding_amd as rp
from axes_refs import pair_tables
from test_cache_gpu import filled, read_want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N, D", [(7, 56), (7, 64), (63, 8), (4, 128), (8, 64), (13, 40), (12, 64), (97, 8), (7, 128),
                                  (15, 64), (127, 8), (1, 1016), (8, 128), (1, 1024), (129, 8), (17, 64), (9, 128), (20, 64)])
@pytest.mark.parametrize("fmt, out", [("e4m3", "bf16"), ("int4", "f32"), ("f16", "f16")])
def test_read_on_both_sides_of_a_border(N, D, fmt, out):
    B, S, page, pages = 3, 90, 16, 30
    c = filled(pages, page, N, D, fmt, D, out, N)
    g = torch.Generator().manual_seed(N)
    table = torch.randperm(pages, generator=g)[:18].view(3, 6).to(torch.int32)
    lengths = torch.tensor([90, 0, 61], dtype=torch.int32)
    starts = [0, 5, 2]
    pos = torch.randint(0, 50000, (1, B, S), generator=g)
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}[out]
    for L in (0, 8, 64, D // 16 * 16):
        if L > D:
            continue
        got = torch.full((B, S, N, D), 3.0, dtype=dtype, device="cuda")
        sl, f = (D - L, D), rp.rope_inv_freq(max(2, L))
        kw = dict(positions=pos[0].cuda(), inv_freq=f.cuda(), rotary_mode="rotate_half", partial_slice=sl) if L else {}
        turn = pair_tables(pos, f, (0,) * (L // 2), out) if L else None
        want = read_want(c, got, table, lengths, starts, turn, "rotate_half", sl, out)
        rp.rope_cache_read(got, c, table.cuda(), lengths.cuda(), starts=torch.tensor(starts, dtype=torch.int32).cuda(), **kw)
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8)), f"{L} lanes turned"
