"""v in another format than k, where k's rotated lanes need the general kernel
and v's do not, and the other way round."""
import pytest
import torch

import transformer_positional_encoding_amd as rp
from axes_refs import pair_tables
from cache_refs import rotate32
from test_cache_gpu import expect_written, make_cache, slots_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D, Dv, sl, mode", [(128, 128, (3, 61), "rotate_half"), (128, 64, (0, 128), "rotate_half"),
                                             (36, 128, (1, 35), "interleave"), (128, 36, (0, 64), "interleave"),
                                             (576, 512, (512, 576), "interleave")])
@pytest.mark.parametrize("kf, vf", [("e4m3", "int8"), ("same", "int4"), ("int8", "same")])
def test_write(D, Dv, sl, mode, kf, vf):
    B, S, N, Nq, pages, page = 2, 9, 2, 5, 7, 4
    g = torch.Generator().manual_seed(D + Dv)
    q, k, v = (torch.randn(B, S, n, d, generator=g).bfloat16() for n, d in ((Nq, D), (N, D), (N, Dv)))
    kc, vc = make_cache(pages, page, N, D, kf, D, "bf16"), make_cache(pages, page, N, Dv, vf, Dv, "bf16")
    slots = slots_for(B, S, pages, page, 3, 2)
    L = sl[1] - sl[0]
    pos, f = torch.randint(0, 9000, (1, B, S), generator=g), rp.rope_inv_freq(L)
    qd = q.cuda()
    rp.rope_cache_write(k.cuda(), v.cuda(), kc, vc, slots.cuda(), pos[0].cuda(), f.cuda(), mode, sl, q=qd)
    cos, sin = pair_tables(pos, f, (0,) * (L // 2), "bf16")
    expect_written(kc, slots, rotate32(k, cos, sin, mode, sl), kf, D, "bf16", "k")
    expect_written(vc, slots, v.float(), vf, Dv, "bf16", "v")
    assert torch.equal(qd.cpu(), rotate32(q, cos, sin, mode, sl).bfloat16())
