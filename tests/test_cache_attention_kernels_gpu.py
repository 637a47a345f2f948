"""Attention over a paged cache in 4 bits: each kernel a call may take, at the
sizes, masks and layouts where it could go wrong, against the definition in 64
bits."""
import pytest
import torch

import transformer_positional_encoding_amd as rp
from test_cache_attention_gpu import call, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads, hq, S", [(4, 4, 1), (4, 16, 4), (8, 32, 1), (12, 24, 2), (8, 8, 16)])
@pytest.mark.parametrize("D, page, dtype", [(128, 16, "bf16"), (128, 48, "f16"), (64, 16, "f16"), (64, 1024, "bf16")])
def test_four_heads_beside_each_other(heads, hq, S, D, page, dtype):
    lengths = [1, 16, 63, 64, 65, 0, 129, 700, S]
    c = inputs(lengths, S, hq, heads, D, D, D, D, page, dtype, seed=31)
    for causal in (True, False):
        check(call(c, causal=causal), c, causal=causal)
    counts = torch.tensor([S, 0, S + 2, 1, S, S, -1, max(1, S // 2), S], dtype=torch.int32)
    got = call(c, counts=counts)
    check(got, c, counts=counts)
    for b, n in enumerate(counts.tolist()):
        assert torch.equal(got[b, min(max(n, 0), S):].cpu(), c["out"][b, min(max(n, 0), S):])


@pytest.mark.parametrize("D", [64, 128])
def test_four_heads_pages_outside_the_cache_and_what_no_row_sees(D):
    c = inputs([200, 170, 90, 333], 2, 8, 4, D, D, D, D, 16, "bf16", seed=32)
    c["table"][0, 3], c["table"][0, 7], c["table"][1, :] = -1, 10 ** 6, -1
    c["table"][2, 0] = c["k"][0].shape[0]
    want = call(c)
    check(want, c)
    assert not bool(want[1].any())
    for name in ("k", "v"):
        data, scales = c[name]
        live = torch.zeros(data.shape[:2], dtype=torch.bool)
        for b, n in enumerate(c["lengths"].tolist()):
            t = torch.arange(n)
            at = c["table"][b, t // 16].long()
            ok = (at >= 0) & (at < data.shape[0])
            live[at[ok], (t % 16)[ok]] = True
        data[~live], scales[~live] = 0x88, float("nan")
    assert torch.equal(call(c), want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("span", [3.0, 12.0])
def test_four_heads_scales_far_apart(D, span):
    c = inputs([500, 333], 2, 8, 4, D, D, D, D, 16, "bf16", seed=33, span=span)
    c["k"] = (c["k"][0], c["k"][1].clamp(max=4.0))
    check(call(c), c)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout", ["halves", "gaps", "heads first", "scales shifted", "scales apart", "codes shifted"])
def test_four_heads_layouts(D, layout):
    """Caches whose heads' rows and scales lie side by side, and those where
    they do not."""
    c = inputs([130, 77, 1], 1, 8, 4, D, D, D, D, 16, "bf16", seed=34)
    on = {n: c[n].cuda() for n in ("q", "table", "lengths")}

    def laid(data, scales):
        data, scales = data.cuda(), scales.cuda()
        P = data.shape[0]
        if layout == "halves":                     # K (or V) of a page beside other bytes
            both = torch.full((P, 2, 16, 4, D // 2), 0x77, dtype=torch.uint8, device="cuda")
            both[:, 1] = data
            data = both[:, 1]
        elif layout == "gaps":                     # more heads than are cached here
            wide = torch.full((P, 16, 8, D // 2), 0x77, dtype=torch.uint8, device="cuda")
            wide[:, :, 4:] = data
            more = torch.full((P, 16, 8, 1), float("nan"), device="cuda")
            more[:, :, 4:] = scales
            data, scales = wide[:, :, 4:], more[:, :, 4:]
        elif layout == "heads first":
            data, scales = data.transpose(1, 2).contiguous().transpose(1, 2), scales.transpose(1, 2).contiguous().transpose(1, 2)
        elif layout == "scales shifted":
            more = torch.full((scales.numel() + 1,), float("nan"), device="cuda")
            more[1:] = scales.reshape(-1)
            scales = more[1:].view(scales.shape)
        elif layout == "scales apart":
            more = torch.full((P, 16, 5, 1), float("nan"), device="cuda")
            more[:, :, :4] = scales
            scales = more[:, :, :4]
        else:
            more = torch.full((data.numel() + 4,), 0x77, dtype=torch.uint8, device="cuda")
            more[4:] = data.reshape(-1)
            data = more[4:].view(data.shape)
        return rp.RopeCache(data, scales)

    got = rp.rope_cache_attention(on["q"], laid(*c["k"]), laid(*c["v"]), on["table"], on["lengths"], out=c["out"].cuda())
    check(got, c)
    if layout != "codes shifted":                  # (codes off 16 bytes: a score's 32-bit sums run in another order)
        assert torch.equal(got, call(c))


@pytest.mark.parametrize("S, hq, heads", [(17, 1, 1), (16, 8, 4), (64, 2, 2), (65, 1, 1), (32, 16, 4), (129, 3, 3)])
@pytest.mark.parametrize("D, Dv, gk, gv, page", [(128, 128, 32, 32, 16), (128, 128, 128, 64, 24), (64, 64, 64, 64, 7), (64, 64, 32, 32, 48),
                                                 (96, 128, 96, 32, 16), (128, 64, 64, 64, 5), (256, 192, 256, 64, 16)])
def test_rows_of_a_prompt(S, hq, heads, D, Dv, gk, gv, page):
    """One token more or less than a tile's, a page's and a block's rows; empty
    sequences; tokens that were there before the prompt."""
    for dtype, lengths in (("bf16", [S, 0, S + 1, 200]), ("f16", [63 + S, 1, 330, S - 1])):
        c = inputs(lengths, S, hq, heads, D, Dv, gk, gv, page, dtype, seed=35)
        counts = torch.tensor([S, S, S - 1, (S + 1) // 2], dtype=torch.int32)
        check(call(c, counts=counts), c, counts=counts, what=f"{dtype} causal")
        check(call(c, causal=False), c, causal=False, what=dtype)


@pytest.mark.parametrize("S, hq, heads, D", [(1, 8, 4, 128), (1, 8, 4, 64), (6, 8, 2, 128), (70, 4, 2, 128)])
def test_two_graphs_share_a_workspace(S, hq, heads, D):
    """Two captured calls that split the same sequences and use one workspace,
    replayed in turn, with the program's own work between them."""
    c = [inputs([900, 333, 70], S, hq, heads, D, D, D, D, 16, "bf16", seed=s) for s in (36, 37)]
    ws = torch.empty(rp.rope_cache_attention_workspace(3, S, hq, heads, D), dtype=torch.uint8, device="cuda")
    args, outs, graphs = [], [], []
    for one in c:
        caches = [rp.RopeCache(one[n][0].cuda(), one[n][1].cuda()) for n in ("k", "v")]
        args.append((one["q"].cuda(), *caches, one["table"].cuda(), one["lengths"].cuda()))
        outs.append(one["out"].cuda())
        rp.rope_cache_attention(*args[-1], out=outs[-1], workspace=ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            rp.rope_cache_attention(*args[-1], out=outs[-1], workspace=ws)
    for i in range(4):
        for a, o, g in zip(args, outs, graphs):
            a[0].mul_(-0.9)
            o.fill_(7.0)
            g.replay()
            assert torch.equal(o, rp.rope_cache_attention(*a)), i


def test_the_same_sequence_twice_and_pages_shared():
    """Rows of the table that name the same pages: sequences with a common
    start, and one sequence asked about twice."""
    c = inputs([400, 400, 380], 1, 8, 4, 128, 128, 128, 128, 16, "bf16", seed=38)
    c["table"][1] = c["table"][0]
    c["table"][2, :20] = c["table"][0, :20]
    c["q"][1] = c["q"][0]
    got = call(c)
    check(got, c)
    assert torch.equal(got[0], got[1])


@pytest.mark.parametrize("B, heads, S", [(2, 4, 1), (3, 1, 5), (65, 4, 1), (70, 2, 2), (130, 1, 1), (500, 1, 1), (900, 1, 1), (300, 4, 1)])
@pytest.mark.parametrize("D, dtype", [(64, "bf16"), (80, "f32")])
def test_sequences_of_all_lengths_are_split_alike(B, heads, S, D, dtype):
    """One long sequence among short and empty ones, the long one at each end
    and in the middle; a workspace of NaN of exactly the bytes asked for."""
    for where in (0, B // 2, B - 1):
        lengths = [(7 * b) % 41 for b in range(B)]
        lengths[where] = 3000 if B < 100 else 700
        c = inputs(lengths, S, 2 * heads, heads, D, D, D, D, 16, dtype, seed=39, cols=-(-lengths[where] // 16))
        counts = torch.tensor([S if b == where or b % 3 else 0 for b in range(B)], dtype=torch.int32)
        ws = torch.full((max(1, rp.rope_cache_attention_workspace(B, S, 2 * heads, heads, D)),), 255, dtype=torch.uint8, device="cuda")
        got = call(c, counts=counts, workspace=ws)
        check(got, c, counts=counts)
        none = counts == 0
        assert torch.equal(got.cpu()[none], c["out"][none])


@pytest.mark.parametrize("lengths", [[0, 0, 0], [5000, 5000, 5000], [1, 8000, 1], [64, 128, 192], [8191, 63, 4097]])
@pytest.mark.parametrize("S, heads, D", [(1, 4, 128), (3, 2, 64), (40, 1, 128)])
def test_parts_of_equal_tokens(lengths, S, heads, D):
    c = inputs(lengths, S, 2 * heads, heads, D, D, D, D, 16, "f16", seed=40, cols=512)
    check(call(c), c)
    check(call(c, causal=False), c, causal=False)


@pytest.mark.parametrize("S, hq, heads, D, gv, dtype", [(3, 8, 4, 128, 128, "bf16"), (3, 4, 2, 64, 64, "f16"), (9, 16, 4, 128, 32, "bf16"),
                                                        (40, 4, 2, 128, 128, "f16"), (3, 4, 2, 256, 64, "bf16"), (3, 4, 2, 80, 80, "bf16"),
                                                        (3, 4, 2, 64, 64, "f32")])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["k", "v"])
def test_scales_that_are_no_numbers_stay_with_those_who_see_them(S, hq, heads, D, gv, dtype, value, which):
    """The newest token's scales: rows before it neither see it nor change."""
    c = inputs([S, 200, 130], S, hq, heads, D, D, D, gv, 16, dtype, seed=41)
    want = call(c)
    for b, n in enumerate(c["lengths"].tolist()):
        c[which][1][c["table"][b, (n - 1) // 16], (n - 1) % 16] = value
    got = call(c)
    assert torch.equal(got[:, :-1], want[:, :-1])
    last = got[:, -1].float()
    if which == "v" or value != value:
        assert not bool(torch.isfinite(last).any())


@pytest.mark.parametrize("D, Dv, gk, gv", [(64, 64, 16, 16), (128, 128, 16, 128), (128, 64, 128, 16), (128, 128, 64, 16), (96, 96, 48, 16),
                                           (80, 80, 80, 16), (80, 128, 16, 32), (256, 256, 16, 16), (192, 80, 48, 80)])
@pytest.mark.parametrize("S, hq, heads, page", [(1, 4, 1, 16), (1, 8, 4, 24), (5, 12, 2, 16), (20, 4, 1, 7), (70, 4, 4, 16)])
def test_groups_of_16_lanes(D, Dv, gk, gv, S, hq, heads, page):
    lengths = [S, 0, 200 + S, 77]
    counts = torch.tensor([S, S, S, (S + 1) // 2], dtype=torch.int32)
    for dtype, span in (("bf16", 0.5), ("f16", 3.0)):
        c = inputs(lengths, S, hq, heads, D, Dv, gk, gv, page, dtype, seed=42, span=span)
        if dtype == "f16":      # values that the type holds
            c["v"] = (c["v"][0], c["v"][1].clamp(max=1000.0))
        c["k"] = (c["k"][0], c["k"][1].clamp(max=4.0))
        check(call(c, counts=counts), c, counts=counts, what=dtype)
    c = inputs([500, 333], S, hq, heads, D, Dv, gk, gv, page, "bf16", seed=43, span=12.0)
    c["k"] = (c["k"][0], c["k"][1].clamp(max=4.0))
    check(call(c, causal=False), c, causal=False, what="far apart")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gk, gv", [(16, None), (None, 16), (16, 16), (32, None), (32, 16), (16, 32), (64, 16), (32, 32)])
@pytest.mark.parametrize("S, hq, heads, page", [(1, 4, 4, 16), (3, 16, 8, 48), (9, 8, 4, 64), (40, 4, 4, 16), (100, 8, 4, 32)])
def test_four_heads_groups_of_lanes(D, gk, gv, S, hq, heads, page):
    gk, gv = gk or D, gv or D
    lengths = [S, 0, 300 + S, 65]
    counts = torch.tensor([S, S, S, (S + 1) // 2], dtype=torch.int32)
    for dtype, span in (("bf16", 3.0), ("f16", 0.5)):
        c = inputs(lengths, S, hq, heads, D, D, gk, gv, page, dtype, seed=44, span=span)
        c["k"] = (c["k"][0], c["k"][1].clamp(max=4.0))
        got = call(c, counts=counts)
        check(got, c, counts=counts, what=dtype)
        for b, n in enumerate(counts.tolist()):
            assert torch.equal(got[b, n:].cpu(), c["out"][b, n:])
    c = inputs([500, 333], S, hq, heads, D, D, gk, gv, page, "bf16", seed=45, span=12.0)
    c["k"] = (c["k"][0], c["k"][1].clamp(max=4.0))
    check(call(c, causal=False), c, causal=False, what="far apart")
