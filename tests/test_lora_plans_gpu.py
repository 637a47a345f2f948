"""The projection with adapters where its kernel is what the test is about: the
plan is asked first, so that a moved threshold shows."""
import pytest
import torch

import transformer_positional_encoding_amd as rp
from test_lora_gpu import check, make, run, tables

pytestmark = pytest.mark.gpu


def plan(c, H, sl, mode, table=torch.bfloat16, out=None):
    M, K = c["x"].shape[1:]
    L = sl[1] - sl[0]
    code = rp._dtype_code(c["x"])
    t = ((1, M, 1, L), (M * L, L, L, 1))
    st, got = rp.raw_proj_lora_launch_info(code if out is None else out, code, (1, M, H, c["w"].shape[0] // H), K,
                                           *c["a"].shape[:2], 4096, *t, 4096, *t,
                                           rp._dtype_code(torch.empty(0, dtype=table)), rp.MODES.get(mode, mode), sl)
    assert st == rp.ROPE_OK, rp.last_error()
    return got["kernel"], got["sorted"]


@pytest.mark.parametrize("M, K, H, Dh, kernel", [(1300, 256, 40, 128, "square"), (600, 192, 128, 96, "heads"),
                                                 (700, 192, 40, 128, "heads")])
def test_replays_of_tiles_follow_the_adapters(M, K, H, Dh, kernel):
    """Sort, order, groups and row count of each replay's own adapters: the
    number of tiles in use changes under a captured grid."""
    sl = (0, Dh)
    c = make(M, K, H, Dh, 16, 9, "bf16", seed=2, ids="mixed")
    assert plan(c, H, sl, "rotate_half") == (kernel, True)
    cos, sin = tables(M, Dh, "rotate_half", "bf16", 2)
    run(c, cos, sin, H, "rotate_half", sl, "bf16")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(c, cos, sin, H, "rotate_half", sl, "bf16")
    t = torch.arange(M, device="cuda")
    for ids in (torch.zeros_like(t), t % 9, t // 700, torch.full_like(t, -1), 8 - t % 9, torch.where(t == M - 1, 3, 11)):
        c["ids"].copy_(ids)
        c["x"].mul_(-0.5)
        y.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, run(c, cos, sin, H, "rotate_half", sl, "bf16"))
    check(y, c, cos, sin, H, "rotate_half", sl, "bf16", "the last replay")


def test_one_workspace_in_turn_of_tiles_and_few_tokens():
    """Calls behind each other on a stream, each sorting into, or past, what
    the one before left."""
    H, Dh, K, R = 64, 128, 128, 16
    ws = torch.empty(rp.rope_proj_lora_workspace(3000, K, R), dtype=torch.uint8, device="cuda").fill_(0x7f)
    kernels = []
    for seed, M in enumerate((3000, 5, 700, 64, 300, 1, 3000, 257)):
        c = make(M, K, H, Dh, R, 7, "bf16", seed=seed, ids="mixed")
        cos, sin = tables(M, Dh, "rotate_half", "bf16", 2)
        kernels.append(plan(c, H, (0, Dh), "rotate_half"))
        got = run(c, cos, sin, H, "rotate_half", (0, Dh), "bf16", workspace=ws)
        check(got, c, cos, sin, H, "rotate_half", (0, Dh), "bf16", f"{M} tokens")
    few, tiles = ("few", False), ("square", True)
    assert kernels == [tiles, few, tiles, few, tiles, few, tiles, tiles]


@pytest.mark.parametrize("M, K, H, Dh, sl", [(1600, 192, 20, 64, (0, 64)), (6500, 192, 1, 576, (512, 576)),
                                             (3300, 192, 2, 576, (512, 576)), (21000, 64, 4, 32, (0, 32))])
@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("f16", "f32")])
def test_tiles_of_whole_heads_and_of_parts(M, K, H, Dh, sl, dtype, out):
    """Tiles of 128 and of 192 lanes, heads over several tiles, more tokens
    than the sort holds in registers."""
    c = make(M, K, H, Dh, 24, 5, dtype, seed=M, ids="mixed")
    assert plan(c, H, sl, "interleave", torch.float32, rp.DTYPE_CODES[out]) == ("heads", True)
    cos, sin = tables(M, sl[1] - sl[0], "interleave", "f32", 6)
    check(run(c, cos, sin, H, "interleave", sl, out), c, cos, sin, H, "interleave", sl, out, "tiles")
