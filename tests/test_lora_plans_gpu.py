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


@pytest.mark.parametrize("K, kernel", [(128, "square"), (192, "heads")])
def test_tiles_with_tables_per_batch_and_per_head(K, kernel):
    B, S, H = 2, 700, 40
    M = B * S
    c = make(M, K, H, 64, 16, 3, "bf16", seed=4, ids="mixed")
    assert plan(c, H, (0, 64), "rotate_half") == (kernel, True)
    g = torch.Generator(device="cuda").manual_seed(9)
    for heads in (H, 1):
        cos, sin = (torch.randn(B, S, heads, 64, generator=g, device="cuda") for _ in range(2))
        got = rp.rope_proj_lora_fwd(c["x"].view(B, S, K), c["w"], c["a"], c["b"], c["ids"].view(B, S), cos, sin, H,
                                    "rotate_half", (0, 64), scales=c["scales"])
        flat = lambda t: t.reshape(1, M, -1, 64)  # noqa: E731
        check(flat(got), c, flat(cos), flat(sin), H, "rotate_half", (0, 64), "bf16", f"tables of {heads} heads")


@pytest.mark.parametrize("K, kernel", [(128, "square"), (192, "heads")])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_tiles_keep_what_is_not_finite_with_its_tokens(K, kernel, dtype):
    M, H = 1400, 40
    c = make(M, K, H, 64, 16, 3, dtype, seed=8, ids="mixed")
    assert plan(c, H, (0, 64), "interleave", torch.float32, 0) == (kernel, True)
    cos, sin = tables(M, 64, "interleave", "f32", 2)
    clean = run(c, cos, sin, H, "interleave", (0, 64), "f32")
    check(clean, c, cos, sin, H, "interleave", (0, 64), "f32", "before")
    c["x"][0, 1] = float("inf")
    c["a"][2], c["b"][2] = float("nan"), float("inf")
    got = run(c, cos, sin, H, "interleave", (0, 64), "f32")
    keep = (torch.arange(M, device="cuda") != 1) & (c["ids"] != 2)
    assert torch.equal(got[:, keep], clean[:, keep]) and not bool(torch.isfinite(got[:, ~keep]).any())


@pytest.mark.parametrize("M, K, kernel", [(1313, 128, "square"), (1400, 192, "heads")])
def test_tiles_write_nothing_past_the_result(M, K, kernel):
    H = 40
    c = make(M, K, H, 64, 8, 2, "bf16", seed=2, ids="mixed")
    assert plan(c, H, (0, 64), "interleave") == (kernel, True)
    cos, sin = tables(M, 64, "interleave", "bf16", 2)
    n = M * H * 64
    guarded = torch.full((n + 8192,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guarded[4096:4096 + n].view(1, M, H, 64)
    size = rp.rope_proj_lora_workspace(M, K, 8)
    ws = torch.full((size + 64,), 9, dtype=torch.uint8, device="cuda")
    run(c, cos, sin, H, "interleave", (0, 64), "bf16", out=out, workspace=ws[:size])
    assert bool((guarded[:4096] == 7).all()) and bool((guarded[4096 + n:] == 7).all()) and bool((ws[-64:] == 9).all())


@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("A, ids", [(70, "runs"), (70, "mixed"), (1023, "mixed"), (1, "none")])
def test_tiles_of_many_adapters(A, ids, dtype, out):
    M, H, K = 1300, 24, 192
    c = make(M, K, H, 96, 24, A, dtype, seed=A, ids=ids)
    assert plan(c, H, (0, 96), "rotate_half", torch.float32, rp.DTYPE_CODES[out]) == ("heads", True)
    cos, sin = tables(M, 96, "rotate_half", "f32", 6)
    check(run(c, cos, sin, H, "rotate_half", (0, 96), out), c, cos, sin, H, "rotate_half", (0, 96), out, f"{A} adapters")
