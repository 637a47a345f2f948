"""The projection with adapters at sizes that its tiled kernels take (more
than 64 tokens and 640 blocks of 64 tokens by 32 output lanes), on the GPU,
against its definition in 64 bits."""
import pytest
import torch

import transformer_positional_encoding_amd as rp
from axes_refs import TORCH
from test_lora_gpu import check, make, run, tables

pytestmark = pytest.mark.gpu

# (M, K, H, Dh, R, A, slice, mode): square tiles with each epilogue, tiles of
# 128 and 192 lanes, heads over several tiles, rotation groups across tiles
CASES = [
    (1300, 256, 16, 128, 32, 3, (0, 128), "rotate_half"),
    (300, 256, 64, 192, 16, 6, (0, 64), "interleave"),
    (130, 128, 64, 128, 40, 11, (3, 61), "interleave"),
    (96, 256, 128, 192, 128, 9, (0, 64), "interleave"),
    (2500, 256, 16, 64, 72, 5, (0, 64), 8),
    (700, 192, 40, 96, 8, 5, (0, 96), "rotate_half"),
    (520, 192, 40, 64, 24, 70, (0, 64), "interleave"),
    (1500, 192, 4, 576, 16, 3, (512, 576), "interleave"),
    (1500, 128, 4, 576, 16, 3, (512, 576), "interleave"),
    (17000, 64, 4, 32, 8, 4, (0, 32), "rotate_half"),
    (1025, 384, 4, 1024, 16, 4, (0, 1024), "rotate_half"),
    (1025, 384, 4, 1024, 16, 4, None, "interleave"),
]


@pytest.mark.parametrize("M, K, H, Dh, R, A, sl, mode", CASES)
@pytest.mark.parametrize("dtype, out, table", [("bf16", "bf16", "bf16"), ("f16", "f16", "f32"), ("bf16", "f32", "f32"),
                                               ("f16", "f32", "f16")])
@pytest.mark.parametrize("ids", ["runs", "mixed", "one", "none"])
def test_against_64_bits(M, K, H, Dh, R, A, sl, mode, dtype, out, table, ids):
    c = make(M, K, H, Dh, R, A, dtype, seed=M + K, ids=ids)
    at = sl or (0, 0)
    cos, sin = tables(M, at[1] - at[0], mode, table, 5)
    check(run(c, cos, sin, H, mode, sl, out), c, cos, sin, H, mode, at, out, "projection")


@pytest.mark.parametrize("K", [128, 192])
def test_tables_per_batch_and_per_head(K):
    B, S, H = 2, 300, 40
    M = B * S
    c = make(M, K, H, 64, 16, 3, "bf16", seed=4, ids="mixed")
    g = torch.Generator(device="cuda").manual_seed(9)
    for heads in (H, 1):
        cos, sin = (torch.randn(B, S, heads, 64, generator=g, device="cuda") for _ in range(2))
        got = rp.rope_proj_lora_fwd(c["x"].view(B, S, K), c["w"], c["a"], c["b"], c["ids"].view(B, S), cos, sin, H,
                                    "rotate_half", (0, 64), scales=c["scales"])
        flat = lambda t: t.reshape(1, M, -1, 64)  # noqa: E731
        check(flat(got), c, flat(cos), flat(sin), H, "rotate_half", (0, 64), "bf16", f"tables of {heads} heads")


@pytest.mark.parametrize("K", [128, 192])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_large_products_and_not_finite_tokens_and_adapters(K, dtype):
    """h past the largest fp16 value; rows of infinities in x and adapters of
    NaNs stay with their tokens."""
    M, H = 600, 40
    c = make(M, K, H, 64, 16, 3, dtype, seed=8, ids="mixed")
    c["x"] = (c["x"].float() * 200).to(TORCH[dtype])
    c["a"] = (c["a"].float() * 300).to(TORCH[dtype])
    c["b"] = (c["b"].float() * 2.0 ** -8).to(TORCH[dtype])
    cos, sin = tables(M, 64, "interleave", "f32", 2)
    clean = run(c, cos, sin, H, "interleave", (0, 64), "f32")
    check(clean, c, cos, sin, H, "interleave", (0, 64), "f32", "large h")
    c["x"][0, 1] = float("inf")
    c["a"][2], c["b"][2] = float("nan"), float("inf")
    got = run(c, cos, sin, H, "interleave", (0, 64), "f32")
    keep = (torch.arange(M, device="cuda") != 1) & (c["ids"] != 2)
    assert torch.equal(got[:, keep], clean[:, keep]) and not bool(torch.isfinite(got[:, ~keep]).any())


@pytest.mark.parametrize("M, K", [(513, 128), (700, 192)])
def test_nothing_past_the_result_is_written(M, K):
    H = 40
    c = make(M, K, H, 64, 8, 2, "bf16", seed=2, ids="mixed")
    cos, sin = tables(M, 64, "interleave", "bf16", 2)
    n = M * H * 64
    guarded = torch.full((n + 8192,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guarded[4096:4096 + n].view(1, M, H, 64)
    size = rp.rope_proj_lora_workspace(M, K, 8)
    ws = torch.full((size + 64,), 9, dtype=torch.uint8, device="cuda")
    run(c, cos, sin, H, "interleave", (0, 64), "bf16", out=out, workspace=ws[:size])
    assert bool((guarded[:4096] == 7).all()) and bool((guarded[4096 + n:] == 7).all()) and bool((ws[-64:] == 9).all())
    assert torch.equal(out, run(c, cos, sin, H, "interleave", (0, 64), "bf16")), "two runs differ"


@pytest.mark.parametrize("K", [128, 192])
def test_graph_replays_follow_the_adapters(K):
    M, H = 300, 20
    c = make(M, K, H, 128, 16, 5, "bf16", seed=2, ids="mixed")
    cos, sin = tables(M, 128, "rotate_half", "bf16", 2)
    run(c, cos, sin, H, "rotate_half", (0, 128), "bf16")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(c, cos, sin, H, "rotate_half", (0, 128), "bf16")
    for k in range(4):
        c["ids"].copy_(torch.roll(c["ids"], 1 + k))
        c["x"].mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, run(c, cos, sin, H, "rotate_half", (0, 128), "bf16"))


def test_two_streams_at_once():
    cs = [make(400, 512, 24, 128, 16, 5, "bf16", seed=k, ids="mixed") for k in range(2)]
    cos, sin = tables(400, 128, "rotate_half", "bf16", 2)
    want = [run(c, cos, sin, 24, "rotate_half", (0, 128), "bf16") for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        got = [run(c, cos, sin, 24, "rotate_half", (0, 128), "bf16", stream=s) for c, s in zip(cs, streams)]
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
