"""The launch plan of the projection with adapters (no GPU)."""
import pytest

import transformer_positional_encoding_amd as rp


def plan(M, K, H, Dh, R=16, A=8, sl=(0, 0), mode=1, ydt=2, r=1 << 20):
    L = sl[1] - sl[0]
    t = ((1, M, 1, L), (M * L, L, L, 1))
    return rp.raw_proj_lora_launch_info(ydt, 2, (1, M, H, Dh), K, A, R, r, *t, r, *t, 2, mode, sl)


def test_kernels_and_their_shapes():
    for M, tokens in ((1, 16), (17, 32), (33, 64), (64, 64)):
        assert plan(M, 1536, 128, 192, sl=(0, 64))[1] == dict(
            kernel="few", blocks=768, threads=256, tile_tokens=tokens, tile_lanes=32, epilogue=None, tables_in_lds=False,
            sorted=False)
    got = plan(8190, 1536, 128, 192, sl=(0, 64))[1]
    # 9 bins leave at most 31 rows open each
    assert got == dict(kernel="square", blocks=-(-(8190 + 9 * 31) // 256) * 96, threads=256, tile_tokens=256, tile_lanes=256,
                       epilogue="vector", tables_in_lds=True, sorted=True)
    assert plan(8190, 1536, 128, 192, A=0, sl=(0, 64))[1]["sorted"] is False
    assert plan(8190, 192, 128, 96, sl=(0, 96), mode=0)[1]["kernel"] == "heads"
    # more adapters than a sort takes; rotation groups that no tile holds
    assert plan(8190, 1536, 128, 192, A=1024, sl=(0, 64))[1]["kernel"] == "few"
    assert plan(8190, 1536, 4, 576, sl=(3, 575), mode=0)[1]["kernel"] == "general"
    assert plan(0, 1536, 128, 192)[1]["kernel"] == "none"


@pytest.mark.parametrize("change, status, text", [
    (dict(R=12), rp.ROPE_ERR_INVALID, "multiple of 8"), (dict(R=136), rp.ROPE_ERR_UNSUPPORTED, "128"),
    (dict(A=-1), rp.ROPE_ERR_INVALID, "negative"), (dict(K=96), rp.ROPE_ERR_UNSUPPORTED, "multiple of 64"),
    (dict(sl=(0, 64), r=None), rp.ROPE_ERR_NULLPTR, "r1"), (dict(Dh=40), rp.ROPE_ERR_UNSUPPORTED, "head"),
])
def test_refusals(change, status, text):
    st, got = plan(**dict(dict(M=100, K=128, H=2, Dh=64), **change))
    assert (st, got) == (status, None) and text in rp.last_error()


def test_null_info():
    L = rp.library()
    assert L.rope_proj_lora_launch_info(2, 2, None, 0, 0, 0, None, None, None, None, None, None, 2, 1, None,
                                        None) == rp.ROPE_ERR_NULLPTR


@pytest.mark.parametrize("M, K, N, R, few", [
    (6000, 2048, 192, 8, True), (6000, 2048, 192, 16, False), (6000, 2048, 192, 128, False), (1280, 1536, 192, 128, True),
    (2560, 1536, 192, 128, False), (640, 1536, 576, 128, True), (1280, 1536, 576, 128, False), (2560, 512, 576, 8, True),
    (640, 1536, 2048, 8, True), (640, 1536, 2048, 32, True), (640, 1536, 2048, 128, False), (1280, 1536, 2048, 8, False),
    (160, 4096, 5120, 128, True), (320, 4096, 5120, 128, False), (64, 1536, 24576, 128, True), (65, 1536, 24576, 8, False),
])
def test_rank_and_tokens_decide_for_tiles(M, K, N, R, few):
    """The kernel that was measured to be the faster one at these sizes."""
    assert plan(M, K, N // 64, 64, R=R, sl=(0, 64))[1]["kernel"] == ("few" if few else "square")
