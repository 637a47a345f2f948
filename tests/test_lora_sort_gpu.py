"""The rows that the tiled projection with adapters works on, as its sort leaves
them in the workspace (behind h: the rows' tokens, the adapter of every 32,
their number), against the order by definition."""
import pytest
import torch

import transformer_positional_encoding_amd as rp

pytestmark = pytest.mark.gpu
RANK, K, H, DH = 8, 64, 8, 64


def want(ids, count):
    """(tokens by row, adapter by 32 rows): adapters ascending, those without
    one last, tokens in their own order, each adapter filled up to 32."""
    key = torch.where((ids >= 0) & (ids < count), ids, torch.full_like(ids, count))
    rows, groups = [], []
    for k in range(count + 1):
        at = torch.nonzero(key == k)[:, 0].tolist()
        if at:
            at += [-1] * (-len(at) % 32)
            rows += at
            groups += [k if k < count else -1] * (len(at) // 32)
    return torch.tensor(rows, dtype=torch.int32), torch.tensor(groups, dtype=torch.int32)


@pytest.mark.parametrize("M, count", [(5200, 1), (5200, 7), (5247, 1023), (16384, 3), (16385, 64), (40001, 5), (70000, 1023)])
@pytest.mark.parametrize("ids", ["mixed", "one", "turns", "none", "late"])
def test_order(M, count, ids):
    g = torch.Generator().manual_seed(M + count)
    t = torch.arange(M)
    a = {"mixed": torch.randint(-2, count + 2, (M,), generator=g), "one": torch.full((M,), count - 1), "turns": t % count,
         "none": torch.full((M,), -7), "late": torch.where(t > M - 3, 0, -1)}[ids].to(torch.int32)
    bf = torch.bfloat16
    x, w = torch.zeros(M, K, dtype=bf, device="cuda"), torch.zeros(H * DH, K, dtype=bf, device="cuda")
    la, lb = torch.zeros(count, RANK, K, dtype=bf, device="cuda"), torch.zeros(count, H * DH, RANK, dtype=bf, device="cuda")
    none = torch.zeros(1, 1, 1, 0, device="cuda")
    ws = torch.full((rp.rope_proj_lora_workspace(M, K, RANK),), 0x55, dtype=torch.uint8, device="cuda")
    rows, groups = want(a, count)
    st, plan = rp.raw_proj_lora_launch_info(2, 2, (1, M, H, DH), K, count, RANK, None, (1, 1, 1, 0), (0, 0, 0, 1), None,
                                            (1, 1, 1, 0), (0, 0, 0, 1), 2, 1, None)
    assert st == rp.ROPE_OK and plan["sorted"]
    places = M + 31 * min(count + 1, M) + 384
    for _ in range(3):
        rp.rope_proj_lora_fwd(x, w, la, lb, a.cuda(), none, none, H, workspace=ws)
        words = ws.cpu().view(torch.int32)[M * RANK:]
        assert int(words[places + places // 32 + 1]) == len(rows)
        assert torch.equal(words[:len(rows)], rows) and bool((words[len(rows):len(rows) + 384] == -1).all())
        got = words[places:]
        assert torch.equal(got[:len(groups)], groups) and bool((got[len(groups):len(groups) + 12] == -1).all())
        ws.fill_(0x55)
