"""No call of the cache reaches a launch with tensors in host memory."""
import pytest
import torch

import transformer_positional_encoding_amd as rp

BF = torch.bfloat16
SLOTS = torch.zeros(2, 3, dtype=torch.int64)
TURN = (torch.zeros(2, 3, dtype=torch.int64), torch.ones(8, dtype=torch.float64), "interleave", (0, 16))


def rows(heads):
    return torch.ones(2, 3, heads, 16, dtype=BF)


def cache(heads):
    return rp.RopeCache(torch.zeros(3, 4, heads, 16, dtype=BF))


def test_q_beside_keys_without_heads():
    with pytest.raises(ValueError, match="q must be a GPU tensor"):
        rp.rope_cache_write(rows(0), None, cache(0), None, SLOTS, *TURN, q=rows(2))


def test_v_beside_keys_without_heads():
    with pytest.raises(ValueError, match="v must be a GPU tensor"):
        rp.rope_cache_write(rows(0), rows(2), cache(0), cache(2), SLOTS)


def test_nothing_at_all():
    rp.rope_cache_write(rows(0), rows(0), cache(0), cache(0), SLOTS, *TURN, q=rows(0))
