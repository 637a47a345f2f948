"""rope_proj_lora_fwd refuses buffers that share memory with what it writes: y,
and the workspace, which is written before the inputs are read (no GPU)."""
import pytest

import transformer_positional_encoding_amd as rp
from test_lora_cpu import BAD, FAKE, call

# bytes of the call's buffers: y and x 6 tokens, w 128 x 128, 3 adapters of rank 16
Y, X, W, A, B = 6 * 128 * 2, 6 * 128 * 2, 128 * 128 * 2, 3 * 16 * 128 * 2, 3 * 128 * 16 * 2
IDS, SCALES, TABLE, WS = 6 * 4, 3 * 4, 6 * 64 * 2, 6 * 16 * 4
AT = dict(y=FAKE, x=FAKE * 2, w=FAKE * 3, la=FAKE * 4, lb=FAKE * 5, ids=FAKE * 6, scales=FAKE * 9, r=FAKE * 7, ws=FAKE * 8)
SIZE = dict(y=Y, x=X, w=W, la=A, lb=B, ids=IDS, scales=SCALES, r=TABLE, ws=WS)
NAME = dict(y="y", x="x", w="w", la="lora a", lb="lora b", ids="lora adapters", scales="lora scales", r="a table", ws="workspace")


OTHERS = ("la", "lb", "ids", "scales", "r")


@pytest.mark.parametrize("written, other", [("y", o) for o in OTHERS + ("ws",)] + [("ws", o) for o in OTHERS + ("x", "w")])
def test_overlaps_are_refused(written, other):
    """The other buffer's last bytes are the written one's first, its first
    the written one's last, and both begin together."""
    unit = 4 if other in ("ids", "scales") else 16      # what its address is aligned to
    for at in (AT[written] - SIZE[other] + unit, AT[written] + SIZE[written] - unit, AT[written]):
        assert call(**{"scales": AT["scales"], other: at}) == BAD, (hex(at), rp.last_error())
        assert f"{NAME[written]} overlaps {NAME[other]}" in rp.last_error()


def test_memory_behind_the_bytes_in_use_is_free():
    """A workspace larger than needed overlaps with its needed bytes only."""
    assert call(ws=FAKE * 8, wsb=1 << 30, la=FAKE * 8 + WS, x=FAKE * 8 + WS + A, mode=7, scales=FAKE * 9) == BAD
    assert "mode" in rp.last_error()
    st = call(ws=FAKE * 8, wsb=1 << 30, la=FAKE * 8 + WS, r=None, scales=FAKE * 9)
    assert st == rp.ROPE_ERR_NULLPTR and "r1" in rp.last_error()


def test_without_adapters_their_buffers_are_not_looked_at():
    st = call(count=0, la=FAKE, lb=FAKE, ids=FAKE, ws=FAKE, r=None)
    assert st == rp.ROPE_ERR_NULLPTR and "r1" in rp.last_error()
