"""What autograd is told of calls that it does not record: in-place changes move
the version counter of what they change, and tensors that need a gradient are
refused where none is given. On the CPU, with the library's calls left out."""
import pytest
import torch

import transformer_positional_encoding_amd as rp

B, S, N, D = 2, 3, 2, 8


@pytest.fixture
def no_library(monkeypatch):
    """The bindings run to their launch, which does nothing."""
    class Library:
        def __getattr__(self, name):
            return lambda *a: rp.ROPE_OK

    monkeypatch.setattr(rp, "library", Library)
    for name in ("_call", "_call_pos"):
        monkeypatch.setattr(rp, name, lambda *a, **k: None)


def test_unrecorded_rotations_in_place_are_seen(no_library):
    """A value that another operation's backward needs, changed by an
    unrecorded call: that backward raises, as for torch's own operations."""
    w = torch.randn(B, S, N, D, requires_grad=True)
    pos, f = torch.zeros(3, B, S, dtype=torch.int64), torch.ones(4, dtype=torch.float64)
    t = torch.ones(B, S, 1, D)
    calls = [lambda x: rp.inplace_partial_rotary_mul(x, t, t, "interleave", (0, 8)),
             lambda x: rp.inplace_partial_rotary_mul_pos(x, pos[0], f, "interleave", (0, 8)),
             lambda x: rp.inplace_partial_rotary_mul_axes(x, pos, f, (0, 1, 2, 0), "interleave", (0, 8))]
    for rotate in calls:
        for x in (torch.randn(B, S, N, D), w * 2.0):
            y = w * x                       # saves x
            with torch.no_grad():
                rotate(x)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.sum().backward()
        with torch.inference_mode():
            rotate(torch.zeros(B, S, N, D))
