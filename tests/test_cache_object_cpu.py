"""A RopeCache describes the tensors it was made of, for as long as it lives."""
import pytest
import torch

import transformer_positional_encoding_amd as rp


def test_its_tensors_cannot_be_exchanged():
    """Another tensor put in the place of data would leave the address of the
    old one, whose memory may be gone, to the kernels."""
    c = rp.rope_cache(2, 3, 4, 32, "int8", 8, device="cpu")
    data, scales = c.data, c.scales
    for name, value in (("data", data.clone()), ("scales", scales.clone()), ("scales", None), ("device", "cuda"),
                        ("words", None), ("tensors", ())):
        with pytest.raises(AttributeError, match="RopeCache"):
            setattr(c, name, value)
        with pytest.raises(AttributeError, match="RopeCache"):
            delattr(c, name)
    assert c.data is data and c.scales is scales
    assert (c.struct.data, c.struct.scales) == (data.data_ptr(), scales.data_ptr())
