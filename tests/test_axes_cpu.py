"""Positions on several axes: the helpers that order pairs and frequencies,
and every refusal of the entry points (no GPU: nothing is launched)."""
import pytest
import torch

import transformer_positional_encoding_amd as rp

FAKE = 1 << 20   # a device address that no check dereferences
SHAPE = (2, 5, 3, 16)
OK = dict(pos_shape=(3, 2, 5), pos_strides=(10, 5, 1), pair_axes=(0, 1, 2, 0))


def call(**kw):
    a = dict(direction="fwd", x_ptr=FAKE, x_shape=SHAPE, dtype=2, pos_ptr=FAKE, inv_freq_ptr=FAKE, table_dtype=2, mode=1,
             partial_slice=(4, 12), **OK)
    a.update(kw)
    return rp.raw_axes_call(**a)


def test_pair_axes_in_blocks_and_dealt():
    assert rp.rope_pair_axes((2, 1, 3)) == (0, 0, 1, 2, 2, 2)
    assert rp.rope_pair_axes((3, 2, 1), dealt=True) == (0, 1, 2, 0, 1, 0)
    assert rp.rope_pair_axes((24, 20, 20), dealt=True)[57:] == (0, 1, 2, 0, 0, 0, 0)
    assert rp.rope_pair_axes((0, 2), dealt=True) == (1, 1)
    for bad in ((), (1, 1, 1, 1, 1), (2, -1)):
        with pytest.raises(ValueError):
            rp.rope_pair_axes(bad)


def test_frequencies_of_axes_that_count_their_own_pairs():
    f = rp.rope_axes_inv_freq((0, 1, 0, 1, 1), 100.0)
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 1.0, 0.1, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)], dtype=torch.float64),
                          rtol=1e-15)


@pytest.mark.parametrize("change, status, text", [
    (dict(pos_ptr=None), rp.ROPE_ERR_NULLPTR, "positions"),
    (dict(inv_freq_ptr=None), rp.ROPE_ERR_NULLPTR, "inv_freq"),
    (dict(pos_shape=None), rp.ROPE_ERR_NULLPTR, "shape"),
    (dict(pair_axes=None), rp.ROPE_ERR_NULLPTR, "pair_axes"),
    (dict(x_ptr=None), rp.ROPE_ERR_NULLPTR, "x is NULL"),
    (dict(pos_shape=(0, 2, 5)), rp.ROPE_ERR_INVALID, "dimension A"),
    (dict(pos_shape=(5, 2, 5)), rp.ROPE_ERR_INVALID, "dimension A"),
    (dict(pos_shape=(3, 3, 5)), rp.ROPE_ERR_INVALID, "dimension B"),
    (dict(pos_shape=(3, 2, 4)), rp.ROPE_ERR_INVALID, "dimension S"),
    (dict(pos_strides=(-1, 5, 1)), rp.ROPE_ERR_INVALID, "negative"),
    (dict(pos_strides=(10, -5, 1)), rp.ROPE_ERR_INVALID, "negative"),
    (dict(pos_strides=(1 << 62, 1 << 62, 1)), rp.ROPE_ERR_INVALID, "64-bit"),
    (dict(pair_axes=(0, 1, 3, 0)), rp.ROPE_ERR_INVALID, "pair 2 has axis 3"),
    (dict(pair_axes=(0, -1, 2, 0)), rp.ROPE_ERR_INVALID, "pair 1 has axis -1"),
    (dict(mode=3), rp.ROPE_ERR_INVALID, "mode"),
    (dict(partial_slice=(4, 18)), rp.ROPE_ERR_INVALID, "end"),
])
@pytest.mark.parametrize("out", [False, True])
def test_refusals(change, status, text, out):
    kw = dict(change, out=out, y_ptr=FAKE + (1 << 20))
    assert call(**kw) == status
    assert text in rp.last_error()


def test_out_of_place_overlap_is_refused():
    assert call(out=True, y_ptr=FAKE + 32) == rp.ROPE_ERR_INVALID
    assert "overlap" in rp.last_error()


def test_empty_calls_read_no_pointer():
    nothing = dict(x_ptr=None, pos_ptr=None, inv_freq_ptr=None, pair_axes=None, pos_shape=None, pos_strides=None)
    assert call(x_shape=(2, 0, 3, 16), **nothing) == rp.ROPE_OK
    assert call(partial_slice=(4, 4), **nothing) == rp.ROPE_OK
    assert rp.raw_axes_multi_call("fwd", [], [], 2, None, None, None, None, None, 2, 1, None) == rp.ROPE_OK


def test_multi_refusals_name_the_tensor():
    def multi(ptrs, shapes, **kw):
        a = dict(OK)
        a.update(kw)
        return rp.raw_axes_multi_call("bwd", ptrs, shapes, 2, FAKE, a["pos_shape"], a["pos_strides"], FAKE,
                                      a["pair_axes"], 2, 1, (4, 12))
    far = FAKE + (1 << 20)
    assert multi([FAKE, None], [SHAPE, SHAPE]) == rp.ROPE_ERR_NULLPTR and "tensor 1" in rp.last_error()
    assert multi([FAKE, far], [SHAPE, (2, 6, 3, 16)]) == rp.ROPE_ERR_INVALID and "tensor 1" in rp.last_error()
    assert multi([FAKE, FAKE], [SHAPE, SHAPE]) == rp.ROPE_ERR_INVALID and "overlap" in rp.last_error()
    assert multi([FAKE, far], [SHAPE, SHAPE], pair_axes=(0, 1, 2, 9)) == rp.ROPE_ERR_INVALID


def test_launch_info_plans_like_one_axis():
    for shape, sl, kernel in (((2, 5, 3, 64), (0, 64), "vector"), ((2, 5, 3, 36), (3, 11), "rows")):
        n = (sl[1] - sl[0]) // 2
        st, got = rp.raw_launch_info_axes(FAKE, shape, 2, FAKE, (2, 1, 5), (5, 5, 1), FAKE, (1,) * n, 2, 0, sl)
        assert (st, got) == (rp.ROPE_OK, kernel)
        st, plan = rp.raw_launch_info_pos(FAKE, shape, 2, FAKE, (1, 5), (5, 1), FAKE, 2, 0, sl)
        assert plan["kernel"] == kernel


def test_tensor_checks_of_the_binding():
    x = torch.zeros(SHAPE, dtype=torch.bfloat16)
    pos = torch.zeros(3, 2, 5, dtype=torch.int64)
    f = torch.ones(4, dtype=torch.float64)
    ok = dict(rotary_mode="interleave", partial_slice=(4, 12))
    with pytest.raises(ValueError, match="3-D int64"):
        rp.rope_partial_fwd_inplace_axes(x, pos[0], f, (0, 1, 2, 0), **ok)
    with pytest.raises(ValueError, match="3-D int64"):
        rp.rope_partial_fwd_inplace_axes(x, pos.int(), f, (0, 1, 2, 0), **ok)
    with pytest.raises(ValueError, match="pair_axes must hold"):
        rp.rope_partial_fwd_inplace_axes(x, pos, f, (0, 1, 2), **ok)
    with pytest.raises(ValueError, match="GPU tensor"):
        rp.rope_partial_fwd_inplace_axes(x, pos, f, (0, 1, 2, 0), **ok)
    with pytest.raises(ValueError, match="must be one of"):
        rp.rope_partial_fwd_inplace_axes(x, pos, f, (0, 1, 2, 0), rotary_mode="spiral", partial_slice=(4, 12))
    with pytest.raises(RuntimeError, match="leaf"):
        rp.inplace_partial_rotary_mul_axes(x.requires_grad_(), pos, f, (0, 1, 2, 0), **ok)
