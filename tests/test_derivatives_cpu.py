"""Derivatives of the autograd operators beyond the first, and in forward mode,
against the same rotation written in recorded torch operations. On the CPU,
with the kernel calls replaced by the rotation in fp64 that autograd does not
see, as it does not see a kernel."""
import numpy as np
import pytest
import torch
import torch.autograd.forward_ad as fw

import transformer_positional_encoding_amd as rp
from axes_refs import half_of, pair_tables, rotate64

SHAPE, SL = (2, 5, 3, 16), (4, 12)
PAIR_AXES = (0, 1, 2, 0)


def unseen(y, x, cos, sin, mode, sl, direction):
    """y's bytes become x's rotated ones; cos and sin a pair's."""
    out = rotate64(x.detach().clone().double(), cos, sin, mode, sl, back=direction == "bwd")[0]
    np.copyto(y.detach().numpy(), out.numpy())


@pytest.fixture(autouse=True)
def kernels(monkeypatch):
    def call_pos(direction, x, positions, inv_freq, mode, partial_slice, table_dtype, stream, pair_axes=None, y=None):
        if pair_axes is None:
            positions, pair_axes = positions[None], (0,) * inv_freq.numel()
        assert x.is_contiguous()
        cos, sin = pair_tables(positions, inv_freq, pair_axes, "f32")
        unseen(x if y is None else y, x, cos, sin, mode, partial_slice, direction)

    def call_out(direction, y, x, r1, r2, mode, partial_slice, stream):
        assert x.is_contiguous()
        unseen(y, x, r1, r2, mode, partial_slice, direction)

    monkeypatch.setattr(rp, "_call_pos", call_pos)
    monkeypatch.setattr(rp, "_call_out", call_out)
    monkeypatch.setattr(rp, "_call", lambda direction, x, *how: call_out(direction, x, x, *how))


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


POSITIONS = torch.randint(0, 900, (3, 2, 5), generator=torch.Generator().manual_seed(1))
FREQ = rp.rope_inv_freq(SL[1] - SL[0], 100.0)


def plain_rotation(x, cos, sin, mode, sl=SL, minus=-1.0):
    """The rotation in operations that autograd records; minus: the sign of
    the first lanes' second term."""
    s, e = sl
    h = half_of(mode, e - s)
    j = torch.arange(e - s)
    first = (j // h) % 2 == 0
    other, pair = torch.where(first, j + h, j - h), j // (2 * h) * h + j % h
    z = x[..., s:e]
    turned = z * cos[..., pair] + torch.where(first, minus, 1.0).double() * z[..., other] * sin[..., pair]
    return torch.cat([x[..., :s], turned, x[..., e:]], dim=-1)


def in_place(rotate):
    def call(x):
        y = x * 1.0
        rotate(y)
        return y
    return call


def operators(form, mode):
    """(the operator, its plain form), functions of x."""
    if form.startswith("axes"):
        how = (POSITIONS, FREQ, PAIR_AXES, mode, SL)
        cos, sin = pair_tables(POSITIONS, FREQ, PAIR_AXES, "f32")
        out, inplace = rp.partial_rotary_mul_axes, rp.inplace_partial_rotary_mul_axes
    elif form.startswith("pos"):
        how = (POSITIONS[0], FREQ, mode, SL)
        cos, sin = pair_tables(POSITIONS[:1], FREQ, (0,) * 4, "f32")
        out, inplace = rp.partial_rotary_mul_pos, rp.inplace_partial_rotary_mul_pos
    else:
        cos, sin = rand((2, 5, 1, 4), 40), rand((2, 5, 1, 4), 41)
        how = (cos, sin, mode, SL)
        out, inplace = rp.partial_rotary_mul, rp.inplace_partial_rotary_mul
    op = in_place(lambda y: inplace(y, *how)) if form.endswith("in place") else lambda x: out(x, *how)
    return op, lambda x: plain_rotation(x, cos, sin, mode)


FORMS = ["axes", "axes in place", "pos", "pos in place", "tables", "tables in place"]
both = [pytest.mark.parametrize("form", FORMS), pytest.mark.parametrize("mode", ["interleave", "rotate_half"])]


def each(test):
    for mark in both:
        test = mark(test)
    return test


def close(got, want):
    # both sides round some tens of fp64 sums and products, of 2^-53 each
    assert torch.allclose(got, want, rtol=1e-12, atol=1e-12 * float(want.abs().max())) and float(want.abs().max()) > 0


@each
def test_gradient_penalty(form, mode):
    """The weight's gradient of a squared gradient, through two backwards."""
    op, ref = operators(form, mode)
    x, w = rand((2, 5, 7), 2), rand((7, 48), 3)

    def penalty(f):
        xx, ww = x.clone().requires_grad_(), w.clone().requires_grad_()
        loss = (f((xx @ ww).view(SHAPE)) ** 3).sum()
        (g,) = torch.autograd.grad(loss, xx, create_graph=True)
        return torch.autograd.grad((g ** 2).sum(), ww)[0]

    close(penalty(op), penalty(ref))


@each
def test_third_derivative(form, mode):
    op, ref = operators(form, mode)

    def third(f):
        x = rand(SHAPE, 4).requires_grad_()
        g = f(x)
        for k in range(3):
            (g,) = torch.autograd.grad((g ** 3 * rand(SHAPE, 5 + k)).sum(), x, create_graph=k < 2)
        return g

    close(third(op), third(ref))


@each
def test_forward_mode(form, mode):
    """The tangent turns with the value, whether or not a gradient is asked
    for, and with gradients disabled."""
    op, ref = operators(form, mode)
    x, t = rand(SHAPE, 6), rand(SHAPE, 7)
    for needs, enabled in ((False, True), (True, True), (False, False)):
        with fw.dual_level(), torch.set_grad_enabled(enabled):
            y = fw.unpack_dual(op(fw.make_dual(x.clone().requires_grad_(needs), t)))
            assert y.tangent is not None
            close(y.tangent.detach(), ref(t))
            close(y.primal.detach(), ref(x))


@pytest.mark.parametrize("form", ["axes", "pos", "tables"])
@pytest.mark.parametrize("mode", ["interleave", "rotate_half"])
def test_forward_mode_in_place_of_a_value_without_gradient(form, mode):
    """In place on the dual tensor itself, its tangent not contiguous."""
    x, t = rand(SHAPE, 6), rand((16, 3, 5, 2), 7).permute(3, 2, 1, 0)
    rotate, how = {"axes": (rp.inplace_partial_rotary_mul_axes, (POSITIONS, FREQ, PAIR_AXES)),
                   "pos": (rp.inplace_partial_rotary_mul_pos, (POSITIONS[0], FREQ)),
                   "tables": (rp.inplace_partial_rotary_mul, (rand((2, 5, 1, 4), 40), rand((2, 5, 1, 4), 41)))}[form]
    _, ref = operators(form, mode)
    with fw.dual_level():
        d = fw.make_dual(x.clone(), t.clone())
        rotate(d, *how, mode, SL)
        y = fw.unpack_dual(d)
        close(y.tangent, ref(t))
        close(y.primal, ref(x))


@each
def test_forward_over_reverse(form, mode):
    """The tangent of a gradient: a Hessian times a direction."""
    op, ref = operators(form, mode)
    x, t = rand(SHAPE, 8), rand(SHAPE, 9)

    def hvp(f):
        with fw.dual_level():
            d = fw.make_dual(x.clone().requires_grad_(), t)
            (g,) = torch.autograd.grad((f(d) ** 3).sum(), d, create_graph=True)
            return fw.unpack_dual(g).tangent.detach()

    close(hvp(op), hvp(ref))


@each
def test_gradients_of_tangents(form, mode):
    """A tangent that needs a gradient: reverse over forward."""
    op, ref = operators(form, mode)
    x = rand(SHAPE, 10)

    def of(f):
        t = rand(SHAPE, 11).requires_grad_()
        with fw.dual_level():
            y = fw.unpack_dual(f(fw.make_dual(x.clone(), t * 1.0)))
            return torch.autograd.grad((y.tangent ** 3).sum(), t)[0]

    close(of(op), of(ref))
