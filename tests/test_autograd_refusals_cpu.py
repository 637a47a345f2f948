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
    monkeypatch.setattr(rp, "_words_entry", lambda name: getattr(Library(), name))
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


def cache_operands(**kw):
    bf = torch.bfloat16
    a = dict(q=torch.zeros(B, S, 3, D, dtype=bf), k=torch.zeros(B, S, N, D, dtype=bf), v=torch.zeros(B, S, N, D, dtype=bf),
             data=torch.zeros(2, 4, N, D, dtype=bf), out=torch.zeros(B, S, N, D, dtype=bf))
    a.update(kw)
    return a


def as_on_a_gpu(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(rp, "_on_device", lambda t, stream: (None, rp._NOTHING))


def write(a):
    c = rp.RopeCache(a["data"])
    v_cache = rp.RopeCache(torch.zeros(2, 4, N, D, dtype=torch.int8), torch.zeros(2, 4, N, 1))
    rp.rope_cache_write(a["k"], a["v"], c, v_cache, torch.zeros(B, S, dtype=torch.int64), q=a["q"])


def read(a):
    rp.rope_cache_read(a["out"], rp.RopeCache(a["data"]), torch.zeros(B, 1, dtype=torch.int32),
                       torch.zeros(B, dtype=torch.int32))


@pytest.mark.parametrize("call, names", [(write, ("q", "k", "v", "data")), (read, ("out", "data"))])
def test_cache_calls_refuse_what_needs_a_gradient(call, names, no_library, monkeypatch):
    as_on_a_gpu(monkeypatch)
    call(cache_operands())
    for name in names:
        a = cache_operands()
        a[name].requires_grad_()
        with pytest.raises(RuntimeError, match="needs a gradient"):
            call(a)
        with torch.no_grad():
            call(a)
        with torch.inference_mode():
            call(cache_operands())
        a[name] = a[name].detach()
        call(a)
        with torch.autograd.forward_ad.dual_level(), torch.no_grad():
            a[name] = torch.autograd.forward_ad.make_dual(a[name], torch.ones_like(a[name]))
            with pytest.raises(RuntimeError, match="needs a gradient"):
                call(a)


@pytest.mark.parametrize("call, name", [(write, "q"), (write, "data"), (read, "out")])
def test_cache_calls_in_place_are_seen(call, name, no_library, monkeypatch):
    as_on_a_gpu(monkeypatch)
    a = cache_operands()
    w = torch.ones_like(a[name], requires_grad=True)
    y = w * a[name]
    call(a)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def project(a):
    return rp.rope_proj_lora_fwd(heads=2, partial_slice=(0, 32), **a)


def lora_operands():
    bf = torch.bfloat16
    return dict(x=torch.zeros(6, 64, dtype=bf), w=torch.zeros(64, 64, dtype=bf), a=torch.zeros(3, 8, 64, dtype=bf),
                b=torch.zeros(3, 64, 8, dtype=bf), adapters=torch.zeros(6, dtype=torch.int32),
                r1=torch.zeros(1, 6, 1, 32, dtype=bf), r2=torch.zeros(1, 6, 1, 32, dtype=bf), scales=torch.ones(3),
                out=torch.zeros(1, 6, 2, 32, dtype=bf), workspace=torch.zeros(1024, dtype=torch.uint8))


def test_the_projection_with_adapters_refuses_what_needs_a_gradient(no_library, monkeypatch):
    as_on_a_gpu(monkeypatch)
    project(lora_operands())
    for name in ("x", "w", "a", "b", "r1", "r2", "scales", "out"):
        a = lora_operands()
        a[name].requires_grad_()
        with pytest.raises(RuntimeError, match=f"{name} needs a gradient"):
            project(a)
        with torch.no_grad():
            project(a)
    w = torch.ones(1, 6, 2, 32, requires_grad=True)
    a = lora_operands()
    y = w.bfloat16() * a["out"]
    project(a)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
