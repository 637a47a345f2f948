"""Norms of query and key heads with their rotation, forward and backward,
against the definition in 64 bits."""
import pytest
import torch

import transformer_positional_encoding_amd as rp
from axes_refs import pair_tables
from serving_refs import TYPES, half_step, norm64, norm_back64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6


def inputs(B, S, hq, hk, D, sl, dtype, weight, seed, lay="fused", axes=1):
    g = torch.Generator().manual_seed(seed)
    t = TYPES[dtype]
    c = {}
    if lay == "fused":        # Q, K and V of a token beside each other
        x = torch.randn(B, S, hq + 2 * hk, D, generator=g)
        x[..., 1::5] *= 7
        x = x.to(t).cuda()
        c["q"], c["k"] = x[:, :, :hq], x[:, :, hq:hq + hk] if hk else None
    elif lay == "heads first":
        c["q"] = torch.randn(B, hq, S, D, generator=g).to(t).cuda().transpose(1, 2)
        c["k"] = torch.randn(B, hk, S, D, generator=g).to(t).cuda().transpose(1, 2) if hk else None
    else:                     # rows that are not aligned to vectors
        c["q"] = torch.randn(B, S, hq, D + 3, generator=g).to(t).cuda()[..., 1:D + 1]
        c["k"] = torch.randn(B, S, hk, D + 5, generator=g).to(t).cuda()[..., 3:D + 3] if hk else None
    c["wq"] = None if weight is None else (1 + 0.4 * torch.randn(D, generator=g)).to(TYPES[weight]).cuda()
    c["wk"] = None if weight is None or not hk else (1 + 0.4 * torch.randn(D, generator=g)).to(TYPES[weight]).cuda()
    c["gq"] = torch.randn(B, S, hq, D, generator=g).to(t).cuda()
    c["gk"] = torch.randn(B, S, hk, D, generator=g).to(t).cuda() if hk else None
    pairs = (sl[1] - sl[0]) // 2
    c["f"] = rp.rope_inv_freq(max(2, 2 * pairs), 10000.0, "cuda")[:pairs].contiguous()
    if axes == 1:
        c["pos"] = torch.randint(0, 50000, (B, S), generator=g).cuda()
        c["axes"] = None
    else:
        c["pos"] = torch.randint(0, 5000, (axes, 1, S), generator=g).cuda()
        c["axes"] = tuple(int(v) for v in torch.randint(0, axes, (pairs,), generator=g))
    return c


def tables(c, table):
    pos = c["pos"] if c["pos"].dim() == 3 else c["pos"][None]
    return pair_tables(pos, c["f"], c["axes"] or (0,) * len(c["f"]), table)


def check_fwd(got, x, w, c, mode, sl, table, what):
    D = x.shape[-1]
    y, size = norm64(x.cpu(), None if w is None else w.cpu(), EPS, *tables(c, table), mode, sl)
    # the sum of D squares, its root, three products, the rotation's three roundings
    lim = (D / 2 + 16) * U * size
    lim = lim + half_step(x.dtype, y.abs() + lim)
    err = (got.cpu().double() - y).abs()
    assert bool((err <= lim).all()), f"{what}: {float((err / lim).nan_to_num(9e9).max()):.3g} of the limit"


def check_bwd(dx, dw, x, w, dy, c, mode, sl, table, what):
    D, rows = x.shape[-1], x.shape[0] * x.shape[1] * x.shape[2]
    want, want_w, size, size_w = norm_back64(x.cpu(), None if w is None else w.cpu(), EPS, dy.cpu(), *tables(c, table), mode, sl)
    lim = (2 * D + 32) * U * size
    lim = lim + half_step(x.dtype, want.abs() + lim)
    err = (dx.cpu().double() - want).abs()
    assert bool((err <= lim).all()), f"{what}: {float((err / lim).nan_to_num(9e9).max()):.3g} of the limit"
    if w is None:
        assert dw is None
        return
    lim = (rows + D + 32) * U * size_w
    lim = lim + half_step(w.dtype, want_w.abs() + lim)
    err = (dw.cpu().double() - want_w).abs()
    assert bool((err <= lim).all()), f"{what} weight: {float((err / lim).nan_to_num(9e9).max()):.3g} of the limit"


CASES = [
    # B, S, hq, hk, D, slice, mode, dtype, weight, table, layout, axes
    (2, 5, 4, 2, 128, (0, 128), "rotate_half", "bf16", "bf16", "bf16", "fused", 1),
    (1, 1, 32, 8, 128, (0, 128), "rotate_half", "bf16", "f32", "f32", "fused", 1),
    (3, 7, 5, 1, 128, (0, 128), "interleave", "f16", "f16", "f32", "fused", 1),
    (2, 9, 3, 3, 64, (0, 64), "rotate_half", "f32", "f32", "f32", "fused", 1),
    (2, 33, 4, 4, 80, (0, 48), "interleave", "f16", "f32", "f32", "fused", 1),
    (2, 17, 4, 2, 80, (0, 80), "rotate_half", "bf16", "bf16", "f32", "fused", 1),
    (1, 40, 2, 1, 256, (64, 192), "rotate_half", "bf16", "bf16", "bf16", "fused", 1),
    (2, 11, 6, 2, 192, (128, 192), 4, "bf16", "f32", "bf16", "fused", 1),
    (2, 13, 3, 2, 36, (4, 32), "rotate_half", "bf16", "bf16", "bf16", "fused", 1),
    (2, 13, 3, 2, 36, (0, 36), "interleave", "f32", "f32", "f32", "fused", 1),
    (1, 6, 2, 2, 2, (0, 2), "interleave", "f32", "f32", "f32", "fused", 1),
    (1, 5, 2, 1, 1024, (0, 1024), "rotate_half", "bf16", "bf16", "bf16", "fused", 1),
    (1, 5, 2, 1, 1024, (0, 1024), "interleave", "f32", "f32", "f32", "fused", 1),
    (1, 4, 1, 1, 520, (8, 24), "interleave", "f16", "f16", "f16", "fused", 1),
    (2, 19, 7, 3, 96, (0, 96), "rotate_half", "f16", "f16", "f16", "heads first", 1),
    (2, 19, 7, 3, 128, (0, 64), "rotate_half", "bf16", "f32", "bf16", "heads first", 1),
    (2, 8, 3, 2, 64, (0, 64), "rotate_half", "bf16", "bf16", "bf16", "unaligned", 1),
    (2, 8, 3, 2, 72, (2, 70), "interleave", "f32", "f32", "f32", "unaligned", 1),
    (2, 21, 4, 2, 128, (0, 128), "rotate_half", "bf16", "bf16", "bf16", "fused", 3),
    (2, 6, 4, 0, 128, (0, 128), "rotate_half", "bf16", "bf16", "bf16", "fused", 1),
    (2, 6, 4, 2, 128, (0, 0), "rotate_half", "bf16", "bf16", "bf16", "fused", 1),
    (2, 6, 4, 2, 128, (0, 128), "rotate_half", "f16", None, "f16", "fused", 1),
    (5, 613, 4, 1, 128, (0, 128), "rotate_half", "bf16", "f32", "bf16", "fused", 1),
    (3, 1100, 3, 2, 40, (0, 20), "rotate_half", "f16", "f32", "f32", "fused", 1),
]


@pytest.mark.parametrize("B, S, hq, hk, D, sl, mode, dtype, weight, table, lay, axes", CASES)
def test_forward_and_backward(B, S, hq, hk, D, sl, mode, dtype, weight, table, lay, axes):
    c = inputs(B, S, hq, hk, D, sl, dtype, weight, 11, lay, axes)
    how = dict(positions=c["pos"], inv_freq=c["f"], rotary_mode=mode, partial_slice=sl, eps=EPS, pair_axes=c["axes"],
               table_dtype=TYPES[table])
    q, k = rp.rope_qk_norm_fwd(c["q"], c["k"], c["wq"], c["wk"], **how)
    check_fwd(q, c["q"], c["wq"], c, mode, sl, table, "q")
    dq, dk, dwq, dwk = rp.rope_qk_norm_bwd(c["gq"], c["gk"], c["q"], c["k"], c["wq"], c["wk"], **how)
    check_bwd(dq, dwq, c["q"], c["wq"], c["gq"], c, mode, sl, table, "dq")
    if hk:
        check_fwd(k, c["k"], c["wk"], c, mode, sl, table, "k")
        check_bwd(dk, dwk, c["k"], c["wk"], c["gk"], c, mode, sl, table, "dk")
    else:
        assert k is None and dk is None and dwk is None


@pytest.mark.parametrize("D, sl, mode, lay", [(128, (0, 128), "rotate_half", "fused"), (96, (32, 96), "interleave", "fused"),
                                              (64, (0, 64), "rotate_half", "unaligned"), (36, (0, 28), "interleave", "fused")])
def test_in_place_equals_out_of_place(D, sl, mode, lay):
    c = inputs(3, 50, 6, 2, D, sl, "bf16", "bf16", 5, lay)
    how = dict(positions=c["pos"], inv_freq=c["f"], rotary_mode=mode, partial_slice=sl)
    q, k = rp.rope_qk_norm_fwd(c["q"], c["k"], c["wq"], c["wk"], **how)
    dq, dk, dwq, dwk = rp.rope_qk_norm_bwd(c["gq"], c["gk"], c["q"], c["k"], c["wq"], c["wk"], **how)
    gq, gk = c["gq"].clone(), c["gk"].clone()
    got = rp.rope_qk_norm_bwd(gq, gk, c["q"], c["k"], c["wq"], c["wk"], dq=gq, dk=gk, **how)
    assert got[0] is gq and torch.equal(gq, dq) and torch.equal(gk, dk) and torch.equal(got[2], dwq) and torch.equal(got[3], dwk)
    beside = c["q"]._base.clone() if c["q"]._base is not None else None
    got = rp.rope_qk_norm_fwd(c["q"], c["k"], c["wq"], c["wk"], q_out=c["q"], k_out=c["k"], **how)
    assert got[0] is c["q"] and torch.equal(c["q"], q) and torch.equal(c["k"], k)
    if lay == "fused":        # V, between and behind, keeps its bytes
        assert torch.equal(c["q"]._base[:, :, 8:], beside[:, :, 8:])


def test_autograd_equals_the_calls_and_differences():
    """Gradients by autograd are the backward call's; the loss's differences
    along random directions agree with them in fp32."""
    sl, mode = (0, 64), "rotate_half"
    c = inputs(2, 9, 3, 2, 64, sl, "f32", "f32", 21)
    how = (c["pos"], c["f"], mode, sl)
    ins = [c[n].detach().clone().requires_grad_(True) for n in ("q", "k", "wq", "wk")]
    y = rp.qk_norm_rotary(*ins, *how, eps=1e-3)
    grads = torch.autograd.grad(y, ins, (c["gq"], c["gk"]))
    want = rp.rope_qk_norm_bwd(c["gq"], c["gk"], c["q"], c["k"], c["wq"], c["wk"], *how, eps=1e-3)
    for a, b in zip(grads, want):
        assert torch.equal(a, b)
    cos, sin = tables(c, "f32")

    def loss(q, k, wq, wk):
        return sum((norm64(x.cpu(), w.cpu(), 1e-3, cos, sin, mode, sl)[0] * gr.cpu().double()).sum()
                   for x, w, gr in ((q, wq, c["gq"]), (k, wk, c["gk"])))

    g = torch.Generator().manual_seed(3)
    base = [c[n].double().cpu() for n in ("q", "k", "wq", "wk")]
    for i in range(4):
        step = torch.randn(base[i].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        moved = [[b + (s * h * step if j == i else 0) for j, b in enumerate(base)] for s in (1, -1)]
        slope = (loss(*moved[0]) - loss(*moved[1])) / (2 * h)
        along = (grads[i].cpu().double() * step).sum()
        # the differences' own error is h^2; the gradient's terms round to fp32
        size = (grads[i].cpu().double() * step).abs().sum()
        assert abs(float(slope - along)) <= float(size) * 2000 * U + 1e-4


def test_some_gradients_only():
    c = inputs(2, 5, 2, 1, 64, (0, 64), "f32", "f32", 2)
    how = (c["pos"], c["f"], "interleave", (0, 64))
    full = rp.rope_qk_norm_bwd(c["gq"], c["gk"], c["q"], c["k"], c["wq"], c["wk"], *how)
    for name, i in (("q", 0), ("k", 1), ("wq", 2), ("wk", 3)):
        ins = {n: c[n].detach().clone() for n in ("q", "k", "wq", "wk")}
        ins[name].requires_grad_(True)
        y = rp.qk_norm_rotary(*ins.values(), *how)
        (got,) = torch.autograd.grad(y, ins[name], (c["gq"], c["gk"]))
        assert torch.equal(got, full[i])
    # only q's result is used: k's gradients are those of zeros
    ins = {n: c[n].detach().clone().requires_grad_(True) for n in ("q", "k", "wq", "wk")}
    y, _ = rp.qk_norm_rotary(*ins.values(), *how)
    got = torch.autograd.grad(y, tuple(ins.values()), c["gq"])
    assert torch.equal(got[0], full[0]) and torch.equal(got[2], full[2])
    assert not bool(got[1].any()) and not bool(got[3].any())
    # an expanded gradient (all strides 0)
    y, _ = rp.qk_norm_rotary(*ins.values(), *how)
    got = torch.autograd.grad(y.sum(), (ins["q"], ins["wq"]))
    want = rp.rope_qk_norm_bwd(torch.ones_like(c["gq"]), torch.zeros_like(c["gk"]), c["q"], c["k"], c["wq"], c["wk"], *how)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[2])


def test_twice_differentiated_and_forward_mode_are_refused():
    c = inputs(1, 3, 2, 1, 64, (0, 64), "f32", "f32", 2)
    q = c["q"].detach().clone().requires_grad_(True)
    y, _ = rp.qk_norm_rotary(q, c["k"], c["wq"], c["wk"], c["pos"], c["f"], "interleave", (0, 64))
    (g,) = torch.autograd.grad(y, q, torch.ones_like(y).requires_grad_(True), create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.sum(), q)
    with pytest.raises(RuntimeError, match="needs a gradient"):
        rp.rope_qk_norm_fwd(q, c["k"])
    with torch.autograd.forward_ad.dual_level():
        d = torch.autograd.forward_ad.make_dual(c["q"].detach().clone(), torch.ones_like(c["q"]))
        with pytest.raises(Exception):
            rp.qk_norm_rotary(d, c["k"], c["wq"], c["wk"], c["pos"], c["f"], "interleave", (0, 64))


@pytest.mark.parametrize("D, lay", [(64, "fused"), (36, "fused")])
def test_zero_rows_and_empty_calls(D, lay):
    sl = (0, D)
    c = inputs(2, 3, 2, 1, D, sl, "f32", "f32", 8, lay)
    c["q"][0, 1, 0] = 0
    how = dict(positions=c["pos"], inv_freq=c["f"], rotary_mode="interleave", partial_slice=sl)
    q, _ = rp.rope_qk_norm_fwd(c["q"], c["k"], c["wq"], c["wk"], **how)
    assert not bool(q[0, 1, 0].any()) and bool(torch.isfinite(q).all())
    q, _ = rp.rope_qk_norm_fwd(c["q"], c["k"], c["wq"], c["wk"], eps=0.0, **how)
    assert bool(torch.isnan(q[0, 1, 0]).all()) and bool(torch.isfinite(q[0, 0]).all())
    e = c["q"][:0]
    q, k = rp.rope_qk_norm_fwd(e, c["k"][:0], c["wq"], c["wk"], **dict(how, positions=c["pos"][:0]))
    assert q.shape == e.shape
    got = rp.rope_qk_norm_bwd(e, c["k"][:0], e, c["k"][:0], c["wq"], c["wk"], **dict(how, positions=c["pos"][:0]))
    assert not bool(got[2].any()) and not bool(got[3].any())


def test_captured_and_on_another_stream():
    c = inputs(2, 65, 4, 2, 128, (0, 128), "bf16", "f32", 9)
    how = dict(positions=c["pos"], inv_freq=c["f"], rotary_mode="rotate_half", partial_slice=(0, 128))
    ws = torch.empty(rp.rope_qk_norm_workspace(128), dtype=torch.uint8, device="cuda")

    def step():
        y = rp.rope_qk_norm_fwd(c["q"], c["k"], c["wq"], c["wk"], **how)
        return y + rp.rope_qk_norm_bwd(c["gq"], c["gk"], c["q"], c["k"], c["wq"], c["wk"], workspace=ws, **how)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        c["q"].mul_(0.9).add_(0.1)
        c["gk"].neg_()
        c["pos"].add_(13)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    want = step()
    torch.cuda.synchronize()
    y = rp.rope_qk_norm_fwd(c["q"], c["k"], c["wq"], c["wk"], stream=s, **how)
    z = rp.rope_qk_norm_bwd(c["gq"], c["gk"], c["q"], c["k"], c["wq"], c["wk"], stream=s, **how)
    s.synchronize()
    for a, b in zip(y + z, want):
        assert torch.equal(a, b)
