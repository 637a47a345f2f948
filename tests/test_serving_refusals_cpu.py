"""Every refusal of the norms, the page bookkeeping and the attention over a
cache (no GPU: nothing is launched)."""
import ctypes

import pytest
import torch

import transformer_positional_encoding_amd as rp

FAKE = 1 << 20
I3 = ctypes.c_int64 * 3
I2 = ctypes.c_int64 * 2
NULL, BAD, NO, OK = rp.ROPE_ERR_NULLPTR, rp.ROPE_ERR_INVALID, rp.ROPE_ERR_UNSUPPORTED, rp.ROPE_OK


def rows(N=2, D=16, strides=(160, 32, 16), data=FAKE):
    return rp.RopeRows(data, N, D, strides)


def cache(**kw):
    a = dict(data=FAKE, scales=FAKE, format=5, pages=3, page_size=4, heads=2, dim=16, group=8, strides=(64, 16, 8),
             scale_strides=(16, 4, 2))
    a.update(kw)
    return rp.RopeCacheStruct(a["data"], a["scales"], a["format"], a["pages"], a["page_size"], a["heads"], a["dim"],
                              a["group"], a["strides"], a["scale_strides"])


def said(st, want, text):
    assert st == want, (st, want, rp.last_error())
    if text:
        assert text in rp.last_error(), rp.last_error()


# ---------------------------------------------------------------- attention

def attention(**kw):
    a = dict(B=2, S=5, dtype=2, out=rows(4, 16, (320, 64, 16)), q=rows(4, 16, (320, 64, 16)), k=cache(), v=cache(), table=FAKE,
             cols=3, stride=3, lengths=FAKE, counts=None, scale=0.1, causal=1, ws=FAKE, bytes=1 << 24)
    a.update(kw)
    return rp.library().rope_cache_attention(a["B"], a["S"], a["dtype"], a["out"], a["q"], a["k"], a["v"], a["table"], a["cols"],
                                             a["stride"], a["lengths"], a["counts"], a["scale"], a["causal"], a["ws"],
                                             a["bytes"], None)


@pytest.mark.parametrize("kw, want, text", [
    (dict(q=None), NULL, "q"), (dict(out=None), NULL, "out"), (dict(k=None), NULL, "k_cache"), (dict(v=None), NULL, "v_cache"),
    (dict(B=-1), BAD, ""), (dict(dtype=5), BAD, ""), (dict(q=rows(4, 1026)), BAD, ""),
    (dict(k=cache(format=9)), BAD, "unknown format"), (dict(k=cache(format=4, strides=(128, 32, 16))), NO, "4 bits"),
    (dict(v=cache(format=2, strides=(256, 64, 32))), NO, "4 bits"), (dict(k=cache(group=3)), BAD, "group"),
    (dict(v=cache(pages=2)), BAD, "v_cache"), (dict(v=cache(page_size=2)), BAD, "v_cache"),
    (dict(v=cache(heads=1)), BAD, "v_cache"), (dict(q=rows(4, 14, (320, 64, 16))), BAD, "q: its lanes"),
    (dict(out=rows(4, 14, (320, 64, 16))), BAD, "out"), (dict(out=rows(2, 16, (320, 64, 16))), BAD, "out"),
    (dict(q=rows(3, 16, (320, 64, 16)), out=rows(3, 16, (320, 64, 16))), BAD, "multiple"),
    (dict(k=cache(heads=0), v=cache(heads=0)), BAD, "multiple"),
    (dict(q=rows(4, 0, (320, 64, 16)), k=cache(dim=0, group=2)), BAD, "without lanes"),
    (dict(q=rows(4, 16, (-1, 64, 16))), BAD, "negative stride"), (dict(out=rows(4, 16, (320, 64, 8))), BAD, "overlap"),
    (dict(q=rows(4, 16, (1 << 62, 64, 16))), BAD, "64-bit"), (dict(cols=-1), BAD, "block_table"),
    (dict(stride=-1), BAD, "block_table"), (dict(stride=1 << 62), BAD, "block_table"),
    (dict(scale=0.0), BAD, "scale"), (dict(scale=-1.0), BAD, "scale"), (dict(scale=float("nan")), BAD, "scale"),
    (dict(scale=float("inf")), BAD, "scale"), (dict(scale=1e300), BAD, "scale"), (dict(scale=1e-300), BAD, "scale"),
    (dict(B=1 << 20, S=1 << 20, q=rows(4, 16, (0, 0, 16)), out=rows(4, 16, (64 << 20, 64, 16))), NO, "2^31"),
    (dict(q=rows(4, 16, (320, 64, 16), None)), NULL, "q"), (dict(out=rows(4, 16, (320, 64, 16), None)), NULL, "out"),
    (dict(q=rows(4, 16, (320, 64, 16), FAKE + 1)), BAD, "aligned"), (dict(lengths=None), NULL, "lengths"),
    (dict(k=cache(data=None)), NULL, "k_cache"), (dict(v=cache(scales=None)), NULL, "v_cache"),
    (dict(v=cache(scales=FAKE + 2)), BAD, "v_cache"), (dict(table=None), NULL, "block_table"),
    (dict(ws=None), NULL, "workspace"), (dict(bytes=100), BAD, "too small"), (dict(ws=FAKE + 8), BAD, "workspace"),
    (dict(B=0), OK, ""), (dict(S=0), OK, ""), (dict(q=rows(0, 16), out=rows(0, 16)), OK, ""),
])
def test_attention_refusals(kw, want, text):
    said(attention(**kw), want, text)


def test_attention_workspace():
    size = rp.rope_cache_attention_workspace
    for bad in ((0, 1, 8, 2, 64), (1, 0, 8, 2, 64), (1, 1, 7, 2, 64), (1, 1, 8, 0, 64), (1, 1, 8, 2, 0), (1, 1, 8, 2, 2000),
                (1 << 20, 1 << 20, 8, 2, 64)):
        assert size(*bad) == 0
    for B, S, hq, hk, Dv in ((1, 1, 8, 8, 128), (64, 1, 32, 8, 128), (1, 1, 128, 1, 512), (16, 5, 40, 8, 128)):
        n = size(B, S, hq, hk, Dv)
        assert n % (B * S * hq * (Dv + 2) * 4) == 0 and 0 < n <= 1 << 27
    assert size(8, 4096, 32, 8, 128) == 0


def test_attention_on_host_tensors():
    q = torch.zeros(1, 1, 4, 16, dtype=torch.bfloat16)
    c = rp.RopeCache(torch.zeros(2, 4, 2, 8, dtype=torch.uint8), torch.zeros(2, 4, 2, 1))
    table, lengths = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        rp.rope_cache_attention(q, c, c, table, lengths)
    e = q[:0]
    got = rp.rope_cache_attention(e, c, c, table[:0], lengths[:0])
    assert got.shape == (0, 1, 4, 16)
    for bad in (dict(q=torch.zeros(1, 4, 16)), dict(q=e.long()), dict(k_cache=1), dict(block_table=table), dict(lengths=lengths),
                dict(lengths=lengths[:0].long()), dict(counts=lengths), dict(out=torch.zeros(0, 1, 4, 18)),
                dict(out=torch.zeros(0, 1, 4, 16)), dict(block_table=table[:0].t().contiguous().t().expand(0, 2).long()),
                dict(workspace=3)):
        a = dict(q=e, k_cache=c, v_cache=c, block_table=table[:0], lengths=lengths[:0])
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            rp.rope_cache_attention(**a)


# ---------------------------------------------------------------- pages

def reserve(**kw):
    a = dict(B=2, S=3, table=FAKE, cols=4, stride=4, lengths=FAKE, counts=FAKE, free=FAKE, cap=9, count=FAKE, page=16, slots=FAKE,
             positions=FAKE, granted=FAKE)
    a.update(kw)
    return rp.library().rope_cache_reserve(a["B"], a["S"], a["table"], a["cols"], a["stride"], a["lengths"], a["counts"],
                                           a["free"], a["cap"], a["count"], a["page"], a["slots"], a["positions"], a["granted"],
                                           None)


@pytest.mark.parametrize("kw, want, text", [
    (dict(B=-1), BAD, "B must"), (dict(S=0), BAD, "S at least 1"), (dict(cols=-1), BAD, "block_table"),
    (dict(stride=-4), BAD, "block_table"), (dict(stride=3), BAD, "overlap"), (dict(page=0), BAD, "page_size"),
    (dict(page=-1), BAD, "page_size"), (dict(cap=-1), BAD, "free_pages"), (dict(B=16385), NO, "RESERVE_MAX"),
    (dict(S=1 << 31), NO, "2^31"), (dict(page=1 << 31), NO, "2^31"), (dict(cap=1 << 31), NO, "2^31"),
    (dict(cols=1 << 31, stride=1 << 31), NO, "2^31"), (dict(stride=1 << 61), BAD, "64-bit"),
    (dict(table=None), NULL, "block_table"), (dict(lengths=None), NULL, "lengths"), (dict(counts=None), NULL, "counts"),
    (dict(free=None), NULL, "free_pages"), (dict(count=None), NULL, "free_count"), (dict(slots=None), NULL, "slots"),
    (dict(positions=None), NULL, "positions"), (dict(granted=None), NULL, "granted"), (dict(table=FAKE + 2), BAD, "aligned"),
    (dict(slots=FAKE + 4), BAD, "aligned"), (dict(B=0), OK, ""), (dict(B=0, table=None, lengths=None), OK, ""),
])
def test_reserve_refusals(kw, want, text):
    said(reserve(**kw), want, text)


def test_reserve_on_host_tensors():
    t = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        rp.rope_cache_reserve(t(2, 3), t(2), t(2), t(5), t(1), 16)
    got = rp.rope_cache_reserve(t(0, 3), t(0), t(0), t(5), t(1), 16, tokens=4)
    assert [tuple(v.shape) for v in got] == [(0, 4), (0, 4), (0,)]
    for bad in (dict(block_table=t(3)), dict(lengths=t(1)), dict(counts=t(0).long()), dict(free_pages=t(2, 2)), dict(free_count=t(2)),
                dict(slots=torch.zeros(0, 3)), dict(positions=t(0, 4)), dict(granted=t(3)), dict(free_pages=None)):
        a = dict(block_table=t(0, 3), lengths=t(0), counts=t(0), free_pages=t(5), free_count=t(1), page_size=16)
        a.update(bad)
        with pytest.raises(ValueError):
            rp.rope_cache_reserve(**a)


# ---------------------------------------------------------------- norms

def norm(backward, **kw):
    a = dict(B=2, S=5, dtype=2, y=rows(), ky=rows(), x=rows(), kx=rows(), g=rows(), kg=rows(), w=FAKE, kw=FAKE, dw=FAKE, dkw=FAKE,
             wdt=0, eps=1e-6, pos=FAKE, pos_shape=(1, 2, 5), pos_strides=(0, 5, 1), f=FAKE, axes=None, tdt=2, mode=1, sl=(4, 12),
             ws=FAKE, bytes=1 << 24)
    a.update(kw)
    arr = lambda t, v: None if v is None else t(*v)  # noqa: E731
    turn = (a["pos"], arr(I3, a["pos_shape"]), arr(I3, a["pos_strides"]), a["f"],
            None if a["axes"] is None else (ctypes.c_int32 * 4)(*a["axes"]), a["tdt"], a["mode"], arr(I2, a["sl"]))
    L = rp.library()
    if not backward:
        return L.rope_qk_norm_fwd(a["B"], a["S"], a["dtype"], a["y"], a["ky"], a["x"], a["kx"], a["w"], a["kw"], a["wdt"], a["eps"],
                                  *turn, None)
    return L.rope_qk_norm_bwd(a["B"], a["S"], a["dtype"], a["y"], a["ky"], a["dw"], a["dkw"], a["g"], a["kg"], a["x"], a["kx"],
                              a["w"], a["kw"], a["wdt"], a["eps"], *turn, a["ws"], a["bytes"], None)


NONE_K = dict(ky=None, kx=None, kg=None, kw=None, dkw=None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("kw, want, text", [
    (dict(x=None), NULL, "NULL"), (dict(y=None), NULL, "NULL"), (dict(kx=None), NULL, "k and what"),
    (dict(ky=None), NULL, "k and what"), (dict(B=-1), BAD, ""), (dict(dtype=3), BAD, ""), (dict(tdt=-1), BAD, ""),
    (dict(mode=3), BAD, ""), (dict(sl=(4, 9)), BAD, ""), (dict(sl=(4, 20)), BAD, ""), (dict(x=rows(2, 1026)), BAD, ""),
    (dict(wdt=3), BAD, "weight_dtype"), (dict(wdt=-1), BAD, "weight_dtype"), (dict(eps=-1e-6), BAD, "eps"),
    (dict(eps=float("nan")), BAD, "eps"), (dict(eps=float("inf")), BAD, "eps"), (dict(kx=rows(2, 14)), BAD, "lanes"),
    (dict(ky=rows(3)), BAD, "heads and lanes"), (dict(y=rows(2, 14)), BAD, "heads and lanes"),
    (dict(x=rows(strides=(-1, 32, 16))), BAD, "negative stride"), (dict(y=rows(strides=(160, 32, 8))), BAD, "overlap"),
    (dict(x=rows(strides=(1 << 62, 32, 16))), BAD, "64-bit"), (dict(w=FAKE + 2), BAD, "aligned"),
    (dict(x=rows(data=None)), NULL, "q"), (dict(kx=rows(data=None)), NULL, "k"), (dict(y=rows(data=None)), NULL, "data"),
    (dict(x=rows(data=FAKE + 1)), BAD, "aligned"), (dict(f=None), NULL, ""), (dict(pos_shape=None), NULL, ""),
    (dict(pos_shape=(1, 3, 5)), BAD, ""), (dict(pos_shape=(2, 2, 5)), NULL, ""), (dict(pos_strides=(0, -5, 1)), BAD, ""),
    (dict(B=0), OK, ""), (dict(S=0, w=None, kw=None, dw=None, dkw=None), OK, ""),
])
def test_norm_refusals(backward, kw, want, text):
    if want == OK:
        kw = dict(kw, dw=None, dkw=None)         # gradients of no rows would be written
    said(norm(backward, **kw), want, text)


@pytest.mark.parametrize("kw, want, text", [
    (dict(g=None), NULL, "q_grad"), (dict(kg=None), NULL, "k and what"), (dict(kg=rows(3)), BAD, "k_grad"),
    (dict(g=rows(2, 14)), BAD, "q_grad"), (dict(w=None), BAD, "no gradient"), (dict(kw=None), BAD, "no gradient"),
    (dict(dw=FAKE + 2), BAD, "aligned"), (dict(ws=None), NULL, "workspace"), (dict(ws=FAKE + 8), BAD, "workspace"),
    (dict(bytes=100), BAD, "too small"), (dict(g=rows(data=None)), NULL, "q_grad"),
    (dict(NONE_K, g=rows(data=None)), NULL, "q_grad"),
])
def test_norm_backward_refusals(kw, want, text):
    said(norm(True, **kw), want, text)


def test_norm_on_host_tensors():
    x, w = torch.zeros(1, 2, 3, 16, dtype=torch.bfloat16), torch.zeros(16)
    with pytest.raises(ValueError, match="GPU"):
        rp.rope_qk_norm_fwd(x, None, w)
    e = x[:0]
    assert rp.rope_qk_norm_fwd(e, e, w, w)[1].shape == e.shape
    for bad in (dict(q=x[0]), dict(k=e.float()), dict(k=x[:, :1]), dict(q_weight=w[:8]), dict(k_weight=w), dict(q_weight=w.double()),
                dict(k=e, q_weight=w, k_weight=w.bfloat16()), dict(q_out=e.float()), dict(q_out=x), dict(k_out=e),
                dict(q=e.long())):
        a = dict(q=e, k=None)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            rp.rope_qk_norm_fwd(**a)
    with pytest.raises(ValueError):
        rp.rope_qk_norm_bwd(e, e, e, None)
    with pytest.raises(ValueError):
        rp.rope_qk_norm_bwd(e.float(), None, e, None)
