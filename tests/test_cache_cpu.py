"""Every refusal of the cache entry points (no GPU: nothing is launched)."""
import ctypes

import pytest
import torch

import transformer_positional_encoding_amd as rp

FAKE = 1 << 20
I3 = ctypes.c_int64 * 3
I2 = ctypes.c_int64 * 2


def rows(N=2, D=16, strides=(160, 32, 16), data=FAKE):
    return rp.RopeRows(data, N, D, strides)


def cache(**kw):
    a = dict(data=FAKE, scales=FAKE, format=rp.CACHE_FORMATS["e4m3"], pages=3, page_size=4, heads=2, dim=16, group=8,
             strides=(128, 32, 16), scale_strides=(16, 4, 2))
    a.update(kw)
    return rp.RopeCacheStruct(a["data"], a["scales"], a["format"], a["pages"], a["page_size"], a["heads"], a["dim"],
                              a["group"], a["strides"], a["scale_strides"])


def write(**kw):
    a = dict(B=2, S=5, dtype=2, q=rows(3, 16, (240, 48, 16)), k=rows(), v=rows(), kc=cache(), vc=cache(), slots=FAKE,
             slot_strides=(5, 1), pos=FAKE, pos_shape=(1, 2, 5), pos_strides=(0, 5, 1), f=FAKE, axes=None, tdt=2, mode=1,
             sl=(4, 12), rotate=1)
    a.update(kw)
    arr = lambda t, v: None if v is None else t(*v)  # noqa: E731
    axes = None if a["axes"] is None else (ctypes.c_int32 * 4)(*a["axes"])
    return rp.library().rope_cache_write(a["B"], a["S"], a["dtype"], a["q"], a["k"], a["v"], a["kc"], a["vc"], a["slots"],
                                         arr(I2, a["slot_strides"]), a["pos"], arr(I3, a["pos_shape"]),
                                         arr(I3, a["pos_strides"]), a["f"], axes, a["tdt"], a["mode"], arr(I2, a["sl"]),
                                         a["rotate"], None)


def read(**kw):
    a = dict(B=2, S=5, dtype=2, out=rows(), c=cache(), table=FAKE, cols=3, stride=3, lengths=FAKE, starts=None, pos=FAKE,
             pos_shape=(1, 2, 5), pos_strides=(0, 5, 1), f=FAKE, axes=None, tdt=2, mode=1, sl=(4, 12))
    a.update(kw)
    arr = lambda t, v: None if v is None else t(*v)  # noqa: E731
    axes = None if a["axes"] is None else (ctypes.c_int32 * 4)(*a["axes"])
    return rp.library().rope_cache_read(a["B"], a["S"], a["dtype"], a["out"], a["c"], a["table"], a["cols"], a["stride"],
                                        a["lengths"], a["starts"], a["pos"], arr(I3, a["pos_shape"]),
                                        arr(I3, a["pos_strides"]), a["f"], axes, a["tdt"], a["mode"], arr(I2, a["sl"]),
                                        None)


NULL, BAD, NO = rp.ROPE_ERR_NULLPTR, rp.ROPE_ERR_INVALID, rp.ROPE_ERR_UNSUPPORTED

CACHE_REFUSALS = [
    (dict(format=6), BAD, "unknown format"), (dict(format=-1), BAD, "unknown format"),
    (dict(format=1), BAD, "storage type"), (dict(pages=-1), BAD, "negative dimension"),
    (dict(strides=(-128, 32, 16)), BAD, "negative stride"), (dict(strides=(1 << 62, 32, 16)), BAD, "64-bit"),
    (dict(pages=1 << 40, page_size=1 << 40), BAD, "slots"),
    (dict(group=0), BAD, "group"), (dict(group=3), BAD, "group"), (dict(group=10), BAD, "group"),
    (dict(scale_strides=(16, -4, 2)), BAD, "negative scale"), (dict(scale_strides=(1 << 61, 4, 2)), BAD, "64-bit"),
    (dict(heads=3, strides=(192, 48, 16), scale_strides=(24, 6, 2)), BAD, "heads and lanes"),
    (dict(dim=32, strides=(256, 64, 32), scale_strides=(32, 8, 4)), BAD, "heads and lanes"),
    (dict(data=None), NULL, "data is NULL"), (dict(scales=None), NULL, "scales is NULL"),
    (dict(scales=FAKE + 2), BAD, "aligned"), (dict(format=2, strides=(256, 64, 31)), BAD, "whole number of elements"),
    (dict(format=2, strides=(256, 64, 32), data=FAKE + 1), BAD, "aligned"),
]


@pytest.mark.parametrize("change, status, text", CACHE_REFUSALS + [
    (dict(strides=(32, 32, 16)), BAD, "overlap"), (dict(scale_strides=(16, 0, 2)), BAD, "overlap")])
def test_write_refuses_caches(change, status, text):
    assert write(kc=cache(**change)) == status, rp.last_error()
    assert text in rp.last_error()
    if "pages" not in change:
        assert write(vc=cache(**change)) == status and text in rp.last_error()


@pytest.mark.parametrize("change, status, text", CACHE_REFUSALS)
def test_read_refuses_caches(change, status, text):
    assert read(c=cache(**change)) == status, rp.last_error()
    assert text in rp.last_error()


@pytest.mark.parametrize("change, status, text", [
    (dict(k=None), NULL, "k or k_cache"), (dict(kc=None), NULL, "k or k_cache"), (dict(v=None), NULL, "v and v_cache"),
    (dict(vc=None), NULL, "v and v_cache"), (dict(B=-1), BAD, "negative"), (dict(dtype=3), BAD, "dtype"),
    (dict(tdt=7), BAD, "table dtype"), (dict(mode=3), BAD, "mode"), (dict(sl=(4, 20)), BAD, "end"),
    (dict(sl=(4, 7)), BAD, "even"),
    (dict(vc=cache(pages=4)), BAD, "pages"), (dict(q=rows(3, 18, (270, 54, 18))), BAD, "lanes"),
    (dict(k=rows(strides=(-1, 32, 16))), BAD, "negative"), (dict(k=rows(strides=(1 << 62, 32, 16))), BAD, "64-bit"),
    (dict(q=rows(3, 16, (240, 0, 16))), BAD, "overlap"), (dict(q=rows(3, 16, (16, 48, 16))), BAD, "overlap"),
    (dict(k=rows(data=None)), NULL, "k: data"), (dict(v=rows(data=None)), NULL, "v: data"),
    (dict(q=rows(3, 16, (240, 48, 16), data=None)), NULL, "q: data"), (dict(k=rows(data=FAKE + 1)), BAD, "aligned"),
    (dict(slots=None), NULL, "slots"), (dict(slot_strides=None), NULL, "slots"),
    (dict(slot_strides=(-5, 1)), BAD, "slots"), (dict(slot_strides=(1 << 61, 1)), BAD, "64-bit"),
    (dict(pos=None), NULL, "positions"), (dict(f=None), NULL, "inv_freq"), (dict(pos_shape=(1, 3, 5)), BAD, "dimension B"),
    (dict(pos_shape=(2, 2, 5)), NULL, "pair_axes"), (dict(pos_shape=(2, 2, 5), axes=(0, 1, 2, 0)), BAD, "pair 2"),
    (dict(B=1 << 20, S=1 << 12, k=rows(strides=(0, 0, 16)), v=None, vc=None, q=None), NO, "2^31"),
])
def test_write_refusals(change, status, text):
    assert write(**change) == status, rp.last_error()
    assert text in rp.last_error()


@pytest.mark.parametrize("change, status, text", [
    (dict(out=None), NULL, "out or cache"), (dict(c=None), NULL, "out or cache"), (dict(S=-1), BAD, "negative"),
    (dict(out=rows(strides=(160, 32, 0))), BAD, "overlap"), (dict(out=rows(strides=(0, 32, 16))), BAD, "overlap"),
    (dict(out=rows(data=None)), NULL, "out: data"), (dict(out=rows(data=FAKE + 1)), BAD, "aligned"),
    (dict(cols=-1), BAD, "block_table"), (dict(stride=-1), BAD, "block_table"), (dict(stride=1 << 61), BAD, "64-bit"),
    (dict(table=None), NULL, "block_table"), (dict(lengths=None), NULL, "lengths"), (dict(f=None), NULL, "inv_freq"),
    (dict(pos_shape=(1, 2, 4)), BAD, "dimension S"), (dict(mode=5), BAD, "mode"),
    (dict(B=1 << 20, S=1 << 11, out=rows(strides=(1 << 16, 32, 16))), NO, "2^31"),
])
def test_read_refusals(change, status, text):
    assert read(**change) == status, rp.last_error()
    assert text in rp.last_error()


def test_empty_calls_read_no_pointer():
    none = dict(slots=None, pos=None, f=None, pos_shape=None, pos_strides=None)
    gone = rows(data=None)
    empty = cache(data=None, scales=None)
    assert write(S=0, q=None, k=gone, v=gone, kc=empty, vc=empty, **none) == rp.ROPE_OK
    assert read(B=0, out=gone, c=empty, table=None, lengths=None) == rp.ROPE_OK
    assert read(cols=0, out=gone, c=empty, table=None, lengths=None) == rp.ROPE_OK
    assert read(out=gone, c=cache(pages=0, data=None, scales=None), table=None, lengths=None) == rp.ROPE_OK


def test_tensor_checks_of_the_binding():
    bf = torch.bfloat16
    k = torch.zeros(2, 5, 2, 16, dtype=bf)
    c = rp.rope_cache(3, 4, 2, 16, "int8", 8, device="cpu")
    slots = torch.zeros(2, 5, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU tensor"):
        rp.rope_cache_write(k, None, c, None, slots)
    empty = k[:0]
    for kw, err, text in [
            (dict(k=k[0]), ValueError, "4-D"), (dict(v=empty.float(), v_cache=c), TypeError, "share a dtype"),
            (dict(v=empty[:, :3], v_cache=c), ValueError, "tokens"), (dict(v=empty), ValueError, "go together"),
            (dict(k_cache=c.data), TypeError, "RopeCache"), (dict(slots=slots), ValueError, "slots"),
            (dict(slots=slots[:0].int()), ValueError, "slots"),
            (dict(positions=slots[:0], inv_freq=torch.ones(4), partial_slice=(0, 8)), ValueError, "float64"),
            (dict(positions=slots[:0].int(), inv_freq=torch.ones(4), partial_slice=(0, 8)), ValueError, "int64"),
            (dict(positions=slots[None, :0], inv_freq=torch.ones(4).double(), partial_slice=(0, 8)), ValueError, "pair_axes"),
            (dict(positions=slots[:0], inv_freq=torch.ones(3).double(), partial_slice=(0, 8)), ValueError, "frequencies"),
            (dict(rotary_mode="spiral"), ValueError, "rotary_mode")]:
        a = dict(k=empty, v=None, k_cache=c, v_cache=None, slots=slots[:0])
        a.update(kw)
        with pytest.raises(err, match=text):
            rp.rope_cache_write(**a)
    out, table, n = empty, torch.zeros(0, 3, dtype=torch.int32), torch.zeros(0, dtype=torch.int32)
    rp.rope_cache_read(out, c, table, n)
    for kw, err, text in [
            (dict(out=k[0]), ValueError, "4-D"), (dict(cache=None), TypeError, "RopeCache"),
            (dict(block_table=table.long()), ValueError, "block_table"), (dict(lengths=n.long()), ValueError, "lengths"),
            (dict(starts=n[None]), ValueError, "starts")]:
        a = dict(out=out, cache=c, block_table=table, lengths=n)
        a.update(kw)
        with pytest.raises(err, match=text):
            rp.rope_cache_read(**a)


def test_cache_objects():
    for fmt in rp.CACHE_FORMATS:
        c = rp.rope_cache(2, 3, 4, 32, fmt, 8 if fmt in ("e4m3", "int8", "int4") else None, device="cpu")
        assert (c.struct.format, c.struct.dim, c.struct.pages) == (rp.CACHE_FORMATS[fmt], 32, 2)
        assert c.group == (8 if c.scales is not None else 32)
        assert tuple(c.struct.strides) == tuple(s * c.data.element_size() for s in c.data.stride()[:3])
    d, sc = torch.zeros(2, 3, 4, 32, dtype=torch.int8), torch.zeros(2, 3, 4, 4)
    for data, scales, err in [(d.short(), sc, TypeError), (d[0], sc, ValueError), (d, None, TypeError),
                              (d, sc.double(), TypeError), (d, sc[:, :2], ValueError), (d, sc[..., :3], ValueError),
                              (d.transpose(2, 3), sc, ValueError), (d.float(), sc, ValueError),
                              (d, torch.zeros(2, 3, 4, 8)[..., ::2], ValueError)]:
        with pytest.raises(err):
            rp.RopeCache(data, scales)
    with pytest.raises(ValueError):
        rp.rope_cache(1, 1, 1, 32, "e5m2", device="cpu")
    with pytest.raises(ValueError):
        rp.rope_cache(1, 1, 1, 32, "int8", 5, device="cpu")
