"""Every refusal of the projection with low-rank adapters (no GPU)."""
import ctypes

import pytest
import torch

import transformer_positional_encoding_amd as rp

FAKE = 1 << 24
I4 = ctypes.c_int64 * 4
I2 = ctypes.c_int64 * 2
NULL, BAD, NO = rp.ROPE_ERR_NULLPTR, rp.ROPE_ERR_INVALID, rp.ROPE_ERR_UNSUPPORTED


def call(**kw):
    a = dict(y=FAKE, ydt=2, x=FAKE * 2, w=FAKE * 3, dt=2, shape=(1, 6, 2, 64), K=128, la=FAKE * 4, lb=FAKE * 5,
             ids=FAKE * 6, scales=None, count=3, rank=16, lora=True, r=FAKE * 7, rshape=(1, 6, 1, 64), rst=(0, 64, 0, 1),
             tdt=2, mode=1, sl=(0, 64), ws=FAKE * 8, wsb=6 * 16 * 4)
    a.update(kw)
    lora = rp.RopeLora(a["la"], a["lb"], a["ids"], a["scales"], a["count"], a["rank"]) if a["lora"] else None
    sh = None if a["shape"] is None else I4(*a["shape"])
    return rp.library().rope_proj_lora_fwd(a["y"], a["ydt"], a["x"], a["w"], a["dt"], sh, a["K"], lora, a["r"],
                                           I4(*a["rshape"]), I4(*a["rst"]), a["r"], I4(*a["rshape"]), I4(*a["rst"]),
                                           a["tdt"], a["mode"], I2(*a["sl"]), a["ws"], a["wsb"], None)


@pytest.mark.parametrize("change, status, text", [
    (dict(shape=None), NULL, "x_shape"), (dict(ydt=1), BAD, "y must have"), (dict(dt=0), BAD, "bf16 or fp16"),
    (dict(K=-1), BAD, "K is negative"), (dict(K=96), NO, "multiple of 64"), (dict(shape=(1, 6, 2, 40), sl=(0, 40)), NO, "head"),
    (dict(y=None), NULL, "y is NULL"), (dict(x=None), NULL, "x is NULL"), (dict(w=None), NULL, "w is NULL"),
    (dict(x=FAKE * 2 + 8), BAD, "16-byte"), (dict(y=FAKE * 2), BAD, "overlaps"),
    (dict(lora=False), NULL, "lora is NULL"), (dict(count=-1), BAD, "negative"), (dict(rank=-8), BAD, "negative"),
    (dict(rank=12), BAD, "multiple of 8"), (dict(rank=136), NO, "128"),
    (dict(la=None), NULL, "a is NULL"), (dict(lb=None), NULL, "b is NULL"), (dict(ids=None), NULL, "adapters"),
    (dict(ws=None), NULL, "workspace"), (dict(la=FAKE * 4 + 2), BAD, "16-byte"), (dict(lb=FAKE * 5 + 8), BAD, "16-byte"),
    (dict(ws=FAKE * 8 + 4), BAD, "16-byte"), (dict(ids=FAKE * 6 + 2), BAD, "aligned"),
    (dict(scales=FAKE * 6 + 1), BAD, "aligned"), (dict(wsb=6 * 16 * 4 - 1), BAD, "needs 384"),
    (dict(count=1 << 31), BAD, "too many"), (dict(K=1 << 62), BAD, "64 bits"),
    (dict(K=64 << 20, shape=(1, 64, 1, 64), sl=(0, 0)), NO, "2^31"),
    (dict(r=None), NULL, "r1"), (dict(rshape=(1, 6, 1, 32)), BAD, "r1"), (dict(mode=7), BAD, "mode"),
])
def test_refusals(change, status, text):
    assert call(**change) == status, rp.last_error()
    assert text in rp.last_error()


def test_an_empty_call_reads_no_pointer():
    assert call(shape=(1, 0, 2, 64), y=None, x=None, w=None, lora=False, r=None, ws=None, wsb=0) == rp.ROPE_OK


def test_workspace_sizes():
    assert rp.rope_proj_lora_workspace(10, 64, 8) == 320
    # past 64 tokens also their order, each adapter's filled up to 32 rows
    assert 100 * 8 * 4 + 32 * 100 * 4 < rp.rope_proj_lora_workspace(100, 64, 8) < 100 * 8 * 4 + 33 * 100 * 4 + 4096
    for M, K, R in ((0, 64, 8), (10, 0, 8), (10, 64, 0), (10, 64, 129), (-1, 64, 8)):
        assert rp.rope_proj_lora_workspace(M, K, R) == 0


def test_tensor_checks_of_the_binding():
    bf = torch.bfloat16
    x, w = torch.zeros(0, 128, dtype=bf), torch.zeros(128, 128, dtype=bf)
    a, b = torch.zeros(3, 16, 128, dtype=bf), torch.zeros(3, 128, 16, dtype=bf)
    ids, r = torch.zeros(0, dtype=torch.int32), torch.zeros(1, 0, 1, 64, dtype=bf)
    ok = dict(x=x, w=w, a=a, b=b, adapters=ids, r1=r, r2=r, heads=2, partial_slice=(0, 64))
    for kw, err, text in [
            (dict(a=None), TypeError, "a must be"), (dict(a=a[0]), ValueError, "rank"), (dict(a=a[:2]), ValueError, "count"),
            (dict(b=b.transpose(1, 2)), ValueError, "rank"), (dict(a=a.float()), ValueError, "dtype"),
            (dict(adapters=ids.long()), ValueError, "int32"), (dict(adapters=torch.zeros(2, dtype=torch.int32)), ValueError, "token"),
            (dict(scales=torch.ones(3).double()), ValueError, "scales"), (dict(scales=torch.ones(2)), ValueError, "scales"),
            (dict(heads=3), ValueError, "heads"), (dict(out=torch.zeros(1, 1, 2, 64, dtype=bf)), ValueError, "out"),
            (dict(rotary_mode="spiral"), ValueError, "rotary_mode"), (dict(x=torch.zeros(128)), ValueError, "x must"),
            (dict(w=torch.zeros(128, 256, dtype=bf)[:, ::2]), ValueError, "contiguous"), (dict(), ValueError, "GPU")]:
        with pytest.raises(err, match=text):
            rp.rope_proj_lora_fwd(**dict(ok, **kw))
