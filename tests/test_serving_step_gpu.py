"""A serving step as a program runs it: pages, slots and positions of the new
tokens, norms and rotation of Q and K, K and V written in 4 bits, and attention
over the cache; prompts and decoding steps of requests that come and go, and a
captured decoding step. Each operator's result is checked against its
definition applied to what the step itself fed it."""
import random

import pytest
import torch

import transformer_positional_encoding_amd as rp
from axes_refs import pair_tables
from cache_refs import encode
from serving_refs import attention64, half_step, norm64, reserve

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HQ, HK, D, PAGE, COLS = 6, 2, 128, 16, 12


class Server:
    def __init__(self, B, group, seed):
        g = torch.Generator().manual_seed(seed)
        self.B, self.group, self.g = B, group, g
        pool = B * 8
        self.table = torch.full((B, COLS), -1, dtype=torch.int32).cuda()
        self.lengths = torch.zeros(B, dtype=torch.int32).cuda()
        self.free = torch.randperm(pool, generator=g).to(torch.int32).cuda()
        self.count = torch.tensor([pool], dtype=torch.int32).cuda()
        self.kc, self.vc = (rp.rope_cache(pool, PAGE, HK, D, "int4", group) for _ in range(2))
        self.wq, self.wk = ((1 + 0.3 * torch.randn(D, generator=g)).cuda() for _ in range(2))
        self.f = rp.rope_inv_freq(D, 10000.0, "cuda")
        self.scratch = dict(workspace=torch.empty(rp.rope_cache_attention_workspace(B, 1, HQ, HK, D), dtype=torch.uint8,
                                                  device="cuda"))

    def step(self, qkv, counts, out, **kw):
        S = qkv.shape[1]
        slots, positions, granted = rp.rope_cache_reserve(self.table, self.lengths, counts, self.free, self.count, PAGE, tokens=S)
        q, k = rp.rope_qk_norm_fwd(qkv[:, :, :HQ], qkv[:, :, HQ:HQ + HK], self.wq, self.wk, positions, self.f, "rotate_half",
                                   (0, D))
        rp.rope_cache_write(k, qkv[:, :, HQ + HK:], self.kc, self.vc, slots)
        rp.rope_cache_attention(q, self.kc, self.vc, self.table, self.lengths, counts=granted, out=out, **kw)
        return slots, positions, granted, q, k

    def state(self):
        return [t.cpu().tolist() for t in (self.table, self.lengths)] + [self.free.cpu().tolist(), self.count.item()]


def qkv_of(s, S):
    x = torch.randn(s.B, S, HQ + 2 * HK, D, generator=s.g)
    x[..., 3::17] *= 5
    return x.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("group", [128, 32])
def test_requests_come_and_go(group):
    rng = random.Random(group)
    s = Server(7, group, 3)
    for i in range(8):
        S = [40, 1, 1, 25, 1, 3, 60, 1][i]
        lengths = s.lengths.tolist()
        counts = [rng.randrange(1, S + 1) if n == 0 or S == 1 else rng.choice([-n, rng.randrange(0, S + 1)]) for n in lengths]
        before = s.state()
        qkv, out = qkv_of(s, S), torch.zeros(s.B, S, HQ, D, dtype=torch.bfloat16).cuda()
        slots, positions, granted, q, k = s.step(qkv, torch.tensor(counts, dtype=torch.int32).cuda(), out)
        want = reserve(before[0], before[1], counts, before[2], before[3], PAGE, S)
        got = [t.tolist() for t in (slots, positions, granted)] + s.state()
        assert got == list(want[:6]) + [want[6]]
        cos, sin = pair_tables(positions[None], s.f, (0,) * (D // 2), "bf16")
        for y, x, w in ((q, qkv[:, :, :HQ], s.wq), (k, qkv[:, :, HQ:HQ + HK], s.wk)):
            z, size = norm64(x.cpu(), w.cpu(), 1e-6, cos, sin, "rotate_half", (0, D))
            lim = (D / 2 + 16) * U * size
            assert bool(((y.cpu().double() - z).abs() <= lim + half_step(y.dtype, z.abs() + lim)).all())
        # what the write put to the slots is the definition's codes
        live = slots.cpu() >= 0
        at = slots.cpu()[live]
        for cache, x in ((s.kc, k), (s.vc, qkv[:, :, HQ + HK:])):
            codes, scales = encode(x.cpu()[live].float(), "int4", group)
            packed = codes.to(torch.int64) & 15
            packed = packed[..., 0::2] | packed[..., 1::2] << 4
            assert torch.equal(cache.data.cpu()[at // PAGE, at % PAGE].long(), packed)
            assert torch.equal(cache.scales.cpu()[at // PAGE, at % PAGE].double(), scales)
        z, lim = attention64(q.cpu(), torch.zeros_like(out.cpu()), *((c.data.cpu(), c.scales.cpu()) for c in (s.kc, s.vc)),
                             s.table.cpu(), s.lengths.cpu(), granted.cpu(), D ** -0.5, True)
        lim = lim + torch.where(lim > 0, half_step(out.dtype, z.abs() + lim), torch.zeros_like(lim))
        assert bool(((out.cpu().double() - z).abs() <= lim).all()), f"step {i}"


def test_a_captured_decoding_step():
    a, b = Server(5, 128, 4), Server(5, 128, 4)
    ones = torch.ones(5, dtype=torch.int32).cuda()
    prompt = qkv_of(a, 30)
    for s in (a, b):
        s.step(prompt, torch.tensor([30, 4, 17, 0, 16], dtype=torch.int32).cuda(),
               torch.zeros(5, 30, HQ, D, dtype=torch.bfloat16).cuda())
    qkv = qkv_of(a, 1)
    outs = [torch.zeros(5, 1, HQ, D, dtype=torch.bfloat16).cuda() for _ in range(2)]
    for s, out in zip((a, b), outs):
        s.step(qkv, ones, out, **s.scratch)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(qkv, ones, outs[0], **a.scratch)
    for i in range(20):          # pages are taken on the way
        qkv.copy_(qkv_of(a, 1))
        if i == 9:               # one request ends, its place is taken up later
            ones[2] = -1000
        if i == 12:
            ones[2] = 1
        graph.replay()
        torch.cuda.synchronize()
        b.step(qkv, ones, outs[1], **b.scratch)
        torch.cuda.synchronize()
        assert torch.equal(*outs) and a.state() == b.state()
        assert torch.equal(a.kc.data, b.kc.data) and torch.equal(a.vc.scales, b.vc.scales)


def test_two_servers_on_two_streams():
    pairs = [(Server(4, 64, s), Server(4, 64, s)) for s in (5, 6)]
    ins = [qkv_of(p[0], 20) for p in pairs]
    counts = torch.tensor([20, 3, 0, 11], dtype=torch.int32).cuda()
    outs = [[torch.zeros(4, 20, HQ, D, dtype=torch.bfloat16).cuda() for _ in p] for p in pairs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    for (s, _), x, o, st in zip(pairs, ins, outs, streams):
        with torch.cuda.stream(st):
            s.step(x, counts, o[0])
    torch.cuda.synchronize()
    for (_, s), x, o in zip(pairs, ins, outs):
        s.step(x, counts, o[1])
        torch.cuda.synchronize()
        assert torch.equal(*o)
