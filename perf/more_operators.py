"""Measured cases of the operators between a layer's projections and its
attention over a paged cache.

Three families, each with a plain form (elementary torch operations in 32
bits) and the call a user makes of the library:

  norm       RMS norms of the heads of Q and K with the position rotation in
             the same pass: for serving, and as a training step with the
             gradients of Q, K and both weights
  reserve    pages of a paged cache given to growing sequences and taken back
             from ended ones, with the slots and positions of the new tokens
  attention  attention of new tokens over a paged cache held in 4 bits, from
             one token a sequence to chunks of a prompt

`own` selects the side; prepare() is the same for both.
"""
import math

import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # decoding 32 requests: Q and K as a fused projection leaves them,
        # normalised by heads and rotated
        dict(name="norm decode", kind="norm", train=False, B=32, S=1, hq=32, hk=8, D=128, start=0, end=128,
             mode="rotate_half", dtype="bf16", weight="bf16", table="bf16"),
        # two prompts of odd length
        dict(name="norm prompt", kind="norm", train=False, B=2, S=8191, hq=32, hk=4, D=128, start=0, end=128,
             mode="rotate_half", dtype="bf16", weight="f32", table="f32"),
        # training a grouped-query layer: forward, and backward to Q, K and
        # the weights
        dict(name="norm train", kind="norm", train=True, B=4, S=4096, hq=32, hk=8, D=128, start=0, end=128,
             mode="rotate_half", dtype="bf16", weight="bf16", table="bf16"),
        # training a smaller tower: heads of 80 lanes, a part of each rotated
        dict(name="norm train part", kind="norm", train=True, B=16, S=1025, hq=16, hk=16, D=80, start=0, end=48,
             mode="interleave", dtype="f16", weight="f32", table="f32"),
        # a decoding step's bookkeeping: a token each, a page for some
        dict(name="reserve decode", kind="reserve", B=256, S=1, page=16, cols=2048, most=8192, pool=300000,
             swap=False),
        # a step that ends half the sequences and admits prompts in their place
        dict(name="reserve prompts", kind="reserve", B=48, S=4096, page=16, cols=300, most=4096, pool=7000,
             swap=True),
        # one request on a small model
        dict(name="attention decode 1", kind="attention", B=1, S=1, hq=16, hk=4, D=64, Dv=64, L=1024, page=16,
             gk=64, gv=64, dtype="bf16"),
        # one request with a long context
        dict(name="attention decode long", kind="attention", B=1, S=1, hq=32, hk=8, D=128, Dv=128, L=131072, page=64,
             gk=128, gv=128, dtype="bf16"),
        # a full batch of requests, lengths ragged
        dict(name="attention decode 64", kind="attention", B=64, S=1, hq=32, hk=8, D=128, Dv=128, L=8192, page=16,
             gk=128, gv=128, dtype="bf16"),
        # five drafted tokens of each request to be verified, finer scales
        dict(name="attention verify", kind="attention", B=16, S=5, hq=40, hk=8, D=128, Dv=128, L=8000, page=32,
             gk=32, gv=32, dtype="f16"),
        # a chunk of three prompts behind what is cached
        dict(name="attention chunk", kind="attention", B=3, S=2039, hq=32, hk=8, D=128, Dv=128, L=6135, page=16,
             gk=128, gv=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm", "reserve", "attention", "attention", "attention"])
    dt = rng.choice(["bf16", "bf16", "f16"])
    if kind == "norm":
        D = rng.choice([64, 80, 96, 128, 128, 192, 256, 36])
        L = rng.choice([D, D, D // 2 // 4 * 4, D // 4 // 4 * 4])
        start = rng.choice([0, (D - L) // 8 * 8, D - L])
        mode = rng.choice(["rotate_half", "interleave"])
        if L % 8 == 0 and rng.random() < 0.2:
            mode = 4
        dt = rng.choice([dt, dt, "f32"])
        B, hq = rng.randrange(1, 33), rng.choice([1, 4, 8, 16, 24, 28, 32])
        S = max(1, min(_log(rng, 1, 16384), (1 << 26) // (B * hq * D)))
        return dict(kind=kind, train=rng.random() < 0.5, B=B, S=S, hq=hq, hk=rng.choice([h for h in (1, 4, 8, 16, 32) if
                    h <= max(1, hq)]), D=D, start=start, end=start + L, mode=mode, dtype=dt,
                    weight=rng.choice([dt, "f32"]), table=rng.choice([dt, "f32"]))
    if kind == "reserve":
        B, page = _log(rng, 1, 512), rng.choice([1, 16, 16, 32, 64, 128])
        swap = rng.random() < 0.5
        S = max(1, min(1 if rng.random() < 0.4 else _log(rng, 1, 4096), 180000 // B))
        most = _log(rng, S, max(S, 4096)) if swap else _log(rng, 1, 8192)
        cols = -(-most // page) + rng.randrange(1, 64)
        return dict(kind=kind, B=B, S=S, page=page, cols=cols, most=most, swap=swap,
                    pool=max(8, int(B * -(-most // page) * rng.uniform(0.9, 1.6))))
    D = rng.choice([64, 128, 128, 128, 96, 256, 80])
    Dv = rng.choice([D, D, D, 64, 128])
    gk = rng.choice([D, D] + [g for g in (32, 64, 16) if D % g == 0])
    gv = rng.choice([Dv, Dv] + [g for g in (32, 64, 16) if Dv % g == 0])
    hk = rng.choice([1, 2, 4, 8, 8])
    hq = hk * rng.choice([1, 2, 4, 4, 5, 7, 8])
    B = _log(rng, 1, 64)
    S = rng.choice([1, 1, 1, rng.randrange(2, 9), _log(rng, 9, 2039)])
    # of cached rows and of products no more than the largest listed cases
    L = max(S, min(_log(rng, S, 131072), (1 << 28) // (B * hk * max(D, Dv)),
                   int(3e10 / (B * S * hq * max(D, Dv)))))
    S = min(S, L)
    return dict(kind=kind, B=B, S=S, hq=hq, hk=hk, D=D, Dv=Dv, L=L, page=rng.choice([1, 16, 16, 32, 64, 128, 24]),
                gk=gk, gv=gv, dtype=dt)


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(case)
    if c["kind"] == "norm":
        return _prepare_norm(c, g)
    if c["kind"] == "reserve":
        return _prepare_reserve(c, g)
    return _prepare_attention(c, g)


def _prepare_norm(c, g):
    B, S, D, t = c["B"], c["S"], c["D"], TORCH[c["dtype"]]
    L = c["end"] - c["start"]
    pairs = L // 2
    c["half"] = 1 if c["mode"] == "interleave" else L // 2 if c["mode"] == "rotate_half" else L // c["mode"]
    i = torch.arange(pairs, dtype=torch.float64, device="cuda")
    c["inv_freq"] = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device="cuda"), -i / max(1, pairs))
    c["positions"] = torch.arange(S, device="cuda") + torch.randint(0, 32768, (B, 1), generator=g, device="cuda")
    w = TORCH[c["weight"]]
    c["wq"] = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(w)
    c["wk"] = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(w)
    # a fused projection's output: Q, K and V of a token beside each other,
    # some channels an order larger
    n = c["hq"] + 2 * c["hk"]
    qkv = torch.randn(B, S, n, D, generator=g, device="cuda")
    qkv[..., 5::16] *= 6
    qkv = qkv.to(t)
    c["q"], c["k"] = qkv[:, :, : c["hq"]], qkv[:, :, c["hq"]: c["hq"] + c["hk"]]
    if c["train"]:
        c["gq"] = torch.randn(B, S, c["hq"], D, generator=g, device="cuda").to(t)
        c["gk"] = torch.randn(B, S, c["hk"], D, generator=g, device="cuda").to(t)
        if own:
            for name in ("q", "k", "wq", "wk"):
                c[name] = c[name].detach().requires_grad_(True)
    return c


def _prepare_reserve(c, g):
    B, cols, page, pool = c["B"], c["cols"], c["page"], c["pool"]
    cpu = torch.Generator().manual_seed(g.initial_seed())
    if c["swap"]:
        # every second sequence is a running one, which ends; prompts of up
        # to S tokens come in the places between them
        lengths = torch.randint((c["most"] + 1) // 2, c["most"] + 1, (B,), generator=cpu)
        lengths[1::2] = 0
        counts = torch.randint((c["S"] + 1) // 2, c["S"] + 1, (B,), generator=cpu)
        counts[0::2] = -lengths[0::2]
    else:
        lengths = torch.randint(0, c["most"] + 1, (B,), generator=cpu)
        counts = torch.full((B,), c["S"])
    order = torch.randperm(pool, generator=cpu)
    table = torch.full((B, cols), -1)
    used = 0
    for b in range(B):
        n = -(-int(lengths[b]) // page)
        if used + n > pool:      # the pool was too small for this one
            lengths[b] = n = 0
            counts[b] = max(0, int(counts[b]))
        table[b, :n] = order[used: used + n]
        used += n
    free = torch.full((pool,), -1)
    free[: pool - used] = order[used:]
    c["table"] = table.to(torch.int32).cuda()
    c["lengths"] = lengths.to(torch.int32).cuda()
    c["counts"] = counts.to(torch.int32).cuda()
    c["free"] = free.to(torch.int32).cuda()
    c["free_count"] = torch.tensor([pool - used], dtype=torch.int32).cuda()
    c["slots"] = torch.zeros(B, c["S"], dtype=torch.int64, device="cuda")
    c["positions"] = torch.zeros(B, c["S"], dtype=torch.int64, device="cuda")
    c["granted"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    return c


def _int4(x, group):
    """Codes, two a byte, and scales of rows of x: the largest magnitude of a
    group takes code 7."""
    z = x.unflatten(-1, (-1, group))
    s = z.abs().amax(-1) / 7
    codes = (z / s[..., None]).round_().clamp_(-7, 7).to(torch.int8).flatten(-2)
    return ((codes[..., 0::2] & 15) | ((codes[..., 1::2] & 15) << 4)).view(torch.uint8), s


def _prepare_attention(c, g):
    B, S, L, page, hk = c["B"], c["S"], c["L"], c["page"], c["hk"]
    per = -(-L // page)
    c["pages"] = per * B + 3
    order = torch.randperm(c["pages"], generator=g, device="cuda")[: per * B].view(B, per)
    c["table"] = order.to(torch.int32).contiguous()
    k = torch.randn(c["pages"], page, hk, c["D"], generator=g, device="cuda")
    k[..., 5::16] *= 4
    c["k_data"], c["k_scales"] = _int4(k, c["gk"])
    del k
    v = torch.randn(c["pages"], page, hk, c["Dv"], generator=g, device="cuda")
    c["v_data"], c["v_scales"] = _int4(v, c["gv"])
    del v
    mix = torch.randperm(B, generator=g, device="cuda")
    lengths, counts = _attention_sizes(c)
    c["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")[mix].contiguous()
    c["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")[mix].contiguous() if S > 1 else None
    t = TORCH[c["dtype"]]
    c["q"] = torch.randn(B, S, c["hq"], c["D"], generator=g, device="cuda").to(t)
    c["out"] = torch.zeros(B, S, c["hq"], c["Dv"], dtype=t, device="cuda")
    if own:
        import transformer_positional_encoding_amd as rp
        c["kc"], c["vc"] = rp.RopeCache(c["k_data"], c["k_scales"]), rp.RopeCache(c["v_data"], c["v_scales"])
        n = rp.rope_cache_attention_workspace(B, S, c["hq"], hk, c["Dv"])
        c["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return c


def _attention_sizes(c):
    """Tokens cached and tokens new of each sequence: spread over the upper
    halves of what the case allows."""
    B, S, L = c["B"], c["S"], c["L"]
    counts = [S - b * (S // 2) // B for b in range(B)]
    return [max(counts[b], L - b * (L // 2) // B) for b in range(B)], counts


# -------------------------------------------------------------- plain forms


def _cos_sin(c):
    """(B, S, 1, pairs) cos and sin of position times frequency, the angle in
    64 bits, rounded once to the table's type."""
    th = c["positions"].double()[..., None] * c["inv_freq"]
    t = TORCH[c["table"]]
    return th.cos().to(t).float()[:, :, None, :], th.sin().to(t).float()[:, :, None, :]


def _rotate(x, cos, sin, c):
    """x (fp32, last dimension the head) with its slice rotated."""
    h, s, e = c["half"], c["start"], c["end"]
    if e == s:
        return x
    z = x[..., s:e].unflatten(-1, (-1, 2, h))
    p, q = z[..., 0, :], z[..., 1, :]
    cos, sin = cos.unflatten(-1, (-1, h)), sin.unflatten(-1, (-1, h))
    turned = torch.stack([p * cos - q * sin, q * cos + p * sin], dim=-2)
    return torch.cat([x[..., :s], turned.flatten(-3), x[..., e:]], dim=-1)


EPS = 1e-6


def _plain_norm(c):
    cos, sin = _cos_sin(c)
    t, w = TORCH[c["dtype"]], TORCH[c["weight"]]
    got, grads, wgrads = [], [], []
    for x, weight, grad in ((c["q"], c["wq"], c.get("gq")), (c["k"], c["wk"], c.get("gk"))):
        x, weight = x.detach().float(), weight.detach().float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        n = x * r
        got.append(_rotate(n * weight, cos, sin, c).to(t))
        if grad is not None:
            back = _rotate(grad.float(), cos, -sin, c)
            wgrads.append((back * n).sum((0, 1, 2)).to(w))
            back = back * weight
            grads.append((r * (back - n * (back * n).mean(-1, keepdim=True))).to(t))
    return tuple(got + grads + wgrads)


def _plain_reserve(c):
    page, S, pool, cols = c["page"], c["S"], c["free"].numel(), c["cols"]
    old, n = c["lengths"].long(), c["counts"].long()
    column = torch.arange(cols, device="cuda")
    had = (old + page - 1) // page
    # ended and shortened sequences give their pages back, in order
    kept = torch.where(n < 0, (old + n).clamp(min=0), old)
    keeps = (kept + page - 1) // page
    gives = had - keeps
    first = gives.cumsum(0) - gives
    free_count = c["free_count"].long()
    leaving = (column >= keeps[:, None]) & (column < had[:, None])
    to = free_count + first[:, None] + column - keeps[:, None]
    pushed = torch.cat([c["free"], c["free"][:1]])          # one place more, for what does not go anywhere
    pushed.scatter_(0, torch.where(leaving & (to < pool), to, pool).flatten(), c["table"].flatten())
    free = pushed[:pool]
    count = (free_count + gives.sum()).clamp(max=pool)
    # growing ones take pages from the end of the list, in order, while it lasts
    new = old + n.clamp(min=0)
    fits = (n > 0) & (n <= S) & (new <= cols * page)
    needs = torch.where(fits, (new + page - 1) // page - had, 0)
    last = needs.cumsum(0)
    given = fits & ((needs == 0) | (last <= count))
    index = count - 1 - (last - needs)[:, None] - (column - had[:, None])
    taking = given[:, None] & (column >= had[:, None]) & (column < (had + needs)[:, None])
    table = torch.where(leaving, -1, c["table"])
    table = torch.where(taking, free[index.clamp(0, pool - 1)], table)
    count = count - torch.where(given, needs, 0).sum()
    granted = torch.where(given, n, kept - old)
    # the new tokens' places
    s = torch.arange(S, device="cuda")
    positions = torch.minimum(old, kept)[:, None] + s
    own_page = table.gather(1, (positions // page).clamp(max=cols - 1)).long()
    slots = torch.where((s < granted[:, None]) & (own_page >= 0), own_page * page + positions % page, -1)
    c["table"].copy_(table)
    c["lengths"].copy_(old + granted)
    c["free"].copy_(free)
    c["free_count"].copy_(count)
    c["slots"].copy_(slots)
    c["positions"].copy_(positions)
    c["granted"].copy_(granted)


def _values(data, scales):
    """Lanes of codes, two a byte, times the scales of their groups."""
    b = data.view(torch.int8)
    v = torch.stack([(b << 4) >> 4, b >> 4], dim=-1).flatten(-2).float()
    return (v.unflatten(-1, (scales.shape[-1], -1)) * scales[..., None]).flatten(-2)


def _plain_attention(c):
    B, S, hq, hk, L = c["B"], c["S"], c["hq"], c["hk"], c["L"]
    rep = hq // hk
    token = torch.arange(L, device="cuda")
    at = c["table"].long()[:, token // c["page"]] * c["page"] + token % c["page"]
    k = _values(c["k_data"].flatten(0, 1)[at], c["k_scales"].flatten(0, 1)[at])     # (B, L, hk, D)
    k = k.permute(0, 2, 3, 1).contiguous()
    counts = c["counts"].long() if S > 1 else torch.ones_like(c["lengths"]).long()
    at_row = c["lengths"].long()[:, None] - counts[:, None] + torch.arange(S, device="cuda")
    q = c["q"].float().view(B, S, hk, rep, -1).permute(0, 2, 1, 3, 4).reshape(B, hk, S * rep, -1).contiguous()
    x = torch.matmul(q, k) / math.sqrt(c["D"])
    del k
    hidden = (token > at_row[..., None]).repeat_interleave(rep, dim=1)[:, None]     # (B, 1, S*rep, L)
    x.masked_fill_(hidden, -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    v = _values(c["v_data"].flatten(0, 1)[at], c["v_scales"].flatten(0, 1)[at]).permute(0, 2, 1, 3).contiguous()
    y = torch.matmul(x, v) / torch.where(total > 0, total, 1)
    y = y.view(B, hk, S, rep, -1).permute(0, 2, 1, 3, 4).reshape(B, S, hq, -1)
    live = (torch.arange(S, device="cuda") < counts[:, None])[..., None, None]
    c["out"].copy_(torch.where(live, y.to(c["out"].dtype), c["out"]))


# ---------------------------------------------------------------------- run


def run(c):
    if own:
        import transformer_positional_encoding_amd as rp
    if c["kind"] == "norm":
        if not own:
            return _plain_norm(c)
        how = (c["positions"], c["inv_freq"], c["mode"], (c["start"], c["end"]))
        t = TORCH[c["table"]]
        if not c["train"]:
            return rp.rope_qk_norm_fwd(c["q"], c["k"], c["wq"], c["wk"], *how, eps=EPS, table_dtype=t)
        ins = (c["q"], c["k"], c["wq"], c["wk"])
        y = rp.qk_norm_rotary(*ins, *how, eps=EPS, table_dtype=t)
        return tuple(y) + torch.autograd.grad(y, ins, (c["gq"], c["gk"]))
    if c["kind"] == "reserve":
        if own:
            rp.rope_cache_reserve(c["table"], c["lengths"], c["counts"], c["free"], c["free_count"], c["page"],
                                  slots=c["slots"], positions=c["positions"], granted=c["granted"])
        else:
            _plain_reserve(c)
        if c["swap"]:      # the next step ends what came in, and the other way round
            c["counts"].neg_()
        return tuple(c[k] for k in RESERVED)
    if own:
        rp.rope_cache_attention(c["q"], c["kc"], c["vc"], c["table"], c["lengths"], counts=c["counts"], out=c["out"],
                                workspace=c["workspace"])
    else:
        _plain_attention(c)
    return c["out"]


RESERVED = ("slots", "positions", "granted", "table", "lengths", "free", "free_count")


def work(case):
    c = case
    if c["kind"] == "norm":
        es, ws = SIZE[c["dtype"]], SIZE[c["weight"]]
        lanes = c["B"] * c["S"] * (c["hq"] + c["hk"]) * c["D"]
        turned = lanes // c["D"] * (c["end"] - c["start"])
        total = 2 * lanes * es + 8 * c["B"] * c["S"] + 2 * c["D"] * ws
        flops = 4 * lanes + 3 * turned
        if c["train"]:
            # backward: the input and the incoming gradient read, the gradient written
            total += 3 * lanes * es + 4 * c["D"] * ws
            flops += 11 * lanes + 3 * turned
        return dict(bytes=total, flops=flops)
    if c["kind"] == "reserve":
        growing = c["B"] * (0.5 if c["swap"] else 1) * c["S"] * (0.75 if c["swap"] else 1)
        return dict(bytes=c["B"] * (16 * c["S"] + 16) + 2 * 4 * 2 * growing / c["page"], flops=4 * c["B"] * c["S"])
    rep = c["hq"] // c["hk"]
    lengths, counts = _attention_sizes(c)
    cached = sum(lengths) * c["hk"]
    lanes = sum(counts) * c["hq"] * (c["D"] + c["Dv"])
    # each new token sees what is cached up to itself
    seen = sum(n * m - n * (n - 1) // 2 for m, n in zip(lengths, counts)) * c["hk"] * rep
    return dict(bytes=cached * ((c["D"] + c["Dv"]) / 2 + 4 * (c["D"] // c["gk"] + c["Dv"] // c["gv"]))
                + lanes * SIZE[c["dtype"]] + sum(lengths) / c["page"] * 4, flops=2 * seen * (c["D"] + c["Dv"]))


# ---------------------------------------------- the definitions in 64 bits


def _norm64(c):
    """Lane by lane: y_j = n_j cos + sign_j n_p(j) sin with n = x w / rms(x),
    and the products with the transposed Jacobian."""
    D, h, s, e = c["D"], c["half"], c["start"], c["end"]
    lane = torch.arange(D, device="cuda")
    j = lane - s
    inside = (j >= 0) & (lane < e)
    up = (j // h) % 2 == 1
    other = torch.where(inside, torch.where(up, lane - h, lane + h), lane)
    sign = torch.where(up, 1.0, -1.0).double() * inside
    pair = (j // (2 * h) * h + j % h)[inside] if e > s else None
    th = c["positions"].double()[..., None] * c["inv_freq"]
    t = TORCH[c["table"]]
    ca = torch.ones(c["B"], c["S"], 1, D, dtype=torch.float64, device="cuda")
    sa = torch.zeros_like(ca)
    if pair is not None:
        ca[:, :, 0, s:e] = torch.cos(th).to(t).double()[..., pair]
        sa[:, :, 0, s:e] = torch.sin(th).to(t).double()[..., pair]
    got, grads, wgrads = [], [], []
    for x, w, grad in ((c["q"], c["wq"], c.get("gq")), (c["k"], c["wk"], c.get("gk"))):
        x, w = x.detach().double(), w.detach().double()
        rms = torch.sqrt(torch.square(x).sum(-1, keepdim=True) / D + EPS)
        z = x / rms * w
        got.append(z * ca + sign * z[..., other] * sa)
        if grad is None:
            continue
        d = grad.double()
        # lane j of z meets lane j of y by cos_j, and lane p(j) by sign_p(j) sin_p(j)
        dz = d * ca + (sign * d * sa)[..., other]
        wgrads.append((dz * x / rms).sum(dim=(0, 1, 2)))
        along = (dz * w * x).sum(-1, keepdim=True) / D
        grads.append(dz * w / rms - x * along / rms ** 3)
    return tuple(got + grads + wgrads)


def _reserve_exact(c):
    """Sequence by sequence on the host."""
    page, S, cols = c["page"], c["S"], c["cols"]
    table, lengths, counts = c["table"].tolist(), c["lengths"].tolist(), c["counts"].tolist()
    free, count = c["free"].tolist(), c["free_count"].item()
    B, pool = len(lengths), len(free)
    granted, start = [0] * B, list(lengths)
    pages = lambda n: -(-n // page)  # noqa: E731
    for b in range(B):
        if counts[b] < 0:
            left = max(0, lengths[b] + counts[b])
            for i in range(pages(left), pages(lengths[b])):
                if count < pool:
                    free[count] = table[b][i]
                    count += 1
                table[b][i] = -1
            granted[b] = left - lengths[b]
            start[b] = left
    out_of_pages = False
    for b in range(B):
        n = counts[b]
        if n <= 0 or n > S or lengths[b] + n > cols * page:
            continue
        have, want = pages(lengths[b]), pages(lengths[b] + n)
        if want > have:
            out_of_pages = out_of_pages or want - have > count
            if out_of_pages:
                continue
            for i in range(have, want):
                count -= 1
                table[b][i] = free[count]
        granted[b] = n
    slots = [[-1] * S for _ in range(B)]
    for b in range(B):
        for s in range(max(0, granted[b])):
            t = start[b] + s
            slots[b][s] = table[b][t // page] * page + t % page
    like = lambda v, k: torch.tensor(v, dtype=c[k].dtype, device="cuda")  # noqa: E731
    return (like(slots, "slots"), like([[start[b] + s for s in range(S)] for b in range(B)], "positions"),
            like(granted, "granted"), like(table, "table"), like([m + d for m, d in zip(lengths, granted)], "lengths"),
            like(free, "free"), like([count], "free_count"))


def _codes64(data):
    v = data.to(torch.int64)
    both = torch.stack([v % 16, v // 16], dim=-1).reshape(*v.shape[:-1], -1)
    return torch.where(both > 7, both - 16, both).double()


def _attention64(c):
    """Sequence by sequence, head by head, rows a few at a time."""
    rep = c["hq"] // c["hk"]
    got = c["out"].double()
    for b in range(c["B"]):
        m = int(c["lengths"][b])
        n = int(c["counts"][b]) if c["counts"] is not None else c["S"]
        t = torch.arange(m, device="cuda")
        page, off = c["table"][b].long()[t // c["page"]], t % c["page"]
        for h in range(c["hk"]):
            sk, sv = c["k_scales"][page, off, h].double(), c["v_scales"][page, off, h].double()
            k = _codes64(c["k_data"][page, off, h]) * sk.repeat_interleave(c["gk"], dim=-1)
            v = _codes64(c["v_data"][page, off, h]) * sv.repeat_interleave(c["gv"], dim=-1)
            for lo in range(0, n, 512):
                hi = min(n, lo + 512)
                q = c["q"][b, lo:hi, h * rep:(h + 1) * rep].double()
                score = torch.tensordot(q, k, dims=([2], [1])) / c["D"] ** 0.5
                seen = t[None, :] <= (m - n + torch.arange(lo, hi, device="cuda"))[:, None]
                p = torch.softmax(torch.where(seen[:, None], score, -math.inf), dim=-1)
                got[b, lo:hi, h * rep:(h + 1) * rep] = torch.tensordot(p, v, dims=([2], [0]))
    return got


def exact(case, seed):
    c = prepare(case, seed)
    return {"norm": _norm64, "reserve": _reserve_exact, "attention": _attention64}[c["kind"]](c)
