"""The definitions in 64 bits of head norms with their rotation, of a cache's
page bookkeeping and of attention over a cache in 4 bits, with the limits that
arithmetic in fp32 and one rounding keep (CPU tensors)."""
from __future__ import annotations

import torch

from axes_refs import rotate64
from cache_refs import decode_codes

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype, v):
    """Most that rounding v to dtype moves it: half a unit of 2^-p of it, or of
    the least normal's."""
    i = torch.finfo(dtype)
    return i.eps / 2 * torch.clamp(v.abs(), min=i.tiny)


def turned64(x, cos, sin, mode, sl, back=False):
    """rotate64 with the size of lanes outside the slice, |x|."""
    y, size = rotate64(x, cos, sin, mode, sl, back)
    size[..., :sl[0]], size[..., sl[1]:] = x[..., :sl[0]].abs(), x[..., sl[1]:].abs()
    return y, size


def norm64(x, w, eps, cos, sin, mode, sl):
    """(y, limit's size): the normalised and rotated rows and the sum of the
    magnitudes that make each lane."""
    x = x.double()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    z = n if w is None else n * w.double()
    return turned64(z, cos, sin, mode, sl)


def norm_back64(x, w, eps, dy, cos, sin, mode, sl):
    """dx, dw and the sizes of what they are sums of. dx = r (g w - n mean(g w n)),
    g the gradient turned back."""
    x = x.double()
    D = x.shape[-1]
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n = x * r
    g, size = turned64(dy.double(), cos, sin, mode, sl, back=True)
    ww = torch.ones(D, dtype=torch.float64) if w is None else w.double()
    m = (g * ww * n).sum(-1, keepdim=True) / D
    dx = r * (g * ww - n * m)
    dx_size = r * (size * ww.abs() + n.abs() * (size * ww.abs() * n.abs()).sum(-1, keepdim=True) / D)
    return dx, (g * n).sum((0, 1, 2)), dx_size, (size * n.abs()).sum((0, 1, 2))


def reserve(table, lengths, counts, free, count, page, S):
    """Sequence by sequence, on lists; returns (slots, positions, granted,
    table, lengths, free, count)."""
    table, free = [list(r) for r in table], list(free)
    lengths, B, cap = list(lengths), len(lengths), len(free)
    cols = len(table[0]) if B else 0
    pages = lambda n: -(-n // page)  # noqa: E731
    count = min(max(count, 0), cap)
    sound = [0 <= n <= cols * page for n in lengths]
    granted, start = [0] * B, [max(0, n) for n in lengths]
    for b in range(B):
        if sound[b] and counts[b] < 0:
            kept = max(0, lengths[b] + counts[b])
            for c in range(pages(kept), pages(lengths[b])):
                if count < cap:
                    free[count] = table[b][c]
                    count += 1
                table[b][c] = -1
            granted[b], start[b] = kept - lengths[b], kept
    have, asked = count, 0
    for b in range(B):
        n = counts[b]
        if not sound[b] or not 0 < n <= S or lengths[b] + n > min(cols * page, 2 ** 31 - 1):
            continue
        need = pages(lengths[b] + n) - pages(lengths[b])
        asked += need
        if need and asked > have:
            continue
        for c in range(pages(lengths[b]), pages(lengths[b] + n)):
            count -= 1
            table[b][c] = free[count]
        granted[b] = n
    slots = [[-1] * S for _ in range(B)]
    for b in range(B):
        for s in range(max(0, granted[b])):
            p = table[b][(start[b] + s) // page]
            if p >= 0:
                slots[b][s] = p * page + (start[b] + s) % page
    positions = [[start[b] + s for s in range(S)] for b in range(B)]
    return slots, positions, granted, table, [n + g for n, g in zip(lengths, granted)], free, count


def cached_rows(data, scales, table_row, tokens, head):
    """(values (tokens, dim), magnitudes' scale per lane, which tokens are
    there) of one sequence and head."""
    pages, page = data.shape[:2]
    t = torch.arange(tokens)
    p = table_row[t // page].long()
    there = (p >= 0) & (p < pages)
    p = torch.where(there, p, torch.zeros_like(p))
    codes = decode_codes(data[p, t % page, head])
    s = scales[p, t % page, head].double().repeat_interleave(codes.shape[-1] // scales.shape[-1], -1)
    return codes * s, s, there


def attention64(q, out, k, v, table, lengths, counts, scale, causal):
    """(out, limit) of attention over caches k and v, (data, scales) each. out:
    what the rows that are not computed hold. The limit, before the rounding to
    out's type, with u = 2^-24:
      scores: the products of q with codes are exact. Sums of D products with
      codes that may be counted from -24 (magnitudes up to 31, and 24 |q| more
      to start from) round D + 8 times at most: |x| is off by d = (D + 8) u
      scale sum_j 56 |q_j| s_j, with the few roundings after it 8 u |x| more;
      exp of it is off by the factor exp(d + ...) < 1 + 2 (d + 8 u |x|) for
      values below 1, and so is their sum;
      a weight times v's scale may be rounded to 11 bits, 2^-11, or where it is
      below 2^-14 of the row's largest by 2^-25 of that or its next power of
      two, 2^-24;
      sums of T terms round T + 8 times.
    Each enters with sum |p v| / l, the rounding of small weights with the
    number of tokens times the largest |p v|."""
    q, got = q.double(), out.double().clone()
    lim = torch.zeros_like(got)
    B, S, H, D = q.shape
    heads = k[0].shape[2]
    rep = H // heads
    page, cols = k[0].shape[1], table.shape[1]
    u = 2.0 ** -24
    for b in range(B):
        n = S if counts is None else min(max(int(counts[b]), 0), S)
        length = max(0, int(lengths[b]))
        T = min(length, cols * page) if page else 0
        first = int(lengths[b]) - n
        got[b, :n] = 0
        if T == 0 or n == 0:
            continue
        for h in range(heads):
            kr, ks, there = cached_rows(*k, table[b], T, h)
            vr, vs, _ = cached_rows(*v, table[b], T, h)
            rows = q[b, :n, h * rep:(h + 1) * rep]                      # (n, rep, D)
            x = (rows.reshape(n * rep, D) @ kr.T).view(n, rep, T) * scale
            d = (D + 8) * u * scale * 56 * (rows.abs().reshape(n * rep, D) @ ks.T).view(n, rep, T)
            seen = there[None, :].expand(n, T)
            if causal:
                seen = seen & (torch.arange(T)[None] <= first + torch.arange(n)[:, None])
            x = torch.where(seen[:, None], x, torch.full_like(x, -float("inf")))
            m = x.amax(-1, keepdim=True)
            m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
            p = torch.exp(x - m)
            l = p.sum(-1, keepdim=True)
            l = torch.where(l > 0, l, torch.ones_like(l))
            off = torch.where(p > 0, 2 * (d + 8 * u * (x.abs() + m.abs())), torch.zeros_like(p)).amax(-1, keepdim=True)
            weighted = (p.reshape(n * rep, T) @ vr.abs()).view(n, rep, -1) / l
            most = (p[..., None] * vs.abs() * 8).amax(-2) / l if p.numel() * vr.shape[-1] < 3e7 else \
                (p.amax(-1, keepdim=True) * vs.abs().amax() * 8 / l).expand_as(weighted)
            sl = slice(h * rep, (h + 1) * rep)
            got[b, :n, sl] = (p.reshape(n * rep, T) @ vr).view(n, rep, -1) / l
            lim[b, :n, sl] = weighted * (2 * off + 2 * (T + 16) * u)
            if out.dtype != torch.float32:
                lim[b, :n, sl] += weighted * 2.0 ** -11 + T * 2.0 ** -24 * most
    return got, lim
