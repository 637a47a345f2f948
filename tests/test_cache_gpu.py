"""Writing rotated keys to paged, quantised caches and reading them back, on
the GPU, against the definition: codes, scales and rows have to be equal."""
import pytest
import torch

import transformer_positional_encoding_amd as rp
from axes_refs import TORCH, bound, pair_tables, rotate64
from cache_refs import decode_codes, encode, rotate32

pytestmark = pytest.mark.gpu

FORMATS = ["e4m3", "int8", "int4", "same"]


def make_cache(pages, page, N, D, fmt, group, dtype):
    c = rp.rope_cache(pages, page, N, D, dtype if fmt == "same" else fmt, None if fmt == "same" else group)
    c.data.view(torch.uint8).fill_(0x33)
    if c.scales is not None:
        c.scales.fill_(-5.0)
    return c


def slots_for(B, S, pages, page, seed, skip=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randperm(pages * page, generator=g)[: B * S].view(B, S).clone()
    flat = t.view(-1)
    for k in range(skip):
        flat[(7 * k + 3) % flat.numel()] = (-1, -(1 << 40), pages * page, 1 << 40)[k % 4]
    return t


def expect_written(cache, slots, z, fmt, group, dtype, what):
    """The cache holds z at the slots, and everywhere else what it held."""
    pages, page = cache.data.shape[:2]
    flat = slots.reshape(-1)
    live = (flat >= 0) & (flat < pages * page)
    at = flat[live]
    got = cache.data.cpu().flatten(0, 1)
    rows = z.flatten(0, 1)[live]
    rest = torch.ones(pages * page, dtype=torch.bool)
    rest[at] = False
    assert bool((got[rest].contiguous().view(torch.uint8) == 0x33).all()), f"{what}: a slot of no token changed"
    if fmt == "same":
        want = rows.to(TORCH[dtype])
        same = (got[at].float() == want.float()) | (torch.isnan(got[at].float()) & torch.isnan(want.float()))
        assert bool(same.all()), f"{what}: rows differ"
        return
    sc = cache.scales.cpu().flatten(0, 1)
    assert bool((sc[rest] == -5.0).all()), f"{what}: a scale of no token changed"
    codes, scales = encode(rows, fmt, group)
    assert torch.equal(sc[at].double(), scales), f"{what}: scales differ"
    have = decode_codes(got[at])
    same = (have == codes) | (torch.isnan(have) & torch.isnan(codes))
    assert bool(same.all()), f"{what}: {int((~same).sum())} codes differ"


# (B, S, Nq, Nk, D, Dv, slice, mode, group): whole heads, latent rows, half
# lines, odd sizes that only the general kernel takes
GEOMETRIES = [
    (2, 5, 8, 2, 128, 128, (0, 128), "rotate_half", 128),
    (1, 9, 0, 1, 576, 0, (512, 576), "interleave", 64),
    (3, 3, 4, 1, 576, 512, (512, 576), "rotate_half", 64),
    (1, 1, 32, 8, 128, 64, (32, 96), "interleave", 32),
    (4, 7, 3, 3, 192, 128, (0, 64), 4, 64),
    (2, 3, 5, 2, 80, 80, (0, 80), "rotate_half", 80),
    (2, 4, 1, 2, 96, 96, (24, 72), "interleave", 96),
    (1, 6, 2, 1, 1024, 256, (0, 1024), "rotate_half", 256),
    (1, 6, 2, 1, 1024, 0, (0, 16), "rotate_half", 1024),
    (2, 5, 2, 3, 36, 20, (3, 31), "rotate_half", 4),
    (2, 5, 2, 3, 50, 10, (1, 47), "interleave", 10),
    (1, 4, 1, 1, 2, 2, (0, 2), "interleave", 2),
    (2, 3, 0, 16, 64, 64, (0, 64), "interleave", 64),
    (1, 70, 0, 1, 32, 32, (16, 32), "rotate_half", 32),
]


@pytest.mark.parametrize("B, S, Nq, Nk, D, Dv, sl, mode, group", GEOMETRIES)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype, table", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", "f16")])
def test_write(B, S, Nq, Nk, D, Dv, sl, mode, group, fmt, dtype, table):
    g = torch.Generator().manual_seed(B * 1000 + D)
    make = lambda n, d: (torch.randn(B, S, n, d, generator=g) * torch.exp(torch.randn(B, S, n, 1, generator=g))).to(TORCH[dtype])  # noqa: E731
    q, k, v = make(Nq, D), make(Nk, D), make(Nk, Dv)
    page, pages = 4, B * S // 4 + 3
    slots = slots_for(B, S, pages, page, 5, skip=min(3, B * S - 1))
    A = 3 if B > 1 else 1
    L = sl[1] - sl[0]
    ax = tuple(i % A for i in range(L // 2))
    pos = torch.randint(0, 90000, (A, 1 if S == 3 else B, S), generator=g)
    f = rp.rope_inv_freq(L)
    kc = make_cache(pages, page, Nk, D, fmt, group, dtype)
    vc = make_cache(pages, page, Nk, Dv, fmt, group, dtype) if Dv else None
    dq = q.cuda() if Nq else None
    for rotate_k in (True, False):
        rp.rope_cache_write(k.cuda(), v.cuda() if Dv else None, kc, vc, slots.cuda(),
                            pos.cuda() if A > 1 else pos[0].cuda(), f.cuda(), mode, sl, q=dq,
                            pair_axes=ax if A > 1 else None, table_dtype=TORCH[table], rotate_k=rotate_k)
        cos, sin = pair_tables(pos, f, ax, table)
        z = rotate32(k, cos, sin, mode, sl) if rotate_k else k.float()
        # the fp32 rotation itself is within its rounding of the 64-bit one
        z64, size = rotate64(k.double(), cos, sin, mode, sl)
        assert not rotate_k or bool(((z.double() - z64).abs() <= bound(z64, size, "f32")).all())
        expect_written(kc, slots, z, fmt, group, dtype, f"k rotate={rotate_k}")
        if Dv:
            expect_written(vc, slots, v.float(), fmt, group, dtype, "v")
        if Nq:
            q = rotate32(q, cos, sin, mode, sl).to(TORCH[dtype])
            assert torch.equal(dq.cpu().view(torch.uint8), q.view(torch.uint8)), "q"


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_of_a_fused_projection_into_one_half_of_a_joint_cache(fmt):
    """q, k and v as slices of one tensor; K and V pages beside each other;
    slots as a column of a larger tensor."""
    B, S, Nq, Nk, D, page, pages = 2, 6, 4, 2, 64, 4, 5
    g = torch.Generator().manual_seed(1)
    fused = torch.randn(B, S, (Nq + 2 * Nk) * D, generator=g).to(torch.bfloat16)
    dev = fused.cuda()
    cut = lambda t: (t[..., :Nq * D].unflatten(-1, (Nq, D)), t[..., Nq * D:(Nq + Nk) * D].unflatten(-1, (Nk, D)),  # noqa: E731
                     t[..., (Nq + Nk) * D:].unflatten(-1, (Nk, D)))
    q, k, v = cut(dev)
    width = {"int4": D // 2}.get(fmt, D)
    ty = {"same": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8, "int4": torch.uint8}[fmt]
    joint = torch.zeros(pages, 2, Nk, page, width, dtype=ty, device="cuda")
    joint.view(torch.uint8).fill_(0x33)
    sc = None if fmt == "same" else torch.full((pages, 2, Nk, page, 2), -5.0, device="cuda")
    half = lambda i: rp.RopeCache(joint[:, i].transpose(1, 2), None if sc is None else sc[:, i].transpose(1, 2))  # noqa: E731
    kc, vc = half(0), half(1)
    slots = slots_for(B, S, pages, page, 3, skip=1)
    wide = torch.full((B, S, 3), -1)
    wide[..., 1] = slots
    pos = torch.arange(S).expand(1, S)
    f = rp.rope_inv_freq(D)
    rp.rope_cache_write(k, v, kc, vc, wide.cuda()[..., 1], pos.cuda(), f.cuda(), "rotate_half", (0, D), q=q)
    cos, sin = pair_tables(pos[None], f, (0,) * (D // 2), "bf16")
    q0, k0, v0 = cut(fused)
    expect_written(kc, slots, rotate32(k0, cos, sin, "rotate_half", (0, D)), fmt, 32, "bf16", "k")
    expect_written(vc, slots, v0.float(), fmt, 32, "bf16", "v")
    assert torch.equal(q.cpu(), rotate32(q0, cos, sin, "rotate_half", (0, D)).to(torch.bfloat16))
    assert torch.equal(k.cpu(), k0) and torch.equal(v.cpu(), v0), "k or v changed"


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
@pytest.mark.parametrize("D, group", [(128, 32), (36, 12)])
def test_write_of_zeros_ties_tiny_and_not_finite_values(fmt, D, group):
    rows = torch.zeros(1, 12, 1, D)
    g = torch.Generator().manual_seed(4)
    rows[0, 1] = torch.randint(-14, 15, (D,), generator=g) / 2.0       # halves: ties of every format
    rows[0, 1, 0, ::group] = 7.0
    rows[0, 2] = torch.arange(D) - D / 2.0
    rows[0, 3, 0, 1] = float("nan")
    rows[0, 4] = torch.randn(D, generator=g)
    rows[0, 4, 0, 3], rows[0, 4, 0, 5] = float("inf"), -float("inf")
    rows[0, 5, 0, 2] = float("inf")
    rows[0, 6] = torch.randn(D, generator=g) * 1e-38
    rows[0, 7] = 2.0 ** -149
    rows[0, 8] = 3.4028234663852886e38
    rows[0, 9] = torch.randn(D, generator=g) * 1e37
    rows[0, 9, 0, 4] = float("nan")
    rows[0, 10] = -(2.0 ** -100)
    rows[0, 11] = torch.linspace(-448, 448, D)
    c = make_cache(3, 5, 1, D, fmt, group, "f32")
    slots = slots_for(1, 12, 3, 5, 2)
    rp.rope_cache_write(rows.cuda(), None, c, None, slots.cuda())
    expect_written(c, slots, rows, fmt, group, "f32", "special rows")
    if fmt == "int4":
        return
    # every magnitude that a bf16 row holds, at many largest values
    n = 64
    g = torch.Generator().manual_seed(9)
    x = torch.randint(0, 1 << 15, (1, n, 4, 128), generator=g).to(torch.int16).view(torch.bfloat16).float()
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).clamp(-1e30, 1e30)
    x = torch.where(torch.rand(x.shape, generator=g) < 0.5, x, -x).to(torch.bfloat16)
    c = make_cache(n, 1, 4, 128, fmt, 128, "bf16")
    slots = torch.arange(n)[None]
    rp.rope_cache_write(x.cuda(), None, c, None, slots.cuda())
    expect_written(c, slots, x.float(), fmt, 128, "bf16", "any bf16")


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "int4"])
def test_quotients_next_to_midpoints(fmt):
    """Values one and two units in the last place around every midpoint of the
    format times the scale: the exact quotient decides."""
    D = 128
    g = torch.Generator().manual_seed(11)
    for trial in range(6):
        m = float(torch.rand(1, generator=g) * 10 + 0.1)
        s = torch.tensor(m, dtype=torch.float32).double() / {"e4m3": 448.0, "int8": 127.0, "int4": 7.0}[fmt]
        s = s.float().double()
        top = {"e4m3": 448, "int8": 127, "int4": 7}[fmt]
        if fmt == "e4m3":
            v = torch.arange(0, 128, dtype=torch.uint8)[:127].view(torch.float8_e4m3fn).double()
            mids = (v[1:] + v[:-1]) / 2
        else:
            mids = torch.arange(0, top).double() + 0.5
        t = (mids * s).float()
        vals = torch.cat([torch.nextafter(t, torch.zeros_like(t)), t, torch.nextafter(t, t * 2)])
        vals = torch.cat([vals, -vals])
        rows = torch.zeros((len(vals) + D - 2) // (D - 1), D)
        rows[:, 1:].reshape(-1)
        flat = torch.zeros(rows.shape[0] * (D - 1))
        flat[: len(vals)] = vals
        rows[:, 1:] = flat.view(-1, D - 1)
        rows[:, 0] = m
        rows = rows[None, :, None]
        n = rows.shape[1]
        c = make_cache(n, 1, 1, D, fmt, D, "f32")
        slots = torch.arange(n)[None]
        rp.rope_cache_write(rows.cuda(), None, c, None, slots.cuda())
        expect_written(c, slots, rows, fmt, D, "f32", f"midpoints, trial {trial}")


def test_v_in_another_format_than_k():
    B, S, D = 2, 5, 64
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(B, S, n, D, generator=g).to(torch.float16) for n in (4, 2, 2))
    kc, vc = make_cache(4, 4, 2, D, "same", 0, "f16"), make_cache(4, 4, 2, D, "int4", 16, "f16")
    slots = slots_for(B, S, 4, 4, 3, skip=2)
    pos, f = torch.arange(S).expand(B, S) + 9, rp.rope_inv_freq(D)
    dq = q.cuda()
    rp.rope_cache_write(k.cuda(), v.cuda(), kc, vc, slots.cuda(), pos.cuda(), f.cuda(), "interleave", (0, D), q=dq)
    cos, sin = pair_tables(pos[None], f, (0,) * (D // 2), "f16")
    expect_written(kc, slots, rotate32(k, cos, sin, "interleave", (0, D)), "same", 0, "f16", "k")
    expect_written(vc, slots, v.float(), "int4", 16, "f16", "v")
    assert torch.equal(dq.cpu(), rotate32(q, cos, sin, "interleave", (0, D)).to(torch.float16))


# ------------------------------------------------------------------- reading back


def filled(pages, page, N, D, fmt, group, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    c = rp.rope_cache(pages, page, N, D, dtype if fmt == "same" else fmt, None if fmt == "same" else group)
    if fmt == "same":
        c.data.copy_(torch.randn(c.data.shape, generator=g))
    elif fmt == "e4m3":
        b = torch.randint(0, 256, c.data.shape, generator=g).to(torch.uint8)
        b[(b & 127) == 127] = 0
        c.data.view(torch.uint8).copy_(b)
    elif fmt == "int8":
        c.data.copy_(torch.randint(-128, 128, c.data.shape, generator=g))
    else:
        c.data.copy_(torch.randint(0, 256, c.data.shape, generator=g))
    if c.scales is not None:
        c.scales.copy_(torch.rand(c.scales.shape, generator=g) + 0.01)
    return c


def read_want(c, out, table, lengths, starts, turn, mode, sl, dtype):
    """The rows a read leaves, from fp32 products."""
    pages, page = c.data.shape[:2]
    v = decode_codes(c.data).float() if c.scales is not None else c.data.cpu().float()
    if c.scales is not None:
        v = (v.unflatten(-1, (c.scales.shape[-1], -1)) * c.scales.cpu()[..., None]).flatten(-2)
    want = out.cpu().clone()
    for b in range(out.shape[0]):
        for s in range(min(int(lengths[b]), out.shape[1])):
            t = int(starts[b]) + s
            if t < 0 or t // page >= table.shape[1]:
                continue
            pg = int(table[b, t // page])
            if not 0 <= pg < pages:
                continue
            row = v[pg, t % page][None, None]
            if turn is not None:
                cos, sin = turn
                bb = min(b, cos.shape[0] - 1)
                row = rotate32(row, cos[bb, s][None, None], sin[bb, s][None, None], mode, sl)
            want[b, s] = row[0, 0].to(TORCH[dtype])
    return want


@pytest.mark.parametrize("N, D, sl, mode, group", [
    (8, 128, (0, 128), "rotate_half", 128), (1, 576, (512, 576), "interleave", 64), (2, 64, (16, 48), "interleave", 32),
    (3, 192, (0, 64), 4, 192), (2, 80, (0, 80), "rotate_half", 16), (2, 36, (3, 31), "rotate_half", 4),
    (1, 50, (1, 47), "interleave", 50), (1, 1024, (0, 1024), "rotate_half", 128), (5, 24, (0, 24), "interleave", 8),
    (1, 2, (0, 2), "interleave", 2)])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype, table_type", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")])
def test_read(N, D, sl, mode, group, fmt, dtype, table_type):
    B, S, page, pages = 4, 13, 3, 23
    c = filled(pages, page, N, D, fmt, group, dtype, D)
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(pages, generator=g)[:20].view(4, 5).to(torch.int32)
    table[2, 1], table[3, 0] = -1, pages                       # pages outside the cache
    lengths = torch.tensor([13, 0, 40, 7], dtype=torch.int32)  # all, none, past the table, a part
    for starts in (None, torch.tensor([2, 0, 1, -3], dtype=torch.int32)):
        for turned in (False, True):
            out = torch.full((B, S, N, D), 3.0, dtype=TORCH[dtype], device="cuda")
            L = sl[1] - sl[0]
            A = 2
            pos = torch.randint(0, 50000, (A, 1 if starts is None else B, S), generator=g)
            f, ax = rp.rope_inv_freq(L), tuple(i % A for i in range(L // 2))
            kw = dict(positions=pos.cuda(), inv_freq=f.cuda(), pair_axes=ax, rotary_mode=mode, partial_slice=sl,
                      table_dtype=TORCH[table_type]) if turned else {}
            turn = pair_tables(pos, f, ax, table_type) if turned else None
            want = read_want(c, out, table, lengths, [0] * B if starts is None else starts, turn, mode, sl, dtype)
            rp.rope_cache_read(out, c, table.cuda(), lengths.cuda(), None if starts is None else starts.cuda(), **kw)
            assert torch.equal(out.cpu().view(torch.uint8), want.view(torch.uint8)), f"turned={turned}"


def test_read_into_a_permuted_output():
    c = filled(6, 4, 2, 64, "int8", 32, "bf16", 1)
    table, lengths = torch.tensor([[5, 0, 3]], dtype=torch.int32), torch.tensor([10], dtype=torch.int32)
    dense = torch.zeros(1, 12, 2, 64, dtype=torch.bfloat16, device="cuda")
    turned = torch.zeros(1, 2, 12, 64, dtype=torch.bfloat16, device="cuda")
    rp.rope_cache_read(dense, c, table.cuda(), lengths.cuda())
    rp.rope_cache_read(turned.transpose(1, 2), c, table.cuda(), lengths.cuda())
    assert torch.equal(dense, turned.transpose(1, 2))
    assert torch.equal(dense.cpu(), read_want(c, torch.zeros_like(dense), table, lengths, [0], None, None, None, "bf16"))


@pytest.mark.parametrize("fmt", FORMATS)
def test_slots_past_32_bit_offsets(fmt):
    """A cache whose last page begins past 2^32 bytes (and, for the storage
    type, 2^32 elements), written and read there."""
    D, page = 128, 16
    width = D // 2 if fmt == "int4" else D
    ty = {"same": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8, "int4": torch.uint8}[fmt]
    stride = (1 << 32) + 256
    store = torch.empty(stride + page * width, dtype=torch.uint8 if fmt != "same" else ty, device="cuda")
    data = torch.as_strided(store, (2, page, 1, width), (stride, width, width, 1))
    data = data if fmt in ("same", "int4") else data.view(ty)
    sc = None if fmt == "same" else torch.as_strided(torch.empty((1 << 31) + 64, device="cuda"), (2, page, 1, 1),
                                                     ((1 << 31) + 8, 1, 1, 1))
    c = rp.RopeCache(data, sc)
    g = torch.Generator().manual_seed(1)
    k = torch.randn(1, 3, 1, D, generator=g).to(torch.bfloat16)
    rp.rope_cache_write(k.cuda(), None, c, None, torch.tensor([[3, page + 5, page + 15]]).cuda())
    out = torch.zeros(1, 2 * page, 1, D, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[0, 1]], dtype=torch.int32).cuda()
    rp.rope_cache_read(out, c, table, torch.tensor([2 * page], dtype=torch.int32).cuda())
    got = out[0, [3, page + 5, page + 15]].cpu()
    if fmt == "same":
        want = k[0]
    else:
        codes, s = encode(k[0].float(), fmt, D)
        want = (codes.float() * s.float()).to(torch.bfloat16)
    assert torch.equal(got, want)


def test_empty_calls():
    c = rp.rope_cache(2, 4, 2, 64, "e4m3")
    nothing = torch.zeros(0, 5, 2, 64, dtype=torch.bfloat16, device="cuda")
    rp.rope_cache_write(nothing, None, c, None, torch.zeros(0, 5, dtype=torch.int64, device="cuda"))
    rp.rope_cache_read(nothing, c, torch.zeros(0, 1, dtype=torch.int32, device="cuda"),
                       torch.zeros(0, dtype=torch.int32, device="cuda"))
    none = rp.rope_cache(0, 4, 2, 64, "e4m3")
    k = torch.ones(1, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    rp.rope_cache_write(k, None, none, None, torch.tensor([[0, 1]], device="cuda"))
    assert bool((c.data.view(torch.uint8) == 0).all())


def test_graph_replays_follow_slots_and_positions():
    B, S, N, D = 4, 1, 2, 128
    g = torch.Generator().manual_seed(2)
    k, v, q = (torch.randn(B, S, n, D, generator=g).to(torch.bfloat16).cuda() for n in (N, N, 8))
    f = rp.rope_inv_freq(D).cuda()
    pos = torch.randint(0, 9000, (B, S), generator=g).cuda()
    slots = slots_for(B, S, 8, 4, 1).cuda()
    table = torch.arange(8, dtype=torch.int32).view(1, 8).cuda()
    lengths = torch.tensor([32], dtype=torch.int32).cuda()
    kc, vc = rp.rope_cache(8, 4, N, D, "e4m3"), rp.rope_cache(8, 4, N, D, "e4m3")
    out, q_in = torch.zeros(1, 32, N, D, dtype=torch.bfloat16, device="cuda"), q.clone()

    def step(kc, vc, out, q):
        rp.rope_cache_write(k, v, kc, vc, slots, pos, f, "rotate_half", (0, D), q=q)
        rp.rope_cache_read(out, kc, table, lengths)

    step(kc, vc, out, q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(kc, vc, out, q)
    for i in range(4):
        pos.add_(3 + i)
        slots.copy_(slots_for(B, S, 8, 4, 10 + i))
        q.copy_(q_in)
        for c in (kc, vc):
            c.data.view(torch.uint8).zero_()
            c.scales.zero_()
        graph.replay()
        torch.cuda.synchronize()
        kc2, vc2 = rp.rope_cache(8, 4, N, D, "e4m3"), rp.rope_cache(8, 4, N, D, "e4m3")
        out2, q2 = torch.zeros_like(out), q_in.clone()
        step(kc2, vc2, out2, q2)
        torch.cuda.synchronize()
        for a, b in ((kc, kc2), (vc, vc2)):
            assert torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8)) and torch.equal(a.scales, b.scales)
        assert torch.equal(out, out2) and torch.equal(q, q2)


def test_on_another_stream():
    k = torch.randn(2, 50, 4, 128).to(torch.bfloat16).cuda()
    slots = slots_for(2, 50, 30, 4, 1).cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a, b = rp.rope_cache(30, 4, 4, 128), rp.rope_cache(30, 4, 4, 128)
    torch.cuda.synchronize()
    rp.rope_cache_write(k, None, a, None, slots, stream=s)
    s.synchronize()
    rp.rope_cache_write(k, None, b, None, slots)
    assert torch.equal(a.data.view(torch.uint8), b.data.view(torch.uint8)) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("N, D", [(8, 128), (1, 64), (1, 50)])
def test_lengths_and_starts_at_the_ends_of_their_type(N, D):
    """Rows without a cached token keep their bytes whatever lengths and
    starts hold."""
    c = filled(4, 3, N, D, "int8", D, "bf16", 1)
    table = torch.tensor([[0, 1], [2, 3], [1, 2], [3, 0]], dtype=torch.int32)
    top, low = 2 ** 31 - 1, -2 ** 31
    for lengths, starts in (([top, low, 5, top], [top, 0, low, 0]), ([5, 5, 5, 5], [5, -4, top - 2, low])):
        out = torch.full((4, 7, N, D), 3.0, dtype=torch.bfloat16, device="cuda")
        lengths, starts = (torch.tensor(v, dtype=torch.int32) for v in (lengths, starts))
        want = read_want(c, out, table, lengths, starts, None, None, None, "bf16")
        rp.rope_cache_read(out, c, table.cuda(), lengths.cuda(), starts.cuda())
        assert torch.equal(out.cpu(), want)


def test_two_streams_at_once():
    """Writes and reads of two caches at a time, against one after the other."""
    g = torch.Generator().manual_seed(3)
    ks = [torch.randn(3, 200, 4, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    slots, f = slots_for(3, 200, 160, 4, 1).cuda(), rp.rope_inv_freq(128).cuda()
    pos = torch.arange(200).expand(3, 200).contiguous().cuda()
    table, lengths = torch.arange(160, dtype=torch.int32).view(1, 160).cuda(), torch.tensor([640], dtype=torch.int32).cuda()
    state = lambda: (rp.rope_cache(160, 4, 4, 128), torch.zeros(1, 640, 4, 128, dtype=torch.bfloat16, device="cuda"))  # noqa: E731
    got, want = [state() for _ in ks], [state() for _ in ks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ks]
    for k, (c, out), s in zip(ks, got, streams):
        rp.rope_cache_write(k, None, c, None, slots, pos, f, "rotate_half", (0, 128), stream=s)
        rp.rope_cache_read(out, c, table, lengths, stream=s)
    torch.cuda.synchronize()
    for k, (c, out), (c2, out2) in zip(ks, want, got):
        rp.rope_cache_write(k, None, c, None, slots, pos, f, "rotate_half", (0, 128))
        rp.rope_cache_read(out, c, table, lengths)
        assert torch.equal(out, out2) and torch.equal(c.scales, c2.scales) and bool(out.any())


@pytest.mark.parametrize("N, D, sl, mode", [(1, 64, (0, 64), "interleave"), (5, 64, (0, 64), "rotate_half"),
                                            (9, 128, (0, 128), "rotate_half"), (1, 1024, (0, 1024), "interleave"),
                                            (17, 64, (32, 64), "interleave"), (1, 8, (0, 8), "interleave"),
                                            (18, 64, (0, 64), "rotate_half")])
@pytest.mark.parametrize("fmt", FORMATS)
def test_read_of_tokens_of_every_width(N, D, sl, mode, fmt):
    """Tokens of 1 to 144 chunks, many blocks of them, padded rows between."""
    B, S, page, pages = 3, 150, 16, 40
    c = filled(pages, page, N, D, fmt, D, "bf16", N)
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(pages, generator=g)[:30].view(3, 10).to(torch.int32)
    lengths = torch.tensor([150, 1, 97], dtype=torch.int32)
    L = sl[1] - sl[0]
    pos, f = torch.randint(0, 50000, (1, B, S), generator=g), rp.rope_inv_freq(L)
    for turned in (False, True):
        out = torch.full((B, S, N, D), 3.0, dtype=torch.bfloat16, device="cuda")
        kw = dict(positions=pos[0].cuda(), inv_freq=f.cuda(), rotary_mode=mode, partial_slice=sl) if turned else {}
        turn = pair_tables(pos, f, (0,) * (L // 2), "bf16") if turned else None
        want = read_want(c, out, table, lengths, [0] * B, turn, mode, sl, "bf16")
        rp.rope_cache_read(out, c, table.cuda(), lengths.cuda(), **kw)
        assert torch.equal(out.cpu().view(torch.uint8), want.view(torch.uint8)), f"turned={turned}"
