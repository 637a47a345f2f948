"""Pages, slots and positions of a step's new tokens against a sequence by
sequence account on the host: every value has to be equal."""
import random

import pytest
import torch

import transformer_positional_encoding_amd as rp
from serving_refs import reserve

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


class State:
    def __init__(self, rng, B, page, cols, capacity, most):
        pages = list(range(capacity))
        rng.shuffle(pages)
        self.page, self.cols = page, cols
        self.lengths, self.table = [], []
        for _ in range(B):
            n = rng.randrange(0, min(most, cols * page) + 1)
            need = -(-n // page)
            if need > len(pages):
                n = need = 0
            self.lengths.append(n)
            self.table.append([pages.pop() for _ in range(need)] + [-1] * (cols - need))
        self.free = pages + [-7] * (capacity - len(pages))
        self.count = len(pages)
        self.on_gpu()

    def on_gpu(self):
        self.d_table = i32(self.table).view(len(self.lengths), self.cols)
        self.d_lengths, self.d_free, self.d_count = i32(self.lengths), i32(self.free), i32([self.count])

    def step(self, counts, S, what, **kw):
        want = reserve(self.table, self.lengths, counts, self.free, self.count, self.page, S)
        got = rp.rope_cache_reserve(self.d_table, self.d_lengths, i32(counts), self.d_free, self.d_count, self.page,
                                    tokens=S, **kw)
        got = [t.cpu().tolist() for t in got + (self.d_table, self.d_lengths, self.d_free, self.d_count)]
        for name, g, w in zip(("slots", "positions", "granted", "table", "lengths", "free", "count"), got,
                              want[:6] + ([want[6]],)):
            assert g == w, f"{what}: {name}"
        self.table, self.lengths, self.free, self.count = want[3:]
        return want


@pytest.mark.parametrize("B, page, cols, capacity, most, S", [
    (1, 16, 8, 20, 100, 1), (7, 1, 40, 150, 30, 5), (64, 16, 30, 1500, 300, 1), (300, 4, 20, 4000, 60, 40),
    (48, 16, 300, 9000, 4096, 700), (1100, 8, 6, 3000, 40, 3), (3000, 2, 5, 9000, 8, 5), (5, 24, 3, 0, 10, 4),
    (3, 100000, 2, 9, 150000, 9000), (2, 16, 1, 3, 16, 17)])
@pytest.mark.parametrize("seed", [1, 2])
def test_steps(B, page, cols, capacity, most, S, seed):
    rng = random.Random(seed * 1000 + B)
    t = State(rng, B, page, cols, capacity, most)
    for i in range(6):
        kind = rng.choice(["grow", "mixed", "end", "decode"])
        counts = []
        for n in t.lengths:
            grow = rng.randrange(0, S + 1)
            counts.append(grow if kind == "grow" else 1 if kind == "decode" else -n if kind == "end" and rng.random() < .6 else
                          rng.choice([grow, 0, -rng.randrange(0, n + 1), -n - 3, S + 1, S]))
        t.step(counts, S, f"step {i} ({kind})")


def test_order_of_giving_and_taking():
    rng = random.Random(5)
    t = State(rng, 4, 4, 6, 10, 0)
    t.table = [[3, 5, -1, -1, -1, -1], [8, -1, -1, -1, -1, -1], [-1] * 6, [1, 2, 4, -1, -1, -1]]
    t.lengths, t.free, t.count = [7, 4, 0, 9], [0, 6, 7, 9, -7, -7, -7, -7, -7, -7], 4
    t.on_gpu()
    # 0 keeps one page of two, 3 ends with three; 1 needs two pages and 2 five
    want = t.step([-4, 6, 18, -9], 18, "by hand")
    assert want[3][1][:3] == [8, 4, 2] and want[3][2][:5] == [1, 5, 9, 7, 6] and want[6] == 1
    # one page left: 0 needs none, 1 takes it, 2 and 3 have to wait
    want = t.step([1, 3, 5, 1], 5, "short")
    assert want[2] == [1, 3, 0, 0] and want[6] == 0


def test_states_that_are_not_sound():
    """Negative or too great lengths and counts of free pages, negative pages
    in a row: nothing outside the arrays is touched."""
    rng = random.Random(6)
    t = State(rng, 6, 4, 5, 12, 12)
    t.lengths[1], t.lengths[3] = -5, 21
    t.on_gpu()
    t.step([3, 2, -2, 1, 2, -40], 3, "lengths")
    t.count = 40
    t.on_gpu()
    t.step([2, 1, 1, 1, -2, 2], 3, "a count of free pages past their list")
    t.count = -3
    t.on_gpu()
    t.step([9, 1, 1, 1, -2, 2], 9, "a negative count of free pages")
    t.table[0][:] = [-1] * 5
    t.lengths[0] = 6
    t.on_gpu()
    t.step([2, 0, 0, 0, 0, 0], 9, "a row without pages")
    # two sequences that own the same pages: the list is full before all are back
    t.table = [[0, 1, 2, 3, 4]] * 6
    t.lengths, t.count, t.free = [20] * 6, 5, list(range(12))
    t.on_gpu()
    t.step([-20, -20, -20, 0, 0, 0], 9, "more pages than the list holds")


def test_given_outputs_strided_table_and_versions():
    rng = random.Random(8)
    t = State(rng, 5, 4, 6, 40, 12)
    wide = torch.full((5, 9), 77, dtype=torch.int32, device="cuda")
    wide[:, :6] = t.d_table
    t.d_table = wide[:, :6]
    slots, positions = (torch.full((5, 3), 99, dtype=torch.int64, device="cuda") for _ in range(2))
    granted = torch.full((5,), 99, dtype=torch.int32, device="cuda")
    before = wide._version
    got = t.step([3, 3, 0, -3, 2], 3, "given", slots=slots, positions=positions, granted=granted)
    assert slots.tolist() == got[0] and granted.tolist() == got[2] and bool((wide[:, 6:] == 77).all())
    assert wide._version > before
    empty = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    out = rp.rope_cache_reserve(empty, i32([]), i32([]), t.d_free, t.d_count, 4)
    assert out[0].shape == (0, 1)


@pytest.mark.parametrize("B, S", [(6, 3), (5, 4000)])
def test_captured(B, S):
    rng = random.Random(9)
    t = State(rng, B, 16, 600, B * 600, 200)
    counts = i32([min(S, 7)] * B)
    ins = (t.d_table, t.d_lengths, counts, t.d_free, t.d_count)
    rp.rope_cache_reserve(*(v.clone() for v in ins), 16, tokens=S)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = rp.rope_cache_reserve(*ins, 16, tokens=S)
    for i in range(4):
        counts.copy_(i32([rng.randrange(-5, S + 1) for _ in range(B)]))
        copies = [v.clone() for v in ins]
        graph.replay()
        torch.cuda.synchronize()
        want = rp.rope_cache_reserve(*copies, 16, tokens=S)
        for a, b in zip(outs + ins, want + tuple(copies)):
            assert torch.equal(a, b)
