"""Room for new rows where held pages behind a sequence's tokens stand in other sequences too: after a table was loaded, and
after the caller wrote a length back."""
import random

import pytest
import torch

from pages_ref import Pages
from test_gpu_pages import BF, FP, Both, i32

pytestmark = pytest.mark.gpu


class Shared(Pages):
    """The definition with such pages: the first of them that the new rows reach, and all held pages behind it, are given back
    before the free ones are handed out; they do not count towards what is free."""

    def reserve(self, new):
        refs, copies, need, cuts = self.refs(), {}, [], []
        if any(n < 0 or self._up(t + n) > self.max_pages for n, t in zip(new, self.length)):
            return 8
        tails = {b: self.table[b][self.length[b] // self.page] for b in range(self.batch)
                 if new[b] > 0 and self.length[b] % self.page}
        for b, p in tails.items():
            holders = [x for x in tails if tails[x] == p]
            if len(holders) < refs[p] or holders[0] != b:
                copies[b] = p
        for b in range(self.batch):
            row, want = self.table[b], self._up(self.length[b] + new[b])
            reach = range(self._up(self.length[b]), min(want, len(row))) if new[b] > 0 else ()
            cuts.append(next((c for c in reach if refs[row[c]] > 1), len(row)))
            need.append(max(0, want - cuts[b]) if new[b] > 0 else 0)
        if sum(need) + len(copies) > sum(n == 0 for n in refs):
            return 2
        self.table = [row[:c] for row, c in zip(self.table, cuts)]
        free = iter([p for p, n in enumerate(self.refs()) if n == 0])
        for b in range(self.batch):
            if b in copies:
                a, z, rows = copies[b], next(free), self.length[b] % self.page
                self.table[b][self.length[b] // self.page] = z
                for x in (self.k, self.v):
                    x[:, z, :rows] = x[:, a, :rows]
            self.table[b] += [next(free) for _ in range(need[b])]
        return 0


class Loaded(Both):
    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        self.ref.__class__ = Shared

    def load(self, table, length):
        self.ref.table, self.ref.length = [list(r) for r in table], list(length)
        self.cache.load(i32([r + [-1] * (self.ref.max_pages - len(r)) for r in table]), i32(length))
        self.same()

    def set_length(self, b, n):
        self.cache.length[b] = n
        self.ref.length[b] = n

    def step(self, new):
        self.reserve(new)
        self.append(new)
        self.accept(new)


@pytest.mark.parametrize("new", [[1, 0], [0, 1], [1, 1], [16, 16], [17, 2], [33, 40]])
@pytest.mark.parametrize("length", [[16, 20], [20, 16], [16, 16], [0, 16], [0, 0], [0, 20], [7, 30], [32, 0]])
def test_loaded_tables(lib, length, new):
    """Two sequences on the same two pages, of which one or both hold no token of them."""
    x = Loaded(2, 20, 16, 2, 2, 6)
    x.load([[7, 3], [7, 3]], length)
    x.step(new)
    x.step([1, 1])


def test_lengths_written_back(lib):
    """An undo into pages that a fork holds too, to a page's beginning and into the middle of one; the fork's rows stay."""
    for back in (0, 1, 15, 16, 17, 31, 32, 40):
        x = Loaded(1, 40, 16, 1, 3, 6)
        x.step([45, 0, 0])
        x.select([0, 0, 2])
        x.set_length(0, back)
        x.step([1, 0, 0])
        x.step([50 - back, 1, 0])
        x.step([1, 20, 1])


def test_too_few_pages_change_nothing(lib):
    """Pages that would be given back do not count: all or nothing."""
    x = Loaded(1, 4, 16, 1, 2, 4)
    x.load([[0, 1], [0, 1]], [0, 0])
    x.reserve([32, 32])                           # four new ones, two are free
    x.reserve([32, 0])
    x.reserve([17, 32])                           # sequence 1 alone holds them now
    x.load([[0, 1, 2], [0, 1]], [3, 16])
    x.reserve([1, 1])                             # one copied, one given back: one is free
    x.reserve([0, 1])
    x.reserve([0, -1])


def test_a_page_that_everyone_gives_back_is_handed_out_again(lib):
    x = Loaded(1, 8, 16, 1, 3, 4)
    x.load([[0, 1], [0, 1], [0, 1]], [0, 0, 0])
    x.step([20, 20, 20])
    assert x.cache.table[0, :2].tolist() == [0, 1]
    x.load([[5, 2], [5, 2], []], [20, 16, 0])     # the copied page's last other holder gives it back
    x.step([1, 1, 0])
    x.reserve([0, 0, 16])


@pytest.mark.parametrize("batch", [2, 40, 300, 1024])
def test_many_held_pages(lib, batch):
    """Hundreds of held pages behind the tokens, some of them shared, for one sequence or all of a large batch."""
    r, page, most = random.Random(batch), 16, 200 if batch < 100 else 12
    pages = batch * most * 2 + 77
    x = Loaded(1, pages, page, 1, batch, most)
    ids, table, length = r.sample(range(pages), batch * most), [], []
    for b in range(batch):
        row = [ids.pop() for _ in range(r.choice([0, 1, most // 2, most]))]
        if b and r.random() < 0.5:                # the first pages of the sequence before
            same = r.randint(0, len(table[-1]))
            row = table[-1][:same] + row[same:]
        table.append(row)
        length.append(r.choice([0, r.randint(0, len(row) * page), len(row) // 2 * page]))
    x.load(table, length)
    for top in (1, 40, most * page // 3):
        new = [min(r.choice([0, 1, r.randint(0, top)]), most * page - length[b]) for b in range(batch)]
        x.reserve(new)
        x.append([min(n, 50) for n in new])


@pytest.mark.parametrize("seed", range(24))
def test_lives_with_loads_and_undos(lib, seed):
    r = random.Random(seed)
    page, batch, most = r.choice([16, 32, 64]), r.randint(2, 6), r.randint(3, 9)
    pages = r.randint(10, 50)
    x = Loaded(2, pages, page, 1, batch, most, r.choice([BF, FP]), r.choice(["apart", "fused", "heads", "tokens"]), seed=seed)
    some = lambda top: [r.choice([0, 1, r.randint(0, top)]) for _ in range(batch)]   # noqa: E731
    for _ in range(40):
        op = r.choice(["load", "length", "length", "step", "step", "step", "reserve", "select", "trim", "compact"])
        if op == "load":                          # page c + most * n at place c, so that every page has one place
            x.load([[c + most * r.randrange(max(1, pages // most)) for c in range(r.randint(0, min(most, pages)))]
                    for _ in range(batch)], [0] * batch)
            for b in range(batch):
                x.set_length(b, r.choice([0, page, r.randint(0, len(x.ref.table[b]) * page)]) if x.ref.table[b] else 0)
            x.same()
        elif op == "length":
            b = r.randrange(batch)
            n = r.randint(0, x.ref.length[b])
            x.set_length(b, n - n % r.choice([1, page]))
        elif op == "step":
            x.step(some(2 * page))
        elif op == "reserve":
            x.reserve(r.choice([some(most * page), r.randint(0, page)]))
        elif op == "select":
            x.select([r.choice([b, b, r.randrange(batch), -1 if r.random() < 0.3 else b]) for b in range(batch)])
        elif op == "trim":
            x.trim([r.choice([-1, -1, 0, r.randint(0, 4 * page)]) for _ in range(batch)])
        else:
            x.compact()


def test_captured_steps_from_a_loaded_state(lib):
    """A reserve that gives pages back, captured and replayed from the same state again and again."""
    x = Loaded(1, 40, 16, 1, 3, 6)
    table, length = [[9, 8, 7], [9, 8, 7], [9, 8]], [16, 40, 32]
    x.load(table, length)
    saved, ref = x.cache.state.clone(), ([list(t) for t in table], list(length))
    new = i32([20, 1, 1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.cache.state.copy_(saved)
        x.cache.reserve(new)
    for _ in range(3):
        g.replay()
        x.ref.table, x.ref.length = [list(t) for t in ref[0]], list(ref[1])
        x.same(x.ref.reserve([20, 1, 1]), rows=False)
