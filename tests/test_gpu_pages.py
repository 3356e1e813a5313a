"""The paged KV cache against its definition: tables, counts and rows, bit for bit, over sequences of calls."""
import random

import pytest
import torch

from pages_ref import Pages
from recoverable_quantized_kv_gb300 import binding

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def pool(layers, pages, page, h, dtype, form, seed=0):
    """k, v of one pool: apart, one behind the other in every page, or head by head."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)   # noqa: E731
    if form == "fused":
        x = make(layers, pages, 2, page, h, 128)
        return x[:, :, 0], x[:, :, 1]
    if form == "heads":
        return (make(layers, pages, h, page, 128).transpose(2, 3) for _ in range(2))
    if form == "tokens":     # keys and values side by side in a token's row, layers innermost of the pages
        x = make(pages, layers, page, 2 * h, 128).transpose(0, 1)
        return x[..., :h, :], x[..., h:, :]
    return make(layers, pages, page, h, 128), make(layers, pages, page, h, 128)


class Both:
    """A cache and its definition, given the same calls."""

    def __init__(self, layers, pages, page, h, batch, max_pages, dtype=BF, form="apart", seed=0):
        k, v = pool(layers, pages, page, h, dtype, form, seed)
        self.cache = binding.PagedCache(layers, pages, page, h, batch, max_pages, dtype=dtype, k=k, v=v)
        self.ref = Pages(k.cpu().contiguous(), v.cpu().contiguous(), batch, max_pages)
        self.shape, self.dtype, self.rng = (layers, pages, page, h), dtype, random.Random(seed)
        self.same()

    def same(self, bits=0, rows=True):
        word = 0
        try:
            self.cache.check()
        except binding.QEvictError as e:
            assert e.status == binding.EDEVICE
            word = e.word
        assert word == bits, (word, bits)
        length, held, table, refs, n_free = self.ref.arrays()
        c = self.cache
        for name, got, want in (("length", c.length, length), ("held", c.held, held), ("table", c.table, table),
                                ("refs", c.refs, refs)):
            assert torch.equal(got.cpu(), want), f"{name}: {got.tolist()} for {want.tolist()}"
        assert int(c.n_free) == n_free
        lay = c.layout
        words = c.state[lay.free_bits:lay.free_bits + (len(refs) + 127) // 128 * 4].cpu().numpy().view("uint32")
        free = [int(words[p // 32]) >> (p % 32) & 1 for p in range(len(words) * 32)]
        assert free == [int(r == 0) for r in refs.tolist()] + [0] * (len(free) - len(refs))
        if rows:
            assert torch.equal(c.k.cpu(), self.ref.k) and torch.equal(c.v.cpu(), self.ref.v)

    def reserve(self, new):
        self.cache.reserve(new if isinstance(new, int) else i32(new))
        self.same(self.ref.reserve([new] * self.ref.batch if isinstance(new, int) else new))

    def append(self, n, layer=None, most=None):
        layers, _, _, h = self.shape
        most = most or max(1, max(n))
        x = [torch.randn(layers if layer is None else 1, self.ref.batch, most, h, 128, device="cuda").to(self.dtype)
             for _ in range(2)]
        given = x if layer is None else [t[0] for t in x]
        self.cache.append(*given, layer=layer, n=i32(n))
        self.same(self.ref.append(x[0].cpu(), x[1].cpu(), range(layers) if layer is None else [layer], n))

    def accept(self, count, path=None):
        self.cache.accept(i32(count), None if path is None else i32(path))
        self.same(self.ref.accept(count, path))

    def select(self, src):
        self.cache.select(i32(src))
        self.same(self.ref.select(src))

    def trim(self, length):
        self.cache.trim(i32(length))
        self.same(self.ref.trim(length))

    def compact(self):
        self.cache.compact()
        self.same(self.ref.compact())


@pytest.mark.parametrize("form", ["apart", "fused", "heads", "tokens"])
@pytest.mark.parametrize("page,h,dtype", [(16, 2, BF), (32, 1, FP), (64, 3, BF), (128, 2, FP)])
def test_a_life_of_calls(lib, form, page, h, dtype):
    """Random calls in turn, those that fail among them, against the definition after every one."""
    x = Both(2, 37, page, h, 5, 9, dtype, form, seed=page + h)
    r = x.rng
    for step in range(60):
        op = r.choice(["reserve", "reserve", "append", "append", "accept", "accept", "path", "select", "trim", "compact"])
        some = lambda top: [r.choice([0, 1, r.randint(0, top)]) for _ in range(5)]   # noqa: E731
        if op == "reserve":
            x.reserve(r.choice([some(3 * page), some(2 * page), r.randint(0, page), some(10 * page)]))
        elif op == "append":
            x.append(some(2 * page), layer=r.choice([None, 0, 1]))
        elif op == "accept":
            x.accept(some(2 * page))
        elif op == "path":
            most = r.randint(1, 20)
            path = [sorted(r.sample(range(40), most)) for _ in range(5)]
            if r.random() < 0.2:
                path[r.randrange(5)] = [0] * most
            x.accept([r.randint(0, most) for _ in range(5)], path)
        elif op == "select":
            x.select([r.choice([b, b, b, r.randrange(5), -1 if r.random() < 0.5 else b]) for b in range(5)])
        elif op == "trim":
            x.trim([r.choice([-1, -1, 0, r.randint(0, 4 * page)]) for _ in range(5)])
        else:
            x.compact()


def test_first_free_pages_in_order(lib):
    x = Both(1, 200, 16, 1, 4, 60)
    x.reserve([33, 0, 1, 100])
    assert x.cache.table[0, :3].tolist() == [0, 1, 2] and x.cache.table[2, 0] == 3 and x.cache.table[3, 6] == 10
    x.trim([0, -1, -1, -1])
    x.reserve([0, 50, 0, 0])
    assert x.cache.table[1, :4].tolist() == [0, 1, 2, 11]
    x.reserve(0)


def test_copy_on_write_among_several_holders(lib):
    """Three sequences share a partly filled page.  All reserve: the first keeps it.  Without one of them: all copy."""
    for new, keeps in (([1, 1, 1], True), ([1, 1, 0], False), ([0, 1, 1], False)):
        x = Both(3, 20, 16, 2, 3, 4, form="fused")
        x.reserve([21, 0, 0])
        x.append([21, 0, 0])
        x.accept([21, 0, 0])
        x.select([0, 0, 0])
        before = int(x.cache.table[0, 1])
        x.append([1, 1, 1])                       # refused: the page is shared
        x.accept([1, 0, 0])
        x.reserve(new)
        assert (int(x.cache.table[0, 1]) == before) == (keeps or not new[0])
        x.append([1 if n else 0 for n in new])
        x.accept([1 if n else 0 for n in new])


def test_too_few_pages_change_nothing(lib):
    x = Both(2, 6, 32, 1, 3, 8)
    x.reserve([64, 32, 0])
    x.reserve([64, 64, 65])                       # three more, and three
    x.reserve([64, 32, 96])
    x.reserve([65, 0, 0])
    x.reserve([-1, 1, 1])
    x.reserve([32 * 8 + 1, 0, 0])
    assert int(x.cache.n_free) == 0


def test_accepted_trees(lib):
    """Paths that overlap the rows they move to, the whole tree, none, and one row moved far, over a page's end."""
    x = Both(4, 64, 16, 2, 6, 8)
    x.reserve([70] * 6)
    x.append([13, 0, 15, 16, 3, 1])
    x.accept([13, 0, 15, 16, 3, 1])
    x.append([40] * 6)
    x.accept([5, 1, 20, 0, 3, 1], [[0, 2, 3, 7, 39] + [0] * 15, [33] + [0] * 19, list(range(20)), [5] * 20,
                                   [1, 2, 3] + [9] * 17, [0] * 20])
    x.accept([1] * 6, [[45]] * 6)                 # within the pages of some
    x.accept([2] * 6, [[3, 3], [4, 2], [-1, 1], [0, 70], [0, 1], [2 ** 31 - 2, 2 ** 31 - 1]])
    x.accept([21, -1, 2 ** 31 - 1, 0, 0, 0])


@pytest.mark.parametrize("n", [1, 100, 256])
def test_long_paths(lib, n):
    x = Both(1, 20, 128, 1, 1, 20)
    x.reserve([1200])
    x.append([1000])
    x.accept([n], [sorted(x.rng.sample(range(900), n))])


def test_beams_cross(lib):
    """Every sequence becomes another one at once, pages that all of them drop in between stay held."""
    x = Both(1, 64, 16, 1, 6, 6)
    x.reserve([5, 17, 33, 16, 80, 0])
    x.append([5, 17, 33, 16, 80, 0])
    x.accept([5, 17, 33, 16, 80, 0])
    for src in ([1, 0, 3, 2, 5, 4], [5, 4, 3, 2, 1, 0], [2, 2, 2, 2, 2, 2], [1, 2, 3, 4, 5, 0], [-1, 0, -1, 1, 6, -2],
                [-1] * 6):
        x.select(src)
        x.reserve(1)
        x.append([1] * 6)
        x.accept([1] * 6)


def test_many_sequences_and_pages(lib):
    """1024 sequences, and a pool of several of the scans' steps with the last bits in use."""
    r = random.Random(5)
    x = Both(1, 140001, 16, 1, 1024, 150)
    k, v = x.ref.k.clone(), x.ref.v.clone()
    new = [r.choice([0, 16, r.randint(1, 2000), 2200]) for _ in range(1024)]
    x.cache.reserve(i32(new))
    x.same(x.ref.reserve(new), rows=False)
    x.cache.accept(i32(new))
    x.same(x.ref.accept(new), rows=False)
    src = [r.choice([b, b, -1, r.randrange(1024)]) for b in range(1024)]
    for _ in range(2):
        x.cache.select(i32(src))
        x.same(x.ref.select(src), rows=False)
        x.cache.reserve(40)
        x.same(x.ref.reserve([40] * 1024))
        x.cache.compact()
        x.same(x.ref.compact())
    assert not (torch.equal(k, x.ref.k) and torch.equal(v, x.ref.v))


def test_load(lib):
    x = Both(1, 50, 16, 1, 4, 5)
    c, P = x.cache, x.ref
    P.table, P.length = [[7, 3], [7, 49, 0, 1, 2], [], [7, 3, 5]], [20, 80, 0, 33]
    table = [r + [-1] * (5 - len(r)) for r in P.table]
    c.load(i32(table), i32(P.length))
    x.same()
    table[0][3] = 9                               # behind the end: not a page of the sequence
    c.load(i32(table), i32([20, 80, 0, 33]))
    x.same()
    for bad in (50, -2, -2 ** 31):                # not a page: the sequence ends there
        table[1][1] = bad
        P.table[1], P.length[1] = [7], 16
        c.load(i32(table), i32([20, 80, -5, 33]))
        x.same(8)
    c.load(i32([[7, 3, -1, -1, -1], [3, -1, -1, -1, -1], [-1] * 5, [-1] * 5]), i32([20, 3, 0, 0]))
    with pytest.raises(binding.QEvictError) as e:   # page 3 at two places
        c.check()
    assert e.value.word == 4
    c.load()
    P.table, P.length = [[], [], [], []], [0] * 4
    x.same()


def test_saved_and_restored(lib):
    x = Both(2, 30, 16, 2, 3, 6)
    x.reserve([20, 30, 0])
    x.append([20, 30, 0])
    x.accept([20, 30, 0])
    x.select([0, 1, 1])
    saved = x.cache.state.clone(), x.cache.k.clone(), x.cache.v.clone()
    ref = [list(r) for r in x.ref.table], list(x.ref.length), x.ref.k.clone(), x.ref.v.clone()
    x.reserve(9)
    x.append([9, 8, 7])
    x.trim([3, -1, 0])
    for t, y in zip((x.cache.state, x.cache.k, x.cache.v), saved):
        t.copy_(y)
    x.ref.table, x.ref.length, x.ref.k, x.ref.v = ref
    x.same()
    x.reserve(1)


def test_lengths_taken_back(lib):
    """Written by the caller: within the pages held, and values that are not."""
    x = Both(1, 30, 16, 1, 3, 6)
    x.reserve([40, 40, 40])
    x.append([40, 40, 40])
    x.accept([40, 40, 40])
    x.cache.length[1] = 17
    x.ref.length[1] = 17
    x.append([3, 3, 3])
    for wild in (10 ** 6, -10 ** 6):
        x.cache.length[2] = wild
        x.ref.length[2] = 48 if wild > 0 else 0   # clamped wherever it is read
        x.cache.accept(i32([0, 0, 0]))
        x.ref.accept([0, 0, 0])
        x.same()


@pytest.mark.parametrize("most", [1, 7, 300])
def test_rows_of_other_strides(lib, most):
    """New rows from a fused projection, all sequences from one, in reverse-ordered dimensions; odd counts."""
    layers, h, b = 2, 3, 4
    x = Both(layers, 100, 32, h, b, 20)
    x.reserve([most + 5] * b)
    n = [most, max(0, most - 3), 0, most]
    fused = torch.randn(b, most, 5 * h + 1, 128, device="cuda").to(BF)
    forms = [(fused[:, :, h:2 * h], fused[:, :, 4 * h + 1:]), (fused[:1, :, :h].expand(b, -1, -1, -1), fused[:, :, h:2 * h]),
             tuple(torch.randn(h, most, b, 128, device="cuda").to(BF).permute(2, 1, 0, 3) for _ in range(2))]
    for k, v in forms:
        x.cache.append(k, v, layer=1, n=i32(n))
        x.same(x.ref.append(k[None].cpu(), v[None].cpu(), [1], n))
    k = torch.randn(b, layers, most, h, 128, device="cuda").to(BF).transpose(0, 1)
    x.cache.append(k, k)
    x.same(x.ref.append(k.cpu(), k.cpu(), range(layers), [most] * b))
    x.append([most + 1, -1, 2 ** 31 - 1, 0], most=most)   # counts out of range


def test_streams_and_graphs(lib):
    """A step captured once and replayed, on a stream of its own, equals the same calls made one by one."""
    x = Both(2, 60, 16, 2, 4, 12)
    x.reserve([9, 20, 0, 33])
    x.append([9, 20, 0, 33])
    x.accept([9, 20, 0, 33])
    k = torch.randn(2, 4, 8, 2, 128, device="cuda").to(BF)
    count, path = i32([1, 3, 0, 2]), i32([[4, 0, 0], [0, 3, 7], [1, 1, 1], [2, 3, 0]])

    def step(stream=None):
        x.cache.reserve(8, stream=stream)
        x.cache.append(k, k, stream=stream)
        x.cache.accept(count, path, stream=stream)

    def ref():
        x.ref.reserve([8] * 4)
        x.ref.append(k.cpu(), k.cpu(), range(2), [8] * 4)
        x.ref.accept(count.tolist(), path.tolist())

    step()
    ref()
    x.same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    ref()
    torch.cuda.current_stream().wait_stream(side)
    x.same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        ref()
        x.same()


def test_other_devices_streams_and_refusals(lib):
    """Arguments on the wrong device, of the wrong shape, type or layout, and sizes that another integer would hold."""
    c = binding.PagedCache(2, 8, 16, 2, 3, 4)
    x, n = torch.zeros(3, 5, 2, 128, dtype=BF, device="cuda"), i32([1, 1, 1])
    for call in (lambda: c.append(x.cpu(), x, layer=0), lambda: c.append(x, x, layer=2), lambda: c.append(x, x, layer=-1),
                 lambda: c.append(x, x), lambda: c.append(x, x[:, :4], layer=0), lambda: c.append(x.to(FP), x, layer=0),
                 lambda: c.append(x[..., ::2], x, layer=0), lambda: c.append(x, x, layer=0, n=n.long()),
                 lambda: c.append(x.clone().requires_grad_(), x, layer=0), lambda: c.accept(n[:2]), lambda: c.accept(None),
                 lambda: c.accept(n, i32([1, 2, 3])), lambda: c.accept(n, i32([[0, 1]] * 2)), lambda: c.select(n.cpu()),
                 lambda: c.trim(i32([[1], [1], [1]])), lambda: c.reserve(n.float()), lambda: c.reserve(-1),
                 lambda: c.reserve(2 ** 32), lambda: c.load(c.table), lambda: c.load(c.table[:, :3], c.length),
                 lambda: c.load(i32([[0] * 4] * 4)[:3].t(), n)):
        with pytest.raises(binding.QEvictError):
            call()
    c.check()
    assert int(c.n_free) == 8 and not bool(c.length.any())
