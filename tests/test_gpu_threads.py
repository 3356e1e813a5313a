"""Host threads that share a plan or a cache on one stream: ctypes lets other threads run during a call, so a call's arguments
are its own, and what it enqueues is enqueued together."""
import threading
import time

import pytest
import torch

from recoverable_quantized_kv_gb300 import binding
from test_gpu_paged_attention import BF, i32, rnd, tree

pytestmark = pytest.mark.gpu


def together(calls):
    """Runs the calls in threads that start at once; errors come back."""
    gate, failed = threading.Barrier(len(calls)), []

    def run(call):
        try:
            gate.wait(30)
            call()
        except BaseException as e:   # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads)
    if failed:
        raise failed[0]


class Slow:
    """The library with one of its calls replaced by one that takes 20 ms, notes who is inside and reads its arguments before
    and after."""

    def __init__(self, lib, name, read):
        self.lib, self.name, self.read, self.inside, self.seen = lib, name, read, 0, []

    def __getattr__(self, name):
        return self.call if name == self.name else getattr(self.lib, name)

    def call(self, *args):
        self.inside += 1
        alone, first = self.inside == 1, self.read(args)
        time.sleep(0.02)
        self.seen.append((alone and self.inside == 1, first, self.read(args)))
        self.inside -= 1
        return binding.OK


def paged():
    plan = binding.PagedAttention(2, 5, 12, 16, 6, 4, 2)
    return plan, (rnd(2, 5, 4, 128), rnd(12, 16, 2, 128), rnd(12, 16, 2, 128), i32([[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11]]),
                  i32([5, 60]))


def test_masks_of_paged_attention_belong_to_their_call(lib, monkeypatch):
    plan, args = paged()
    parents = [i32([tree(5, s), tree(5, s + 9)]) for s in range(4)]

    def read(a):
        return a[1]._obj.parents

    slow = Slow(lib, "qevict_paged_attn", read)
    monkeypatch.setattr(binding, "_lib", slow)
    together([lambda p=p: plan.run(*args, parents=p) for p in parents])
    assert sorted(x[1] for x in slow.seen) == sorted(p.data_ptr() for p in parents)
    assert all(first == last for _, first, last in slow.seen)


@pytest.mark.parametrize("kind", ["paged", "dense", "prefix", "reserve", "compact", "load"])
def test_calls_of_one_plan_or_cache_take_turns(lib, monkeypatch, kind):
    """A call enqueues kernels that belong together: another thread's does not come between them."""
    if kind == "paged":
        plan, args = paged()
        name, call = "qevict_paged_attn", lambda: plan.run(*args)
    elif kind == "dense":
        plan, q, k = binding.Attention(2, 1, 64, 4, 2), rnd(2, 1, 4, 128), rnd(2, 64, 2, 128)
        name, call = "qevict_attn", lambda: plan.run(q, k, k)
    elif kind == "prefix":
        plan, q, k = binding.PrefixAttention(2, 1, 64, 32, 4, 2), rnd(2, 1, 4, 128), rnd(2, 32, 2, 128)
        pre = rnd(64, 2, 128)
        name, call = "qevict_prefix_attn", lambda: plan.run(q, pre, pre, k, k)
    else:
        cache = binding.PagedCache(1, 8, 16, 1, 2, 4)
        name, call = "qevict_pages_" + kind, {"reserve": lambda: cache.reserve(1), "compact": cache.compact,
                                             "load": cache.load}[kind]
    slow = Slow(lib, name, lambda a: None)
    monkeypatch.setattr(binding, "_lib", slow)
    together([call] * 4)
    assert len(slow.seen) == 4 and all(alone for alone, _, _ in slow.seen)


def test_one_plan_from_several_threads(lib):
    """Trees of each thread's own against contexts that are cut into parts and merged: every result is the one it has alone."""
    B, m, n, page = 1, 24, 6000, 32
    need = -(-(n + m) // page)
    k, v = rnd(need, page, 2, 128, seed=2), rnd(need, page, 2, 128, seed=3)
    table = torch.randperm(need, device="cuda").to(torch.int32)[None]
    plan = binding.PagedAttention(B, m, need, page, need, 8, 2)
    mine = [(rnd(B, m, 8, 128, seed=10 + t), i32([n - 700 * t]), i32([tree(m, t)])) for t in range(4)]
    want = [plan.run(q, k, v, table, ln, parents=par) for q, ln, par in mine]
    got = [[] for _ in mine]

    def work(t):
        q, ln, par = mine[t]
        for _ in range(100):
            got[t].append(plan.run(q, k, v, table, ln, parents=par))

    together([lambda t=t: work(t) for t in range(4)])
    plan.check()
    for x, outs in zip(want, got):
        assert len(outs) == 100
        assert all(torch.equal(o, x[0]) and torch.equal(s, x[1]) for o, s in outs)


def test_rows_of_many_shapes_from_several_threads(lib):
    """More shapes of new rows than a cache keeps descriptors of, from threads at once."""
    cache = binding.PagedCache(1, 64, 16, 1, 1, 64)
    cache.reserve(700)
    x = torch.zeros(1, 700, 1, 128, dtype=BF, device="cuda")

    def work(t):
        for n in range(1, 600):
            cache.append(x[:, :n + t % 2], x[:, :n + t % 2], layer=0)

    together([lambda t=t: work(t) for t in range(3)])
    cache.check()
