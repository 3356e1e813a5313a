"""The paged cache and its attention: arguments of the right shape in another layout, the smallest caches, tables loaded in
place, calls on a stream of their own."""
import pytest
import torch

import ops_ref as R
from recoverable_quantized_kv_gb300 import binding
from test_gpu_paged_attention import expect, rnd
from test_gpu_pages import BF, FP, Both, i32

pytestmark = pytest.mark.gpu


def every_second(x):
    """The same numbers, every second element of a longer array."""
    return torch.stack([x, x], dim=-1).flatten(-2)[..., ::2]


def test_integers_that_do_not_follow_one_another_are_refused(lib):
    c = binding.PagedCache(1, 8, 16, 2, 3, 4)
    one, table, path = i32([1, 1, 1]), i32([[0, 1, -1, -1], [2, -1, -1, -1], [-1] * 4]), i32([[0, 2], [1, 2], [0, 1]])
    c.load(table, i32([1, 1, 0]))
    rows = torch.zeros(3, 1, 2, 128, dtype=BF, device="cuda")
    for call in (lambda: c.load(table.t().contiguous().t(), one), lambda: c.load(table, every_second(one)),
                 lambda: c.load(every_second(table), one), lambda: c.reserve(every_second(one)),
                 lambda: c.append(rows, rows, layer=0, n=every_second(one)), lambda: c.accept(every_second(one)),
                 lambda: c.accept(one, path.t().contiguous().t()), lambda: c.accept(one, every_second(path)),
                 lambda: c.select(every_second(one)), lambda: c.trim(every_second(one)),
                 lambda: c.select(one[:1].expand(3))):
        with pytest.raises(binding.QEvictError) as e:
            call()
        assert e.value.status == binding.EINVAL
    c.check()
    assert c.length.tolist() == [1, 1, 0]
    assert c.table.tolist() == table.tolist()


def test_attention_refuses_other_layouts(lib):
    q, k, v = rnd(2, 3, 4, 128), rnd(8, 16, 2, 128), rnd(8, 16, 2, 128)
    plan, table, length = binding.PagedAttention(2, 3, 8, 16, 4, 4, 2), i32([[0, 1, 2, 3], [4, 5, 6, 7]]), i32([5, 40])
    par, ql, sl, lse = i32([[-1, 0, 0]] * 2), i32([3, 2]), torch.ones(4, device="cuda"), torch.zeros(2, 3, 4, device="cuda")
    plan.run(q, k, v, table, length, parents=par, q_len=ql, slopes=sl, lse=lse)
    side = torch.cuda.Stream()
    for stream in (None, side):
        for bad in (dict(table=table.t().contiguous().t()), dict(table=every_second(table)), dict(length=every_second(length)),
                    dict(parents=par.t().contiguous().t()), dict(parents=every_second(par[0])), dict(q_len=every_second(ql)),
                    dict(slopes=every_second(sl)), dict(lse=lse.transpose(0, 1).contiguous().transpose(0, 1)),
                    dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), dict(table=table.cpu()), dict(length=length.cpu()),
                    dict(table=table.long()), dict(parents=par.cpu()), dict(q=q.cpu()), dict(table=None)):
            args = dict(q=q, k=k, v=v, table=table, length=length, parents=par, q_len=ql, slopes=sl, lse=lse)
            args.update(bad)
            with pytest.raises(binding.QEvictError):
                plan.run(stream=stream, **args)
    plan.check()


def test_attention_behind_a_prefix_refuses_host_tensors(lib):
    plan, q, own = binding.PrefixAttention(2, 1, 64, 32, 4, 2), rnd(2, 1, 4, 128), rnd(2, 32, 2, 128)
    pre, n, sl, side = rnd(64, 2, 128), i32([5, 6]), torch.ones(4, device="cuda"), torch.cuda.Stream()
    for stream in (None, side):
        for bad in (dict(kv_len=n.cpu()), dict(slopes=sl.cpu()), dict(kv_len=every_second(n)), dict(k=own.cpu())):
            args = dict(q=q, k_prefix=pre, v_prefix=pre, k=own, v=own, kv_len=n, slopes=sl)
            args.update(bad)
            with pytest.raises(binding.QEvictError):
                plan.run(stream=stream, **args)
    plan.check()


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_the_smallest_caches(lib, page, dtype):
    """One layer, one page, one head, one sequence: rows, attention of the first token and of the last that fits."""
    x = Both(1, 1, page, 1, 1, 1, dtype)
    plan = binding.PagedAttention(1, 1, 1, page, 1, 1, 1, dtype=dtype)
    for n in (0, page - 1):
        x.cache.length[0] = n
        x.ref.length[0] = n
        x.reserve(1)
        x.append([1])
        q = rnd(1, 1, 1, 128, seed=n, dtype=dtype)
        out, lse = plan.run(q, x.cache.k[0], x.cache.v[0], x.cache.table, x.cache.length)
        plan.check()
        R.compare(out, lse, expect(q, x.cache.k[0], x.cache.v[0], x.cache.table, [n], [1]))
        x.accept([1])
    x.reserve(1)
    x.compact()
    x.trim([0])
    x.select([-1])


def test_one_page_of_odd_strides(lib):
    """A pool of one page cut out of a larger tensor, whose page step is no multiple of 8: it is never taken."""
    base = torch.randn(16 * 2 * 128 + 5, device="cuda").to(BF)
    k = torch.as_strided(base, (1, 1, 16, 2, 128), (3, 5, 256, 128, 1))
    c = binding.PagedCache(1, 1, 16, 2, 1, 1, k=k, v=k.clone())
    c.reserve(9)
    c.accept(i32([9]))
    plan, q = binding.PagedAttention(1, 2, 1, 16, 1, 4, 2), rnd(1, 2, 4, 128)
    out, lse = plan.run(q, c.k[0], c.v[0], c.table, c.length)
    plan.check()
    c.check()
    R.compare(out, lse, expect(q, c.k[0], c.v[0], c.table, [9], [2]))


def test_loaded_from_its_own_arrays(lib):
    x = Both(1, 30, 16, 1, 4, 5)
    x.reserve([30, 5, 0, 70])
    x.append([30, 5, 0, 60])
    x.accept([30, 5, 0, 60])
    x.select([0, 0, 3, 3])
    x.cache.load(x.cache.table, x.cache.length)
    x.same()
    x.reserve(3)


def test_other_streams(lib):
    """Every call on a stream that is not the current one, and without naming it inside a stream's context."""
    x, side = Both(2, 40, 16, 2, 3, 6), torch.cuda.Stream()
    rows = [torch.randn(2, 3, 20, 2, 128, device="cuda").to(BF) for _ in range(2)]
    n, src, path, length = i32([20, 7, 0]), i32([0, 0, 1]), i32([[1, 3], [0, 1], [2, 4]]), i32([-1, 5, 3])
    two = i32([2, 2, 2])

    def ref():
        P = x.ref
        P.reserve([20] * 3)
        P.append(rows[0].cpu(), rows[1].cpu(), range(2), n.tolist())
        P.accept(n.tolist())
        P.select(src.tolist())
        P.reserve([5] * 3)
        P.append(rows[0][:, :, :5].cpu(), rows[1][:, :, :5].cpu(), range(2), [5] * 3)
        P.accept(two.tolist(), path.tolist())
        P.trim(length.tolist())
        P.compact()

    for named in (True, False):
        x.cache.load()
        x.ref.table, x.ref.length = [[], [], []], [0] * 3
        torch.cuda.synchronize()
        kw = dict(stream=side) if named else {}
        with torch.cuda.stream(None if named else side):
            x.cache.reserve(20, **kw)
            x.cache.append(*rows, n=n, **kw)
            x.cache.accept(n, **kw)
            x.cache.select(src, **kw)
            x.cache.reserve(5, **kw)
            x.cache.append(*(t[:, :, :5] for t in rows), **kw)
            x.cache.accept(two, path, **kw)
            x.cache.trim(length, **kw)
            x.cache.compact(**kw)
            x.cache.check(side)
        torch.cuda.synchronize()
        ref()
        x.same()
