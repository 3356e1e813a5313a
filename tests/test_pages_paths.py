"""Accepted paths whose width is none or too many: refused on the host, before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

from recoverable_quantized_kv_gb300 import binding as B
from test_ops_host import PTR
from test_pages_host import lib, pages_desc   # noqa: F401


@pytest.mark.parametrize("width", [-1, 1, 3, 256, 257])
def test_a_width_without_a_path(lib, width):   # noqa: F811
    d = ctypes.byref(pages_desc())
    assert lib.qevict_pages_accept(d, PTR, PTR, PTR, PTR, None, width, None) == B.EINVAL


def host_cache(calls, batch=3):
    """A cache's argument checks on host tensors; what would be enqueued is listed."""
    c = object.__new__(B.PagedCache)
    c.batch, c.index, c._i32, c._seqs, c._pool, c._state = batch, -1, torch.int32, torch.Size([batch]), (PTR, PTR), PTR
    c._run = lambda name, stream, tensors, *args: calls.append((name, args))
    return c


@pytest.mark.parametrize("width", [0, 257, 1000])
def test_paths_of_no_or_too_many_columns(width):
    calls = []
    c, count = host_cache(calls), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(B.QEvictError) as e:
        c.accept(count, torch.zeros(3, width, dtype=torch.int32))
    assert e.value.status == B.EINVAL and not calls


@pytest.mark.parametrize("width", [1, 256])
def test_paths_that_are_passed_on(width):
    calls = []
    c, count = host_cache(calls), torch.zeros(3, dtype=torch.int32)
    path = torch.zeros(3, width, dtype=torch.int32)
    c.accept(count, path)
    c.accept(count)
    assert [x[1][3:] for x in calls] == [(count.data_ptr(), path.data_ptr(), width), (count.data_ptr(), None, 0)]


@pytest.mark.gpu
def test_an_empty_path_accepts_nothing(lib):   # noqa: F811
    from test_gpu_pages import Both
    x = Both(1, 20, 16, 1, 3, 4)
    x.reserve(5)
    x.append([5, 5, 5])
    path = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    for empty in (path[:, :0], torch.zeros(3, 0, dtype=torch.int32, device="cuda")):
        with pytest.raises(B.QEvictError):
            x.cache.accept(torch.ones(3, dtype=torch.int32, device="cuda"), empty)
        x.same()
    x.accept([1, 0, 1], [[4]] * 3)
