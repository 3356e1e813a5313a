"""Refusals of the paged cache and its attention: host checks that return before anything is enqueued, so they run without a
GPU (the pointers are never used)."""
import ctypes
import math

import pytest
import torch

from recoverable_quantized_kv_gb300 import binding as B
from recoverable_quantized_kv_gb300 import build
from test_ops_host import PTR


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def pages_desc(**kw):
    d = dict(layers=2, pages=10, page=16, h_kv=2, d_head=128, batch=3, max_pages=4, reserved0=0)
    d.update({n: x for n, x in kw.items() if n in d})
    st = (d["pages"] * d["page"] * d["h_kv"] * 128, d["page"] * d["h_kv"] * 128, d["h_kv"] * 128, 128)
    return B.PagesDesc(*(d[n] for n in d), B._Stride4(*kw.get("k", st)), B._Stride4(*kw.get("v", st)))


BAD_PAGES = [dict(layers=0), dict(layers=32768), dict(pages=0), dict(pages=(1 << 24) + 1), dict(page=8), dict(page=48),
             dict(page=256), dict(h_kv=0), dict(h_kv=5000), dict(d_head=64), dict(batch=0), dict(batch=1025), dict(max_pages=0),
             dict(max_pages=(1 << 26) + 1), dict(batch=1024, max_pages=(1 << 20) + 1), dict(reserved0=1),
             dict(k=(40960, 4096, 256, 64)), dict(v=(40960, 4096, 255, 128)), dict(k=(40960, 4096, 0, 128)),
             dict(k=(40960, 4096, -256, 128)), dict(v=(4096, 4096, 256, 128)), dict(k=(1 << 41, 4096, 256, 128))]


@pytest.mark.parametrize("kw", BAD_PAGES)
def test_pages_descriptors(lib, kw):
    d, lay = ctypes.byref(pages_desc(**kw)), B.PagesLayout()
    rows = B.PagesRows(0, 1, 1, 0, B._Stride4(0, 256, 256, 128), B._Stride4(0, 256, 256, 128))
    assert lib.qevict_pages_get_layout(d, ctypes.byref(lay)) == B.EINVAL
    assert lib.qevict_pages_load(d, PTR, None, None, None) == B.EINVAL
    assert lib.qevict_pages_reserve(d, PTR, PTR, PTR, PTR, 0, None) == B.EINVAL
    assert lib.qevict_pages_append(d, ctypes.byref(rows), PTR, PTR, PTR, PTR, PTR, None, None) == B.EINVAL
    assert lib.qevict_pages_accept(d, PTR, PTR, PTR, PTR, None, 0, None) == B.EINVAL
    assert lib.qevict_pages_select(d, PTR, PTR, None) == B.EINVAL
    assert lib.qevict_pages_trim(d, PTR, PTR, None) == B.EINVAL
    assert lib.qevict_pages_compact(d, PTR, PTR, PTR, None) == B.EINVAL


def test_pages_layout(lib):
    """Arrays that do not overlap, in the documented order, each on 256 bytes."""
    lay = B.PagesLayout()
    for kw in (dict(), dict(pages=1, max_pages=1, batch=1), dict(pages=100003, batch=1024, max_pages=77)):
        d = pages_desc(**kw)
        assert lib.qevict_pages_get_layout(ctypes.byref(d), ctypes.byref(lay)) == B.OK
        ends = [(lay.length, d.batch), (lay.held, d.batch), (lay.table, d.batch * d.max_pages), (lay.refs, d.pages),
                (lay.free_bits, (d.pages + 31) // 32), (lay.ints, 0)]
        assert (lay.status, lay.n_free) == (0, 1) and lay.length >= 4
        for (at, n), (nxt, _) in zip(ends, ends[1:]):
            assert at % 64 == 0 and at + n <= nxt


@pytest.mark.parametrize("i", range(4))
@pytest.mark.parametrize("bad", [0, PTR + 2])
def test_pages_pointers(lib, i, bad):
    d, rows = ctypes.byref(pages_desc()), B.PagesRows(0, 1, 1, 0, B._Stride4(0, 256, 256, 128), B._Stride4(0, 256, 256, 128))
    a = [PTR] * 4                                  # k v state, argument
    a[i] = bad
    optional = bad == 0 and i == 3
    assert lib.qevict_pages_accept(d, *a, None, 0, None) == B.EINVAL
    if not optional:
        assert lib.qevict_pages_reserve(d, *a, 0, None) == B.EINVAL
        assert lib.qevict_pages_append(d, ctypes.byref(rows), *a[:3], PTR, PTR, a[3], None) == B.EINVAL
    if i < 3:
        assert lib.qevict_pages_compact(d, *a[:3], None) == B.EINVAL
        assert lib.qevict_pages_append(d, ctypes.byref(rows), PTR, PTR, PTR, *([bad, PTR] if i else [PTR, bad]), None,
                                       None) == B.EINVAL
    else:
        assert lib.qevict_pages_select(d, PTR, bad, None) == B.EINVAL
        assert lib.qevict_pages_trim(d, PTR, bad, None) == B.EINVAL
        assert lib.qevict_pages_load(d, PTR, PTR, bad, None) == B.EINVAL
    assert lib.qevict_pages_load(d, PTR + 128, None, None, None) == B.EINVAL


def test_pages_arguments(lib):
    d = ctypes.byref(pages_desc())
    assert lib.qevict_pages_reserve(d, PTR, PTR, PTR, None, -1, None) == B.EINVAL
    assert lib.qevict_pages_accept(d, PTR, PTR, PTR, PTR, PTR, 0, None) == B.EINVAL
    assert lib.qevict_pages_accept(d, PTR, PTR, PTR, PTR, PTR, 257, None) == B.EINVAL
    st = B._Stride4(0, 256, 256, 128)
    for rows in (B.PagesRows(-1, 1, 1, 0, st, st), B.PagesRows(0, 3, 1, 0, st, st), B.PagesRows(2, 1, 1, 0, st, st),
                 B.PagesRows(2 ** 31 - 1, 2, 1, 0, st, st), B.PagesRows(0, 0, 1, 0, st, st), B.PagesRows(0, 1, 0, 0, st, st),
                 B.PagesRows(0, 1, 1, 1, st, st), B.PagesRows(0, 1, 2, 0, B._Stride4(0, 256, 4, 128), st),
                 B.PagesRows(0, 1, 1, 0, st, B._Stride4(0, -256, 256, 128)), B.PagesRows(0, 1, 2 ** 31 - 1, 0, st, st)):
        assert lib.qevict_pages_append(d, ctypes.byref(rows), PTR, PTR, PTR, PTR, PTR, None, None) == B.EINVAL


def paged_desc(**kw):
    v = dict(dtype=0, batch=2, s_q=3, h_q=4, h_kv=2, d_head=128, scale=0.0, softcap=0.0, pages=9, page=16, max_pages=5,
             reserved0=0)
    v.update({n: x for n, x in kw.items() if n in v})
    q, p = (v["s_q"] * v["h_q"] * 128, v["h_q"] * 128, 128), (v["page"] * v["h_kv"] * 128, v["h_kv"] * 128, 128)
    return B.PagedAttnDesc(*(v[n] for n in v), *(B._Stride3(*kw.get(n, p if n in "kv" else q)) for n in "qokv"))


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(batch=0), dict(s_q=0), dict(h_q=3), dict(h_kv=0), dict(d_head=64),
                                dict(scale=-1.0), dict(softcap=math.nan), dict(h_q=512), dict(pages=0), dict(page=17),
                                dict(pages=(1 << 24) + 1), dict(max_pages=0), dict(max_pages=1 << 27), dict(s_q=81),
                                dict(reserved0=2), dict(k=(4096, 252, 128)), dict(v=(0, 256, 128)), dict(k=(4096, 256, -128)),
                                dict(q=(1536, 516, 128)), dict(o=(0, 512, 128)), dict(softcap=1e-6)])
def test_paged_attention_descriptors(lib, kw):
    n, d = ctypes.c_size_t(), paged_desc(**kw)
    assert lib.qevict_paged_attn_bytes(ctypes.byref(d), ctypes.byref(n)) == B.EINVAL
    assert lib.qevict_paged_attn(ctypes.byref(d), None, *[PTR] * 6, None, PTR, 1 << 40, None) == B.EINVAL


@pytest.mark.parametrize("i", range(6))
@pytest.mark.parametrize("bad", [0, PTR + 2])
def test_paged_attention_pointers(lib, i, bad):
    a = [PTR] * 6                                  # q k v table length out
    a[i] = bad
    assert lib.qevict_paged_attn(ctypes.byref(paged_desc()), None, *a, None, PTR, 1 << 40, None) == B.EINVAL


def test_paged_attention_masks_and_workspace(lib):
    d, n = paged_desc(s_q=65, max_pages=9), ctypes.c_size_t()
    call = lambda d, m, lse=None, w=PTR, size=1 << 40: lib.qevict_paged_attn(   # noqa: E731
        ctypes.byref(d), ctypes.byref(m), *[PTR] * 6, lse, w, size, None)
    assert call(d, B.PagedAttnMask(None, None, PTR, 0)) == B.EINVAL   # a tree of more than 64 nodes
    d = paged_desc()
    for m in (B.PagedAttnMask(PTR + 1, None, None, 0), B.PagedAttnMask(None, PTR + 2, None, 0), B.PagedAttnMask(None, None, PTR + 2, 1)):
        assert call(d, m) == B.EINVAL
    none = B.PagedAttnMask(None, None, None, 0)
    assert call(d, none, lse=PTR + 2) == B.EINVAL and call(d, none, w=PTR + 128) == B.EINVAL
    assert lib.qevict_paged_attn_bytes(ctypes.byref(d), ctypes.byref(n)) == B.OK
    assert call(d, none, size=n.value - 1) == B.ENOMEM


def test_binding_refuses_before_the_library(lib):
    with pytest.raises(B.QEvictError):
        B.PagedCache(1, 4, 16, 2, 1, 4, device="cpu")
    x = torch.zeros(1, 4, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(B.QEvictError):
        B.PagedCache(1, 4, 16, 2, 1, 4, k=x, v=x)
    with pytest.raises(B.QEvictError):
        B.PagedCache(1, 4, 16, 2, 1, 4, k=x)
    with pytest.raises(B.QEvictError):
        B.PagedCache(1, 4, 16, 2, 1, 4, dtype=torch.float32)
    for kw in (dict(pages=2 ** 32 + 4), dict(max_pages=2 ** 32 + 4), dict(batch=-2 ** 33)):
        with pytest.raises(B.QEvictError):
            B._sizes("PagedCache", **kw)
