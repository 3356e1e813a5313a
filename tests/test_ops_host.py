"""Refusals of the rotary and attention entry points: host checks that return before anything is enqueued, so they run
without a GPU (the pointers are never used)."""
import ctypes
import math

import pytest
import torch

from recoverable_quantized_kv_gb300 import binding as B
from recoverable_quantized_kv_gb300 import build

PTR = 0x7F0000000000   # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


def rope_cfg(**kw):
    d = dict(rot_dim=128, scaling=0, base=10000.0, factor=1.0, orig_len=0.0, low=1.0, high=32.0)
    d.update(kw)
    return B.RopeConfig(*(d[n] for n, _ in B.RopeConfig._fields_))


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=514), dict(scaling=4), dict(scaling=-1),
                                dict(base=0.0), dict(base=-1.0), dict(base=math.inf), dict(base=math.nan),
                                dict(scaling=1, factor=0.0), dict(scaling=1, factor=math.nan),
                                dict(scaling=2, rot_dim=2, factor=2.0), dict(scaling=3, factor=2.0, orig_len=0.0),
                                dict(scaling=3, factor=2.0, orig_len=4096.0, low=4.0, high=4.0),
                                dict(scaling=3, factor=2.0, orig_len=4096.0, low=-1.0, high=4.0)])
def test_rope_configurations(lib, kw):
    out = (ctypes.c_double * 512)()
    assert lib.qevict_rope_angles(ctypes.byref(rope_cfg(**kw)), out) == B.EINVAL
    assert lib.qevict_rope_table(ctypes.byref(rope_cfg(**kw)), 0, 4, PTR, None) == B.EINVAL


@pytest.mark.parametrize("first,rows,ptr", [(-1, 4, PTR), (0, 0, PTR), (0, 4, 0), (0, 4, PTR + 4), (2 ** 31 - 3, 4, PTR),
                                            (0, 2 ** 31 + 1, PTR), (2 ** 62, 2 ** 62, PTR)])
def test_rope_table_ranges(lib, first, rows, ptr):
    assert lib.qevict_rope_table(ctypes.byref(rope_cfg()), first, rows, ptr, None) == B.EINVAL


def test_rope_angles_formulas(lib):
    """By-parts scaling keeps the pairs that turn more than `high` times over the original context and divides those below
    `low`; the NTK base leaves the first pair and divides the last one by the factor."""
    plain, parts = B.rope_angles(128), B.rope_angles(128, scaling="parts", factor=4.0, orig_len=4096)
    for a, b in zip(plain, parts):
        turns = 4096 * a / (2 * math.pi)
        if turns >= 32:
            assert b == a
        elif turns <= 1:
            assert b == pytest.approx(a / 4, rel=1e-15)
        else:
            assert a / 4 < b < a
    ntk = B.rope_angles(128, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and ntk[-1] == pytest.approx(plain[-1] / 4, rel=1e-12)


def rope_desc(**kw):
    hq, hk, d, b, s = kw.get("h_q", 4), kw.get("h_k", 2), kw.get("d_head", 128), kw.get("batch", 2), kw.get("seq", 3)
    st = lambda h: B._Stride3(max(s, 1) * h * d, h * d, d)   # noqa: E731
    v = dict(dtype=0, batch=b, seq=s, h_q=hq, h_k=hk, d_head=d, rot_dim=128, interleaved=0, inverse=0, factor=1.0,
             table_rows=100, pos0=0, q_in=st(hq), q_out=st(hq), k_in=st(hk), k_out=st(hk))
    v.update(kw)
    return B.RopeDesc(*(v[n] for n, _ in B.RopeDesc._fields_))


def rope_call(lib, desc, table=PTR, pos=PTR, q=PTR, qo=PTR + (1 << 30), k=PTR + (2 << 30), ko=PTR + (3 << 30), st=PTR):
    return lib.qevict_rope_apply(ctypes.byref(desc), table, pos, q, qo, k, ko, st, None)


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(batch=0), dict(seq=0), dict(h_q=-1), dict(h_q=0, h_k=0), dict(rot_dim=130),
                                dict(rot_dim=127), dict(rot_dim=0), dict(interleaved=2), dict(inverse=2),
                                dict(factor=math.nan), dict(table_rows=0), dict(pos0=-1), dict(d_head=2048),
                                dict(q_out=B._Stride3(0, 512, 128)), dict(q_out=B._Stride3(1536, 512, 64)),
                                dict(q_in=B._Stride3(-1536, 512, 128)), dict(k_out=B._Stride3(256, 256, 128))])
def test_rope_descriptors(lib, kw):
    assert rope_call(lib, rope_desc(**kw)) == B.EINVAL


@pytest.mark.parametrize("kw", [dict(table=0), dict(table=PTR + 8), dict(st=0), dict(q=0), dict(qo=0), dict(k=0), dict(ko=0),
                                dict(q=PTR + 1), dict(qo=PTR + 2), dict(qo=PTR + 256), dict(ko=PTR + (2 << 30) - 2),
                                dict(pos=PTR + 2)])
def test_rope_pointers(lib, kw):
    """Missing, misaligned, and partly overlapping tensors."""
    assert rope_call(lib, rope_desc(), **kw) == B.EINVAL


@pytest.mark.parametrize("kw", [dict(qo=PTR + (2 << 30)), dict(ko=PTR), dict(qo=PTR + (3 << 30))])
def test_rope_outputs_over_the_other_tensor(lib, kw):
    """Queries written over the keys, keys over the queries, both to one place."""
    assert rope_call(lib, rope_desc(), **kw) == B.EINVAL


def test_rope_positions_past_the_table_without_a_list(lib):
    assert rope_call(lib, rope_desc(pos0=98), pos=0) == B.EINVAL
    assert rope_call(lib, rope_desc(pos0=2 ** 62), pos=0) == B.EINVAL


def attn_desc(**kw):
    b, sq, skv, hq, hkv = (kw.get(n, x) for n, x in (("batch", 2), ("s_q", 3), ("s_kv", 50), ("h_q", 4), ("h_kv", 2)))
    st = lambda s, h: B._Stride3(s * h * 128, h * 128, 128)   # noqa: E731
    v = dict(dtype=0, batch=b, s_q=sq, s_kv=skv, h_q=hq, h_kv=hkv, d_head=128, causal=1, scale=0.0, softcap=0.0,
             q=st(sq, hq), k=st(skv, hkv), v=st(skv, hkv), o=st(sq, hq))
    v.update(kw)
    return B.AttnDesc(*(v[n] for n, _ in B.AttnDesc._fields_))


BAD_DESC = [dict(dtype=2), dict(batch=0), dict(s_q=0), dict(s_kv=0), dict(h_q=3), dict(h_kv=0), dict(d_head=64), dict(causal=2),
            dict(scale=-1.0), dict(scale=math.inf), dict(softcap=-1.0), dict(softcap=math.nan), dict(h_q=512, h_kv=2),
            dict(q=B._Stride3(1536, 516, 128)), dict(k=B._Stride3(0, 0, 128)), dict(v=B._Stride3(12800, 256, 0)),
            dict(k=B._Stride3(-12800, 256, 128)), dict(o=B._Stride3(0, 512, 128)), dict(s_kv=(1 << 30) + 1)]


@pytest.mark.parametrize("kw", BAD_DESC)
def test_attention_descriptors(lib, kw):
    n = ctypes.c_size_t()
    assert lib.qevict_attn_bytes(ctypes.byref(attn_desc(**kw)), ctypes.byref(n)) == B.EINVAL
    assert lib.qevict_attn(ctypes.byref(attn_desc(**kw)), None, PTR, PTR, PTR, PTR, None, PTR, 1 << 40, None) == B.EINVAL


@pytest.mark.parametrize("scale,lo,hi", [(0.0, 2.0 ** -14 / math.sqrt(128), 2.0 ** 100 / math.sqrt(128)),
                                         (0.25, 2.0 ** -16, 2.0 ** 98)])
def test_attention_caps(lib, scale, lo, hi):
    """A cap far below or above the scale leaves fp32's range in its powers."""
    n = ctypes.c_size_t()
    for cap, want in ((lo * 1.001, B.OK), (hi * 0.999, B.OK), (lo * 0.99, B.EINVAL), (hi * 1.01, B.EINVAL)):
        assert lib.qevict_attn_bytes(ctypes.byref(attn_desc(scale=scale, softcap=cap)), ctypes.byref(n)) == want
        assert lib.qevict_prefix_attn_bytes(ctypes.byref(prefix_desc(scale=scale, softcap=cap)), ctypes.byref(n)) == want


@pytest.mark.parametrize("i", range(9))
def test_attention_pointers_and_masks(lib, i):
    d, m = attn_desc(), B.AttnMask(None, None, None, None, None)
    a = [PTR, PTR, PTR, PTR, PTR, PTR]   # q k v out lse work
    want, size = B.EINVAL, 1 << 40
    if i < 4:
        a[i] = 0 if i % 2 else PTR + 8
    elif i == 4:
        a[4] = PTR + 2
    elif i == 5:
        a[5] = PTR + 128
    elif i == 6:
        d = attn_desc(causal=0)
        m.prefix_len = PTR
    elif i == 7:
        m.kv_len = PTR + 2
    else:
        n = ctypes.c_size_t()
        assert lib.qevict_attn_bytes(ctypes.byref(d), ctypes.byref(n)) == B.OK
        want, size = B.ENOMEM, n.value - 1
    assert lib.qevict_attn(ctypes.byref(d), ctypes.byref(m), *a, size, None) == want


def test_attention_output_rows_may_not_meet(lib):
    d = attn_desc(o=B._Stride3(1536, 256, 128))
    assert lib.qevict_attn(ctypes.byref(d), None, PTR, PTR, PTR, PTR, None, PTR, 1 << 40, None) == B.EINVAL


def prefix_desc(pre=100, kp=(256, 128), vp=(256, 128), **kw):
    return B.PrefixAttnDesc(attn_desc(**kw), pre, B._Stride2(*kp), B._Stride2(*vp))


@pytest.mark.parametrize("d", [dict(pre=0), dict(pre=-5), dict(kp=(0, 128)), dict(vp=(256, 4)), dict(causal=0), dict(s_q=65),
                               dict(q=B._Stride3(0, 512, 128))] + BAD_DESC)
def test_prefix_attention_descriptors(lib, d):
    n = ctypes.c_size_t()
    assert lib.qevict_prefix_attn_bytes(ctypes.byref(prefix_desc(**d)), ctypes.byref(n)) == B.EINVAL


@pytest.mark.parametrize("i", [1, 2, 3, 4, 5])
def test_prefix_attention_pointers(lib, i):
    a = [PTR] * 6   # q kp vp k v out
    a[i] = PTR + 4
    d = prefix_desc()
    assert lib.qevict_prefix_attn(ctypes.byref(d), None, None, *a, None, PTR, 1 << 40, None) == B.EINVAL


def test_workspace_sizes(lib):
    """256 bytes of status, the document runs, and the split results when the keys are split."""
    n = ctypes.c_size_t()
    short = attn_desc(batch=64, s_q=1, s_kv=256, h_q=32, h_kv=8)
    assert lib.qevict_attn_bytes(ctypes.byref(short), ctypes.byref(n)) == B.OK
    assert n.value == 256 + 64 * 256 * 8
    one = attn_desc(batch=1, s_q=1, s_kv=32768, h_q=32, h_kv=8)
    assert lib.qevict_attn_bytes(ctypes.byref(one), ctypes.byref(n)) == B.OK
    assert n.value > 256 + 32768 * 8


def test_status_word_pointer(lib):
    assert lib.qevict_ops_status(None, None, None) == B.EINVAL
    assert lib.qevict_ops_status(PTR + 1, None, None) == B.EINVAL


def test_binding_refuses_before_the_library(lib):
    x = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(B.QEvictError):
        B.Rope(torch.zeros(8, 64, 2))                    # not on a GPU
    with pytest.raises(B.QEvictError):
        B.rope_table(8, scaling="cubic", device="cpu")
    with pytest.raises(B.QEvictError):
        B.rope_table(8, rot_dim=5, device="cpu")
    with pytest.raises(B.QEvictError):
        B._tensor(x, "t", "x", (1, 4, 2, 128), torch.bfloat16, x.device)
