"""Refusals of the rotary and attention operators that need no GPU: no gradient is recorded, and sizes whose products leave 64
bits are refused."""
import ctypes

import pytest
import torch

from recoverable_quantized_kv_gb300 import binding as B
from recoverable_quantized_kv_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load()


@pytest.mark.parametrize("name", ["q", "k", "v", "slopes", "k_prefix", "v_prefix"])
def test_inputs_that_require_a_gradient(name):
    """Refused before anything else is looked at (these are CPU tensors, refused for that otherwise)."""
    t = {n: torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16) for n in ("q", "k", "v")}
    t.update(k_prefix=torch.zeros(3, 4, 128, dtype=torch.bfloat16), v_prefix=torch.zeros(3, 4, 128, dtype=torch.bfloat16),
             slopes=torch.zeros(4))
    t[name].requires_grad_()
    attn, step, rope = (object.__new__(c) for c in (B.Attention, B.PrefixAttention, B.Rope))
    rope.index = attn.index = step.index = 0
    step.desc = attn.desc = None
    calls = [lambda: step.run(t["q"], t["k_prefix"], t["v_prefix"], t["k"], t["v"], slopes=t["slopes"])]
    if "prefix" not in name:
        calls.append(lambda: attn.run(t["q"], t["k"], t["v"], slopes=t["slopes"]))
    if name in ("q", "k"):
        calls.append(lambda: rope.apply(t["q"], t["k"]))
    for call in calls:
        with pytest.raises(B.QEvictError, match="no gradient is recorded") as e:
            call()
        assert e.value.status == B.EINVAL
        with torch.no_grad(), pytest.raises(Exception) as e:
            call()
        assert "gradient" not in str(e.value)


def desc(**kw):
    v = dict(dtype=0, batch=1, s_q=1, s_kv=1, h_q=1, h_kv=1, d_head=128, causal=1, scale=0.0, softcap=0.0)
    v.update(kw)
    st = B._Stride3(128, 128, 128)
    return B.AttnDesc(*(v[n] for n, _ in B.AttnDesc._fields_[:10]), st, st, st, st)


@pytest.mark.parametrize("kw", [dict(batch=2 ** 30, h_q=2 ** 30, h_kv=2 ** 30, s_q=2 ** 12), dict(batch=2 ** 30, s_q=2 ** 30, h_q=2 ** 30, h_kv=2 ** 30),
                                dict(batch=2 ** 31 - 1, h_q=2 ** 31 - 1, h_kv=2 ** 31 - 1), dict(batch=2 ** 24 + 1),
                                dict(h_q=2 ** 24 + 1, h_kv=2 ** 24 + 1), dict(batch=2 ** 13, h_q=2 ** 12, h_kv=2 ** 12)])
def test_sizes_whose_products_wrap(lib, kw):
    """2^24 pairs of row tiles and KV heads are the limit, however large the factors."""
    n = ctypes.c_size_t()
    assert lib.qevict_attn_bytes(ctypes.byref(desc(**kw)), ctypes.byref(n)) == B.EINVAL
    p = B.PrefixAttnDesc(desc(**kw), 5, B._Stride2(128, 128), B._Stride2(128, 128))
    assert lib.qevict_prefix_attn_bytes(ctypes.byref(p), ctypes.byref(n)) == B.EINVAL


@pytest.mark.parametrize("n", range(3))
def test_strides_whose_reach_wraps(lib, n):
    st = [128, 128, 128]
    st[n] = 2 ** 37
    kw = dict(batch=2 ** 12) if n == 0 else dict(s_q=2 ** 12, s_kv=2 ** 12) if n == 1 else dict(h_q=2 ** 12, h_kv=2 ** 12)
    d = desc(**kw)
    big = B._Stride3(*st)
    d.q = d.k = d.v = d.o = big
    size = ctypes.c_size_t()
    assert lib.qevict_attn_bytes(ctypes.byref(d), ctypes.byref(size)) == B.EINVAL
    st[n] = 2 ** 40
    big = B._Stride3(*st)
    r = B.RopeDesc(0, 2 ** 9 if n == 0 else 1, 2 ** 9 if n == 1 else 1, 2 ** 9 if n == 2 else 1, 0, 128, 128, 0, 0, 1.0, 2 ** 20, 0,
                   big, big, big, big)
    at = 0x7F0000000000   # no refused call touches it
    assert lib.qevict_rope_apply(ctypes.byref(r), at, at, at, at, None, None, at, None) == B.EINVAL
