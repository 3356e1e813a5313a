"""Attention where a choice inside the kernel could let through what a row does not see, or lose what it does."""
import math

import pytest
import torch

import ops_strict as S
from recoverable_quantized_kv_gb300 import binding

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def rnd(*shape, seed=0, dtype=BF, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed * 6151 + len(shape) + sum(shape))
    return (gain * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same_bits(a, b):
    return torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32),
                       b.view(torch.int16 if b.element_size() == 2 else torch.int32))


# ------------------------------------------------------------------------------------------------ capped logits

CAPS = (30.0, 6.0, 1.0)   # of logits of deviation 1.5: felt by none, by the largest, by all


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("sq,skv", [(1, 700), (3, 5000), (300, 300), (40, 2100)])
def test_capped_rows_do_not_feel_keys_behind_the_end(lib, cap, sq, skv):
    """The same rows over a cache that holds small numbers, or thousands, behind each sequence's end: the same bits."""
    n = [skv - 97, skv // 3 + 1]
    ql = [min(sq, x) for x in n]
    q, k, v = rnd(2, sq, 8, 128, gain=1.5), rnd(2, skv, 2, 128, seed=2), rnd(2, skv, 2, 128, seed=3)
    plan = binding.Attention(2, sq, skv, 8, 2, softcap=cap)
    got = []
    for fill in (0.01, 3000.0):
        for b in range(2):
            k[b, n[b]:] = rnd(skv - n[b], 2, 128, seed=4 + b, gain=fill)
            v[b, n[b]:] = rnd(skv - n[b], 2, 128, seed=6 + b, gain=fill)
        got.append(plan.run(q, k, v, kv_len=i32(n), q_len=i32(ql)))
    plan.check()
    for b in range(2):
        assert same_bits(got[0][0][b, :ql[b]], got[1][0][b, :ql[b]]) and same_bits(got[0][1][b, :ql[b]], got[1][1][b, :ql[b]])


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("slopes", [False, True])
def test_capped_rows_do_not_feel_later_tokens_and_other_documents(lib, cap, slopes):
    s, at = 500, 333
    q, k, v = rnd(1, s, 6, 128, gain=1.5), rnd(1, s, 2, 128, seed=2), rnd(1, s, 2, 128, seed=3)
    sl = torch.tensor([2.0 ** -h for h in range(1, 7)], device="cuda") if slopes else None
    plan = binding.Attention(1, s, s, 6, 2, softcap=cap)
    ids = (torch.arange(s, device="cuda") >= at).to(torch.int32)[None]
    got, docs = [], []
    for fill in (0.01, 3000.0):
        k[0, at:] = rnd(s - at, 2, 128, seed=4, gain=fill)
        got.append(plan.run(q, k, v, slopes=sl))
    k[0, at:] = rnd(s - at, 2, 128, seed=4)
    for fill in (0.01, 3000.0):
        k[0, :at] = rnd(at, 2, 128, seed=5, gain=fill)
        docs.append(plan.run(q, k, v, slopes=sl, doc_ids=ids))
    plan.check()
    assert same_bits(got[0][0][:, :at], got[1][0][:, :at]) and same_bits(got[0][1][:, :at], got[1][1][:, :at])
    assert same_bits(docs[0][0][:, at:], docs[1][0][:, at:]) and same_bits(docs[0][1][:, at:], docs[1][1][:, at:])


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("skv", [300, 6000])
def test_capped_rows_do_not_feel_rows_behind_the_queries(lib, cap, skv):
    sq, ql = 300, [41, 300]
    q, k, v = rnd(2, sq, 4, 128, gain=1.5), rnd(2, skv, 2, 128, seed=2), rnd(2, skv, 2, 128, seed=3)
    plan = binding.Attention(2, sq, skv, 4, 2, softcap=cap)
    got = []
    for fill in (0.01, 3000.0):
        q[0, ql[0]:] = rnd(sq - ql[0], 4, 128, seed=4, gain=fill)
        got.append(plan.run(q, k, v, q_len=i32(ql)))
    plan.check()
    for b in range(2):
        assert same_bits(got[0][0][b, :ql[b]], got[1][0][b, :ql[b]]) and same_bits(got[0][1][b, :ql[b]], got[1][1][b, :ql[b]])


@pytest.mark.parametrize("cap", CAPS)
def test_capped_rows_do_not_feel_what_ran_before(lib, cap):
    """Groups of 3 heads fill 126 of a tile's 128 rows, and 3 sequences of a prefix tile fewer still: the rest of the tile holds
    what an earlier kernel left on the SM."""
    big = [rnd(4, 600, 8, 128, gain=g) for g in (0.01, 3000.0)]
    kb = rnd(4, 600, 2, 128, seed=2)
    other = binding.Attention(4, 600, 600, 8, 2)
    q, k, v = rnd(3, 400, 6, 128, gain=1.5), rnd(3, 400, 2, 128, seed=4), rnd(3, 400, 2, 128, seed=5)
    kp, vp = rnd(900, 2, 128, seed=6), rnd(900, 2, 128, seed=7)
    plan = binding.Attention(3, 400, 400, 6, 2, softcap=cap)
    step = binding.PrefixAttention(3, 3, 900, 400, 6, 2, softcap=cap)
    got = []
    for n in range(6):
        other.run(big[n % 2], kb, kb)
        a = plan.run(q, k, v)
        other.run(big[n % 2], kb, kb)
        got.append(a + step.run(q[:, :3], kp, vp, k, v))
    plan.check()
    step.check()
    for g in got[1:]:
        assert all(same_bits(x, y) for x, y in zip(g, got[0]))
