"""Attention over pages: rows of a tree beside a key or value of another branch that is no number, plain and capped."""
import math

import pytest
import torch

import ops_ref as R
from recoverable_quantized_kv_gb300 import binding
from test_gpu_paged_attention import BF, FP, expect, i32, line, rnd, table_of, tree

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("cap", [0.0, 9.0, 100.0])
@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("n,m,hq,page", [(290, 20, 4, 32), (120, 33, 2, 16), (5000, 61, 8, 64), (0, 64, 2, 128)])
def test_a_key_of_another_branch(lib, dtype, bad, cap, slopes, n, m, hq, page):
    """The key of one node, one channel of it or all, is not finite: rows that do not see it are what they are with a key of
    zeros there; rows that do are not looked at."""
    par, node = [tree(m, 11), tree(m, 12)], m // 3
    need = [-(-(x + m) // page) for x in (n, 40)]
    pages = sum(need) + 2
    q, k, v = rnd(2, m, hq, 128, dtype=dtype, gain=1.5), rnd(pages, page, 2, 128, seed=2, dtype=dtype), \
        rnd(pages, page, 2, 128, seed=3, dtype=dtype)
    table, length = table_of(need, max(need), pages), [n, 40]
    sl = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda") if slopes else None
    at = (table[0, (n + node) // page].long(), (n + node) % page)
    k[at[0], at[1]] = 0.0
    want = expect(q, k, v, table, length, [m, m], par, sl, cap)
    sees = torch.tensor([node in line(par[0], i) for i in range(m)], device="cuda")
    assert sees.any() and not sees.all()
    plan = binding.PagedAttention(2, m, pages, page, max(need), hq, 2, dtype=dtype, softcap=cap)
    for channels in (slice(None), slice(7, 8)):
        k[at[0], at[1], :, channels] = bad
        out, lse = plan.run(q, k, v, table, i32(length), parents=i32(par), slopes=sl)
        plan.check()
        R.compare(out, lse, {key: x for key, x in want.items() if key[0] == 1}, "other sequence")
        for (b, h), x in want.items():
            if b == 0:
                o, ls, eo, el = (y[~sees] for y in x)
                R.compare(out[:1, :m][:, ~sees], lse[:1, :m][:, ~sees], {(0, h): (o, ls, eo, el)}, f"channels {channels}")
        k[at[0], at[1], :, channels] = 0.0
