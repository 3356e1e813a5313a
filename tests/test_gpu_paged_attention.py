"""Attention over a cache in pages against the definition in 64 bits: single tokens, chains, trees of drafts."""
import math
import random

import pytest
import torch

import ops_ref as R
from recoverable_quantized_kv_gb300 import binding

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


def rnd(*shape, seed=0, dtype=BF, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + len(shape) + sum(shape))
    return (gain * torch.randn(*shape, generator=g, device="cuda")).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tree(n, seed, wide=2):
    r = random.Random(seed)
    return [r.randint(max(-1, i // wide - 3), i - 1) for i in range(n)]


def line(parents, i):
    found = []
    while i >= 0:
        found.append(i)
        i = parents[i]
    return found


def table_of(need, max_pages, pages, seed=0):
    """Distinct pages for every sequence, in random order; places behind them hold numbers that are no pages."""
    ids, r = random.Random(seed).sample(range(pages), sum(need)), random.Random(seed)
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [r.choice([-1, 10 ** 9, -7]) for _ in range(max_pages - n)])
        at += n
    return i32(rows)


def joined(x, table, b, n):
    """The first n rows of sequence b."""
    page = x.shape[1]
    return x[table[b, :-(-n // page)].long()].flatten(0, 1)[:n]


def expect(q, k, v, table, length, q_len, parents=None, slopes=None, cap=0.0, scale=0.0):
    B, s_q, hq, d = q.shape
    G, res = hq // k.shape[2], {}
    for b in range(B):
        m, n = q_len[b], length[b]
        if m == 0:
            continue
        lines = [line(parents[b], i) if parents else list(range(i, -1, -1)) for i in range(m)]
        pos = torch.tensor([n + len(x) - 1 for x in lines], device="cuda")
        key_pos = torch.cat([torch.arange(n, device="cuda"), pos])
        ok = torch.zeros(m, n + m, dtype=torch.bool)
        ok[:, :n] = True
        for i, x in enumerate(lines):
            ok[i, [n + y for y in x]] = True
        kk, vv = joined(k, table, b, n + m), joined(v, table, b, n + m)
        for h in range(hq):
            res[b, h] = R.attention_rows(q[b, :m, h], kk[:, h // G], vv[:, h // G], ok.cuda(), pos, key_pos,
                                         scale or 1.0 / math.sqrt(d), cap, None if slopes is None else slopes[h].double(),
                                         R.HALF[q.dtype])
    return res


def run_case(length, s_q, hq, hkv, page, dtype=BF, q_len=None, parents=None, one=False, slopes=False, cap=0.0, scale=0.0,
             seed=1, gain=1.5, spare=2, change=None):
    B = len(length)
    ql = q_len or [s_q] * B
    need = [-(-(n + m) // page) for n, m in zip(length, ql)]
    max_pages, pages = max(max(need), -(-s_q // page)) + spare, sum(need) + 3
    q, k, v = rnd(B, s_q, hq, 128, seed=seed, dtype=dtype, gain=gain), rnd(pages, page, hkv, 128, seed=seed + 1, dtype=dtype), \
        rnd(pages, page, hkv, 128, seed=seed + 2, dtype=dtype)
    table = table_of(need, max_pages, pages, seed)
    if change:
        change(q, k, v, table)
    sl = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda") if slopes else None
    plan = binding.PagedAttention(B, s_q, pages, page, max_pages, hq, hkv, dtype=dtype, softcap=cap, scale=scale)
    out, lse = torch.full_like(q, 7.0), torch.full((B, s_q, hq), 7.0, device="cuda")
    par = None if parents is None else i32(parents[0] if one else parents)
    plan.run(q, k, v, table, i32(length), out=out, lse=lse, parents=par, q_len=None if q_len is None else i32(q_len), slopes=sl)
    plan.check()
    R.compare(out, lse, expect(q, k, v, table, length, ql, parents, sl, cap, scale))
    for b in range(B):   # rows behind a sequence's queries keep what they held
        assert torch.all(out[b, ql[b]:] == 7.0) and torch.all(lse[b, ql[b]:] == 7.0)
    return plan, (q, k, v, table, out, lse)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hkv,dtype", [(8, 2, BF), (4, 4, FP)])
@pytest.mark.parametrize("n", [0, 1, 15, 16, 17, 127, 128, 129, 1000, 5000])
def test_single_tokens(lib, page, hq, hkv, dtype, n):
    run_case([n, max(0, n - 5)], 1, hq, hkv, page, dtype)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("nodes", [1, 2, 9, 26, 63, 64])
@pytest.mark.parametrize("n,dtype", [(0, BF), (100, FP), (127, BF), (1500, BF)])
def test_trees(lib, page, nodes, n, dtype):
    run_case([n, n + 3], nodes, 8, 2, page, dtype, parents=[tree(nodes, 1), tree(nodes, 2)])


@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 16, 33, 128])
@pytest.mark.parametrize("nodes", [1, 7, 64])
def test_head_groups(lib, G, nodes):
    run_case([260], nodes, 2 * G, 2, 16, BF, parents=[tree(nodes, 3)])


@pytest.mark.parametrize("wide", [1, 64, 1000])
def test_stars_and_chains_as_trees(lib, wide):
    """A tree that is a chain gives the bits of the chain; one of roots alone, the context and itself."""
    n, m = 700, 40
    if wide == 1:
        a = run_case([n], m, 8, 2, 32, parents=[list(range(-1, m - 1))])[1]
        b = run_case([n], m, 8, 2, 32)[1]
        assert torch.equal(a[4], b[4]) and torch.equal(a[5], b[5])
    else:
        run_case([n], m, 8, 2, 32, parents=[[-1] * m if wide == 64 else [max(-1, i - 9) for i in range(m)]])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cap,slopes,scale", [(30.0, False, 0.0), (0.0, True, 0.0), (5.0, True, 0.25), (0.0, False, 0.03),
                                              (200.0, True, 0.0)])
@pytest.mark.parametrize("n,nodes", [(700, 1), (90, 26), (1300, 61), (0, 64)])
def test_scores_capped_biased_scaled(lib, dtype, cap, slopes, scale, n, nodes):
    run_case([n, n + 41], nodes, 8, 2, 16, dtype, cap=cap, slopes=slopes, scale=scale, parents=[tree(nodes, 5), tree(nodes, 6)])


@pytest.mark.parametrize("s_q", [2, 64, 65, 200, 700])
@pytest.mark.parametrize("cap,slopes,dtype", [(0.0, False, BF), (20.0, True, FP)])
def test_chains(lib, s_q, cap, slopes, dtype):
    """A prompt's chunk, and a whole prompt."""
    run_case([0, 333], s_q, 8, 2, 64, dtype, cap=cap, slopes=slopes)


@pytest.mark.parametrize("s_q,n", [(200, 9000), (33, 20000), (300, 33000)])
def test_last_chunk_of_a_long_context(lib, s_q, n):
    run_case([n], s_q, 8, 2, 16, BF)
    run_case([n - 77, 5], s_q, 4, 4, 128, FP, cap=15.0)


def test_ragged_batches(lib):
    """Sequences without tokens, without queries, without either; one tree for all or a tree each."""
    length, ql = [500, 0, 0, 128, 300, 1, 77], [9, 3, 0, 0, 1, 9, 8]
    run_case(length, 9, 8, 2, 16, q_len=ql)
    run_case(length, 9, 8, 2, 16, q_len=ql, parents=[tree(9, b) for b in range(7)], slopes=True)
    run_case(length, 9, 8, 2, 32, q_len=ql, parents=[tree(9, 4)] * 7, one=True)


def test_many_sequences_of_all_lengths(lib):
    g = torch.Generator().manual_seed(5)
    length = [int(x) for x in torch.randint(0, 1501, (70,), generator=g)]
    length[0], length[33], length[34], length[69] = 0, 0, 1, 1500
    run_case(length, 1, 8, 2, 16)
    run_case(length[:40], 13, 16, 8, 64, FP, parents=[tree(13, b) for b in range(40)])


def test_more_units_than_sms_drawn_again_and_again(lib):
    """240 units of all lengths drawn one by one, sequences without queries or tokens among them; the count starts again for the
    next call, and for replays of a captured one."""
    g = torch.Generator().manual_seed(7)
    length = [int(x) for x in torch.randint(0, 901, (60,), generator=g)]
    ql = [int(x) for x in torch.randint(0, 6, (60,), generator=g)]
    length[0], length[50], ql[3], ql[59] = 0, 900, 0, 0
    plan, (q, k, v, table, out, lse) = run_case(length, 5, 4, 4, 32, q_len=ql, parents=[tree(5, b) for b in range(60)])
    args, kw = (q, k, v, table, i32(length)), dict(parents=i32([tree(5, b) for b in range(60)]), q_len=i32(ql))
    o, s = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    for _ in range(3):
        plan.run(*args, out=o, lse=s, **kw)
        assert torch.equal(o, out) and torch.equal(s, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            plan.run(*args, out=o, lse=s, **kw)
    for _ in range(3):
        o.fill_(7.0)
        graph.replay()
        assert torch.equal(o, out) and torch.equal(s, lse)
    plan.check()


@pytest.mark.parametrize("b,nodes,n,hq,hkv", [(1, 16, 4200, 32, 8), (1, 32, 4200, 32, 8), (1, 1, 20000, 4, 1), (2, 60, 2000, 32, 8),
                                              (13, 64, 3000, 8, 2), (1, 3, 33000, 6, 2)])
def test_parts_merged_by_one_to_sixteen_warps(lib, b, nodes, n, hq, hkv):
    """Few rows of many parts to many rows of few, counts of rows that are no multiple of four, one row without parts."""
    run_case([n - 77 * i for i in range(b)], nodes, hq, hkv, 64, parents=[tree(nodes, 20 + i) for i in range(b)])
    if b > 1:
        run_case([n] + [5] * (b - 1), nodes, hq, hkv, 16, FP, q_len=[nodes] + [max(1, nodes - 7 * i) for i in range(1, b)])


@pytest.mark.parametrize("n,nodes,hkv,page", [(40000, 26, 2, 16), (131000, 1, 1, 16), (70000, 64, 1, 128)])
def test_long_contexts(lib, n, nodes, hkv, page):
    """Units cut into parts, tables longer than the copying warp holds, trees cut by a tile's end."""
    run_case([n], nodes, 4 * hkv, hkv, page, parents=[tree(nodes, 8)])
    run_case([n - n % 128 + 120, 700], nodes, 4 * hkv, hkv, page, parents=[tree(nodes, 8), tree(nodes, 9)])


@pytest.mark.parametrize("form", ["fused", "heads", "layers"])
def test_pools_of_other_strides(lib, form):
    page, h, n, m = 32, 2, 333, 12
    pages = 20
    if form == "fused":
        x = rnd(pages, 2, page, h, 128)
        k, v = x[:, 0], x[:, 1]
    elif form == "heads":
        k, v = rnd(pages, h, page, 128).transpose(1, 2), rnd(pages, h, page, 128, seed=4).transpose(1, 2)
    else:
        x = rnd(pages, page, 3, 2 * h, 128)
        k, v = x[:, :, 1, :h], x[:, :, 2, h:]
    table, par = table_of([11], 11, pages), tree(m, 2)
    fused = rnd(1, m, 3 * 8, 128, seed=3)
    q = fused[:, :, 8:16]
    out = torch.full((8, 1, m, 128), 7.0, dtype=BF, device="cuda").permute(1, 2, 0, 3)
    plan = binding.PagedAttention(1, m, pages, page, 11, 8, h)
    o, lse = plan.run(q, k, v, table, i32([n]), out=out, parents=i32([par]))
    plan.check()
    assert o is out
    R.compare(out, lse, expect(q, k, v, table, [n], [m], [par]))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("cap", [0.0, 9.0])
def test_unseen_places_may_hold_anything(lib, dtype, bad, cap):
    """Rows of the last page behind the last query's, other branches, whole pages of others: rows that do not see them keep
    their bounds; rows that do get what the definition gives."""
    n, m, page = 290, 20, 32
    par = [tree(m, 11), tree(m, 12)]

    def behind(q, k, v, table):
        for b, used in enumerate((n + m, 40 + m)):
            k[table[b, used // page].long(), used % page:] = bad
            v[table[b, used // page].long(), used % page:] = bad
        free = sorted(set(range(k.shape[0])) - set(table[table >= 0].tolist()))
        k[free] = bad
        v[free] = bad

    run_case([n, 40], m, 4, 2, page, dtype, parents=par, change=behind, cap=cap, spare=0)

    def branch(q, k, v, table):
        at = n + 7
        v[table[0, at // page].long(), at % page, 0, 5] = bad

    _, (_, _, _, _, out, _) = run_case([n, 40], m, 4, 2, page, dtype, parents=par, change=branch, cap=cap)
    sees = torch.tensor([7 in line(par[0], i) for i in range(m)], device="cuda")
    assert not torch.isfinite(out[0, sees][:, :2, 5].float()).any() and torch.isfinite(out[0, ~sees].float()).all()

    def key(q, k, v, table):
        at = n + 7
        k[table[0, at // page].long(), at % page, 1] = bad

    _, (_, _, _, _, out, _) = run_case([n, 40], m, 4, 2, page, dtype, parents=par, change=key, cap=0.0) \
        if math.isnan(bad) else (None, (None,) * 4 + (torch.zeros(1, m, 4, 128, device="cuda"), None))
    assert torch.isfinite(out[0, ~sees].float()).all()


@pytest.mark.parametrize("s_q,n", [(20, 300), (150, 700), (3, 0), (150, 5000)])
@pytest.mark.parametrize("dtype,bad", [(BF, math.nan), (FP, math.inf)])
def test_a_later_tokens_value_in_a_chain(lib, s_q, n, dtype, bad):
    """Rows before the token are unchanged to the bound: whole units and parts of them, over pages."""
    page, at = 16, n + s_q // 2

    def later(q, k, v, table):
        v[table[0, at // page].long(), at % page, 1, 70] = bad

    out = run_case([n, 44], s_q, 4, 2, page, dtype, change=later)[1][4]
    assert torch.isfinite(out[0, :s_q // 2].float()).all() and not torch.isfinite(out[0, s_q // 2:, 2:, 70].float()).any()


def test_logits_beyond_whole_numbers(lib):
    """Rows whose largest logit is past 2^23: worked out again over pages and lines of the tree."""
    n, m, page = 200, 10, 16
    par = [tree(m, 3)]
    q, k, v = rnd(1, m, 4, 128), rnd(20, page, 2, 128, seed=2), rnd(20, page, 2, 128, seed=3)
    table = table_of([14], 14, 20)
    plan = binding.PagedAttention(1, m, 20, page, 14, 4, 2, scale=1e7)
    out, lse = plan.run(q, k, v, table, i32([n]), parents=i32(par))
    plan.check()
    for i in range(m):
        own = line(par[0], i)
        keys = torch.cat([torch.arange(n), torch.tensor([n + x for x in own])]).cuda()
        for h in range(4):
            kk, vv = joined(k, table, 0, n + m)[keys, h // 2].double(), joined(v, table, 0, n + m)[keys, h // 2]
            s = kk @ q[0, i, h].double()
            top, second = s.topk(2).values.tolist()
            # logits are off by 130 roundings of the sum of magnitudes; where the first leads by more, it is alone
            if (top - second) > 2 * 130 * 2.0 ** -24 * float((kk.abs() @ q[0, i, h].double().abs()).max()):
                assert torch.equal(out[0, i, h], vv[s.argmax()])


def test_faults_are_reported(lib):
    """Lengths, counts, parents and pages out of range: clamped, reported, nothing outside read or written."""
    page, pages, B, m = 16, 12, 2, 5
    q, k, v = rnd(B, m, 4, 128), rnd(pages, page, 2, 128, seed=2), rnd(pages, page, 2, 128, seed=3)
    table, par = table_of([5, 5], 5, pages), [[-1, 0, 1, 1, 0]] * B
    plan = binding.PagedAttention(B, m, pages, page, 5, 4, 2)

    def call(length, q_len=None, parents=par, t=table):
        out, lse = plan.run(q, k, v, t, i32(length), parents=None if parents is None else i32(parents),
                            q_len=None if q_len is None else i32(q_len))
        try:
            plan.check()
            return 0, out, lse
        except binding.QEvictError as e:
            return e.word, out, lse

    word, out, lse = call([75, 75])
    assert word == 0
    R.compare(out, lse, expect(q, k, v, table, [75, 75], [m, m], par))
    for length, ql, want in (([76, 75], None, [75, 75]), ([75, -3], None, [75, 0]), ([2 ** 31 - 1, 75], None, [75, 75]),
                             ([75, 75], [m + 1, m], [75, 75])):
        word, out, lse = call(length, ql)
        assert word == 8
        R.compare(out, lse, expect(q, k, v, table, want, [m, m], par))
    for wrong in (1, 4, -2, 2 ** 31 - 1, -2 ** 31):   # of node 1: itself, a later one, none
        word, out, lse = call([75, 75], parents=[[-1, wrong, 1, 1, 0], par[1]])
        assert word == 8
        R.compare(out, lse, expect(q, k, v, table, [75, 75], [m, m], [[-1, -1, 1, 1, 0], par[1]]))
    for wrong in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 2] = wrong
        word, out, lse = call([75, 75], t=t)
        t[1, 2] = 0
        assert word == 8
        R.compare(out, lse, expect(q, k, v, t, [75, 75], [m, m], par))


def test_results_repeat_and_do_not_depend_on_pages(lib):
    """The same sequences in other pages, and in pages of another size."""
    n, m = 3000, 24
    dense = rnd(2, n + m, 2, 128, seed=6), rnd(2, n + m, 2, 128, seed=7)
    q, par, first = rnd(2, m, 8, 128), i32([tree(m, 1), tree(m, 2)]), None
    for page, seed in ((16, 1), (16, 2), (64, 3), (128, 4), (128, 4)):
        need = -(-(n + m) // page)
        pages = 2 * need + 1
        table = table_of([need, need], 200 * 16 // page, pages, seed)
        k, v = rnd(pages, page, 2, 128, seed=seed), rnd(pages, page, 2, 128, seed=seed + 9)
        for x, y in ((k, dense[0]), (v, dense[1])):
            for b in range(2):
                for e in range(need):
                    rows = y[b, e * page:(e + 1) * page]
                    x[table[b, e].long(), :len(rows)] = rows
        plan = binding.PagedAttention(2, m, pages, page, 200 * 16 // page, 8, 2)
        out, lse = plan.run(q, k, v, table, i32([n, n - 500]), parents=par)
        plan.check()
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_inputs_that_ask_for_a_gradient_are_refused(lib):
    q, k, v = rnd(1, 1, 4, 128), rnd(4, 16, 2, 128), rnd(4, 16, 2, 128)
    plan, args = binding.PagedAttention(1, 1, 4, 16, 4, 4, 2), (i32([[0, 1, 2, 3]]), i32([20]))
    for i in range(3):
        x = [q, k, v]
        x[i] = x[i].clone().requires_grad_()
        with pytest.raises(binding.QEvictError):
            plan.run(*x, *args)
        with torch.no_grad():
            plan.run(*x, *args)
    with pytest.raises(binding.QEvictError):
        plan.run(q, k, v, args[0][:, :3], args[1])
    with pytest.raises(binding.QEvictError):
        plan.run(q, k, v, None, args[1])
    with pytest.raises(binding.QEvictError):
        plan.run(q, k[:, :8], v, *args)
    with pytest.raises(binding.QEvictError):
        plan.run(q, k, v, *args, parents=i32([[0, 1]]))


def test_streams_graphs_and_plans_side_by_side(lib):
    """Two plans on two streams at once, and a captured call replayed after its inputs changed in place."""
    n, m, page = 2000, 16, 32
    par = tree(m, 4)
    q, k, v = rnd(1, m, 8, 128), rnd(70, page, 2, 128, seed=2), rnd(70, page, 2, 128, seed=3)
    table, length = table_of([64], 64, 70), i32([n])
    make = lambda: binding.PagedAttention(1, m, 70, page, 64, 8, 2)   # noqa: E731
    want = make().run(q, k, v, table, length, parents=i32([par]))
    plans, streams = [make(), make()], [torch.cuda.Stream(), torch.cuda.Stream()]
    parents = i32([par])
    torch.cuda.synchronize()
    outs = [p.run(q, k, v, table, length, parents=parents, stream=s) for _ in range(5) for p, s in zip(plans, streams)]
    torch.cuda.synchronize()
    for out, lse in outs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    g, plan = torch.cuda.CUDAGraph(), make()
    with torch.cuda.graph(g):
        out, lse = plan.run(q, k, v, table, length, parents=parents)
    length.fill_(n - 333)
    parents[0, 3] = -1
    g.replay()
    plan.check()
    par[3] = -1
    R.compare(out, lse, expect(q, k, v, table, [n - 333], [m], [par]))


def test_a_decoding_loop_with_drafts(lib):
    """Rotations, rows appended, attention, accepted paths, forks and a compaction, against dense attention over what each
    sequence has kept: bit for bit the same keys, outputs within the bound."""
    layers, page, hq, h, B, m = 2, 16, 8, 2, 3, 7
    r = random.Random(1)
    cache = binding.PagedCache(layers, 40, page, h, B, 9)
    plan = binding.PagedAttention(B, m, 40, page, 9, hq, h)
    rope = binding.Rope(binding.rope_table(200))
    kept = [[[torch.zeros(0, h, 128, dtype=BF, device="cuda") for _ in range(2)] for _ in range(layers)] for _ in range(B)]
    for step in range(14):
        par = [tree(m, 100 * step + b) for b in range(B)]
        lens = [kept[b][0][0].shape[0] for b in range(B)]
        pos = i32([[lens[b] + len(line(par[b], i)) - 1 for i in range(m)] for b in range(B)])
        cache.reserve(m)
        rows = []
        for l in range(layers):
            q, k, v = rnd(B, m, hq, 128, seed=step * 9 + l), rnd(B, m, h, 128, seed=step * 9 + l + 3), \
                rnd(B, m, h, 128, seed=step * 9 + l + 6)
            q, k = rope.apply(q, k, positions=pos)
            cache.append(k, v, layer=l)
            rows.append((k, v))
            out, lse = plan.run(q, cache.k[l], cache.v[l], cache.table, cache.length, parents=i32(par))
            dense = [torch.stack([torch.cat([kept[b][l][x], rows[l][x][b],
                                             torch.zeros(200 - lens[b], h, 128, dtype=BF, device="cuda")]) for b in range(B)])
                     for x in range(2)]
            ident = torch.arange(B, device="cuda")[:, None]
            R.compare(out, lse, expect(q, *dense, ident, lens, [m] * B, par), f"step {step} layer {l}")
        paths = [line(par[b], r.randrange(m))[::-1] for b in range(B)]
        cache.accept(i32([len(p) for p in paths]), i32([p + [0] * (m - len(p)) for p in paths]))
        for b in range(B):
            for l in range(layers):
                for x in range(2):
                    kept[b][l][x] = torch.cat([kept[b][l][x], rows[l][x][b][paths[b]]])
        if step % 3 == 2:
            src = [r.randrange(B) for _ in range(B)]
            cache.select(i32(src))
            kept = [[[kept[s][l][x] for x in range(2)] for l in range(layers)] for s in src]
        if step == 9:
            cache.trim(i32([5, -1, 30]))
            for b, n in ((0, 5), (2, 30)):
                kept[b] = [[x[:n] for x in pair] for pair in kept[b]]
        if step % 5 == 4:
            cache.compact()
        cache.check()
        for b in range(B):
            for l in range(layers):
                for x, name in enumerate("kv"):
                    n = kept[b][l][x].shape[0]
                    assert int(cache.length[b]) == n
                    if n:
                        assert torch.equal(joined(getattr(cache, name)[l], cache.table, b, n), kept[b][l][x])
    plan.check()
