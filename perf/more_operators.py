"""Performance cases of the paged KV cache: attention of drafted trees, chains and single tokens over pages, and the
operators that keep the pages (writing rows, accepting drafted rows, forking with copy on write, compaction).

Every case runs in two forms on the same inputs: the plain form (elementary torch operations, attention in fp32) and,
with own = True, the library's operators through the binding.  A cache is a pool of pages of `page` tokens for each
layer, k and v [layers][pages][page][h_kv][128], a table [batch][max_pages] of page numbers (-1: none) and the lengths
of the sequences; refs counts the table entries of each page, a page with none is free.  Shapes are those of the
package's workloads (8 or 32 query heads over 2 or 8 KV heads of 128 channels; 1K, 4K and 33K contexts) and odd ones.
"""
import math
import random

import torch

own = False

D = 128   # head dimension of every workload of the package
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a small tree of drafts for one sequence and a short context: latency
        {"name": "tree_b1_1k", "op": "attn", "b": 1, "nodes": 8, "ctx": 1040, "hq": 8, "hkv": 2, "page": 16,
         "type": "bf16", "cap": 0.0, "alibi": False, "tree": True, "ragged": False},
        # an ordinary decode step: one token of 64 sequences of different lengths, small pages
        {"name": "tokens_b64_4k", "op": "attn", "b": 64, "nodes": 1, "ctx": 4160, "hq": 32, "hkv": 8, "page": 16,
         "type": "bf16", "cap": 0.0, "alibi": False, "tree": False, "ragged": True},
        # trees of 26 drafts for 16 long contexts: memory bound
        {"name": "tree_b16_33k", "op": "attn", "b": 16, "nodes": 26, "ctx": 33024, "hq": 32, "hkv": 8, "page": 64,
         "type": "bf16", "cap": 0.0, "alibi": False, "tree": True, "ragged": True},
        # trees of up to 61 drafts, odd lengths, capped scores and distance biases, one KV head per query head
        {"name": "tree_b3_8209_cap_alibi", "op": "attn", "b": 3, "nodes": 61, "ctx": 8209, "hq": 8, "hkv": 8, "page": 32,
         "type": "fp16", "cap": 30.0, "alibi": True, "tree": True, "ragged": True},
        # one layer of a decode step writes its rows: latency
        {"name": "append_step_b64", "op": "append", "layers": 1, "b": 64, "n": 1, "ctx": 515, "hkv": 8, "page": 16,
         "type": "bf16", "ragged": False},
        # a prefill's keys and values of 8 layers are taken over into pages, prompts of different odd lengths
        {"name": "append_prompts_8l_2x4099", "op": "append", "layers": 8, "b": 2, "n": 4099, "ctx": 0, "hkv": 8, "page": 64,
         "type": "fp16", "ragged": True},
        # drafts of a small batch accepted in all 32 layers
        {"name": "accept_b4_32l", "op": "accept", "layers": 32, "b": 4, "nodes": 26, "most": 5, "ctx": 131, "hkv": 2,
         "page": 16, "type": "bf16"},
        # drafts of a large batch accepted in 8 layers
        {"name": "accept_b256_8l", "op": "accept", "layers": 8, "b": 256, "nodes": 64, "most": 8, "ctx": 100, "hkv": 8,
         "page": 64, "type": "bf16"},
        # a beam step: 3 of 8 beams go on, the others become copies of them and of their last, partly filled pages
        {"name": "fork_beams_b8", "op": "fork", "layers": 32, "b": 8, "keep": 3, "ctx": 407, "new": 1, "hkv": 2, "page": 16,
         "type": "fp16"},
        # 4 prompts, each forked into 16 samples
        {"name": "fork_samples_b64", "op": "fork", "layers": 16, "b": 64, "keep": 4, "ctx": 1125, "new": 2, "hkv": 8,
         "page": 128, "type": "bf16"},
        # pages moved down after sequences ended: a small pool
        {"name": "compact_300", "op": "compact", "layers": 4, "pages": 300, "used": 0.6, "b": 7, "hkv": 2, "page": 16,
         "type": "bf16"},
        # and a large one
        {"name": "compact_700_8l", "op": "compact", "layers": 8, "pages": 700, "used": 0.55, "b": 37, "hkv": 8, "page": 64,
         "type": "fp16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "tokens", "tokens", "chain", "append", "accept", "fork", "compact"])
    typ, page = rng.choice(["bf16", "bf16", "fp16"]), rng.choice([16, 32, 64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    if op in ("attn", "tokens", "chain"):
        hq, hkv = rng.choice([(8, 2), (32, 8), (8, 8), (16, 8), (32, 4), (4, 1), (6, 2)])
        ctx = _log_int(rng, 1, 65536)
        nodes = 1 if op == "tokens" else _log_int(rng, 2, 300) if op == "chain" else rng.randint(2, 64)
        b = _log_int(rng, 1, max(1, min(64, 400000 // (ctx + nodes))))
        nodes = max(1, min(nodes, 16 * 20000 * 26 * 32 // (b * (ctx + nodes) * hq)))
        return {"op": "attn", "b": b, "nodes": nodes, "ctx": ctx, "hq": hq, "hkv": hkv, "page": page, "type": typ,
                "cap": rng.choice([0.0, 0.0, 30.0, 50.0]), "alibi": rng.random() < 0.3, "tree": op == "attn",
                "ragged": rng.random() < 0.6}
    layers = _log_int(rng, 1, 32)
    row = layers * hkv * D * 2   # bytes of a token's keys in all layers
    if op == "append":
        n = _log_int(rng, 1, 4096)
        b = _log_int(rng, 1, max(1, min(256, 100000000 // (row * (n + page)))))
        if row * n * b > 100000000:
            layers = 1
        return {"op": "append", "layers": layers, "b": b, "n": n, "ctx": _log_int(rng, 1, 600) - 1, "hkv": hkv,
                "page": page, "type": typ, "ragged": rng.random() < 0.5}
    if op == "accept":
        nodes = rng.randint(9, 64)
        b = _log_int(rng, 1, max(1, min(256, 400000000 // (row * (nodes + 200)))))
        return {"op": "accept", "layers": layers, "b": b, "nodes": nodes, "most": rng.randint(2, 8),
                "ctx": _log_int(rng, 1, 200) - 1, "hkv": hkv, "page": page, "type": typ}
    if op == "fork":
        ctx = _log_int(rng, 2, 2000)
        b = _log_int(rng, 2, max(2, min(64, 400000000 // (row * (ctx + page)))))
        return {"op": "fork", "layers": layers, "b": b, "keep": rng.randint(1, max(1, b // 2)), "ctx": ctx,
                "new": rng.randint(1, 40), "hkv": hkv, "page": page, "type": typ}
    pages = _log_int(rng, 20, max(21, min(4000, 700000000 // (row * page))))
    return {"op": "compact", "layers": layers, "pages": pages, "used": rng.uniform(0.2, 0.95), "b": _log_int(rng, 1, 64),
            "hkv": hkv, "page": page, "type": typ}


# ------------------------------------------------------------------------------------------------ sizes of a case
# (functions of the case alone, so that its work is known without its inputs)

def _lengths(c):
    """Tokens in the cache of every sequence: between a quarter of the longest and all of it in a ragged batch."""
    b, n = c["b"], c["ctx"]
    if c["op"] == "attn":
        return [n - (i * n * 3) // (4 * b) for i in range(b)] if c["ragged"] else [n] * b
    if c["op"] == "fork":   # survivors of different lengths; the others' own pages are dropped
        return [max(1, n - 7 * (i % 5)) for i in range(b)]
    return [n + (i * 5) % 23 for i in range(b)]


def _new_rows(c):
    """New tokens of every sequence: queries, or rows to write."""
    most = c["nodes"] if c["op"] in ("attn", "accept") else c["n"]
    if c["op"] == "accept" or not c["ragged"]:
        return [most] * c["b"]
    return [most - (i % 3) * (most // 4) for i in range(c["b"])]


def _parents(c, i):
    """The tree of sequence i: every node's parent among the nodes before it, -1 for the context's last token."""
    rng = random.Random(1000 * c["nodes"] + i)
    return [-1 if n == 0 else rng.randint(max(-1, n // 4 - 2), n // 2) if n > 2 else rng.randint(-1, n - 1)
            for n in range(c["nodes"])]


def _ancestors(parents, n):
    """n and its ancestors."""
    found = []
    while n >= 0:
        found.append(n)
        n = parents[n]
    return found


def _paths(c):
    """Accepted nodes of every sequence: the first one and later ones that lie behind the places they go to."""
    rng = random.Random(c["nodes"] * 100 + c["most"])
    return [[0] + sorted(rng.sample(range(c["most"], c["nodes"]), min(n, c["nodes"] - c["most"])))
            for n in (rng.randint(0, c["most"] - 1) for _ in range(c["b"]))]


def _sources(c):
    """Where every sequence's pages come from: the first sequence of each of `keep` groups goes on, the others become
    copies of it."""
    size = -(-c["b"] // c["keep"])
    return [i - i % size for i in range(c["b"])]


def _used(c):
    """Which pages of a pool are in use before a compaction."""
    rng = random.Random(c["pages"])
    used = [rng.random() < c["used"] for _ in range(c["pages"])]
    used[rng.randrange(c["pages"])] = True
    return used


def work(c):
    size, hkv = 2, c["hkv"]
    if c["op"] == "attn":   # keys and values of every sequence read once, queries read, outputs and lse written
        ctx, new = _lengths(c), _new_rows(c)
        pairs = 0
        for i, (n, m) in enumerate(zip(ctx, new)):
            par = _parents(c, i) if c["tree"] else list(range(-1, c["nodes"] - 1))
            pairs += n * m + (sum(len(_ancestors(par, x)) for x in range(m)) if c["tree"] else m * (m + 1) // 2)
        rows = sum(new) * c["hq"]
        return {"bytes": 2 * hkv * D * size * (sum(ctx) + sum(new)) + rows * (2 * D * size + 4),
                "flops": 4 * D * c["hq"] * pairs}
    token = 2 * c["layers"] * hkv * D * size   # keys and values of a token in all layers
    if c["op"] == "append":
        return {"bytes": 2 * token * sum(_new_rows(c)), "flops": 0}
    if c["op"] == "accept":
        return {"bytes": 2 * token * sum(x != j for p in _paths(c) for j, x in enumerate(p)) + 8 * c["b"], "flops": 0}
    if c["op"] == "fork":   # rows of the pages that two sequences would write to; tables
        src, n = _sources(c), _lengths(c)
        rows = sum(n[s] % c["page"] for i, s in enumerate(src) if s != i)
        return {"bytes": 2 * token * rows + 8 * sum(-(-(n[s] + c["new"]) // c["page"]) for s in src), "flops": 0}
    used = _used(c)
    return {"bytes": 2 * token * c["page"] * sum(used[sum(used):]) + 4 * c["pages"], "flops": 0}


# ------------------------------------------------------------------------------------------------ inputs

def _heads_of(gen, *shape, typ, gain=0.0, plant=None):
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
    if plant is not None:
        x = x + gain * plant
    return x.to(TYPES[typ])


def _ints(x):
    return torch.tensor(x, device="cuda", dtype=torch.int32)


def _table(gen, held, max_pages, pages, among=None):
    """Distinct pages in random order for every sequence."""
    ids = torch.randperm(pages, generator=gen, device="cuda") if among is None else among
    slot = torch.arange(max_pages, device="cuda")[None]
    held = torch.tensor(held, device="cuda")
    at = (held.cumsum(0) - held)[:, None] + slot
    return torch.where(slot < held[:, None], ids[at.clamp(max=len(ids) - 1)], -1).to(torch.int32)


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c}
    b, page, hkv, typ = c["b"], c["page"], c["hkv"], c["type"]
    layers = c.get("layers", 1)
    up = lambda n: -(-n // page)   # noqa: E731
    if c["op"] == "compact":
        used = torch.tensor(_used(c), device="cuda").nonzero()[:, 0]
        ids = used[torch.randperm(len(used), generator=gen, device="cuda")]
        held = [len(used) // b + (i < len(used) % b) for i in range(b)]
        pages, max_pages, lens = c["pages"], max(held), [max(0, n * page - i % page) for i, n in enumerate(held)]
        table = _table(gen, held, max_pages, pages, ids)
    else:
        lens = _lengths(c)
        extra = [c["new"]] * b if c["op"] == "fork" else _new_rows(c)
        held = [up(n) if c["op"] == "fork" else up(n + m) for n, m in zip(lens, extra)]
        max_pages = max(up(n + m) for n, m in zip(lens, extra)) + 1
        pages = sum(up(n + m) for n, m in zip(lens, extra)) + b + 3
        table = _table(gen, held, max_pages, pages)
    u = torch.randn(D, generator=gen, device="cuda")
    u = u / u.norm()
    if c["op"] == "attn":   # some pages of keys lie along a direction that the queries share, as retrieved passages do
        hit = (torch.rand(1, pages, 1, 1, 1, generator=gen, device="cuda") < 0.05) * u
        st["k"] = _heads_of(gen, layers, pages, page, hkv, D, typ=typ, gain=4.0, plant=hit)
    else:
        st["k"] = _heads_of(gen, layers, pages, page, hkv, D, typ=typ)
    st["v"] = _heads_of(gen, layers, pages, page, hkv, D, typ=typ)
    st["table"], st["length"] = table, _ints(lens)
    if own and c["op"] != "attn":
        from recoverable_quantized_kv_gb300 import binding
        st["cache"] = binding.PagedCache(layers, pages, page, hkv, b, max_pages, dtype=TYPES[typ], k=st["k"], v=st["v"])
        st["cache"].load(table, st["length"])
    if c["op"] == "attn":
        st["q"] = _heads_of(gen, b, c["nodes"], c["hq"], D, typ=typ, gain=4.0, plant=u)
        st["q_len"] = _ints(_new_rows(c)) if c["ragged"] else None
        st["parents"] = _ints([_parents(c, i) for i in range(b)]) if c["tree"] else None
        st["slopes"] = None
        if c["alibi"]:   # one slope per head, a geometric sequence
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["hq"]) for h in range(c["hq"])], device="cuda")
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(b, c["nodes"], c["hq"], device="cuda", dtype=torch.float32)
        if own:
            from recoverable_quantized_kv_gb300 import binding
            st["plan"] = binding.PagedAttention(b, c["nodes"], pages, page, max_pages, c["hq"], hkv, dtype=TYPES[typ],
                                                softcap=c["cap"])
    elif c["op"] == "append":
        st["k_new"] = _heads_of(gen, layers, b, c["n"], hkv, D, typ=typ)
        st["v_new"] = _heads_of(gen, layers, b, c["n"], hkv, D, typ=typ)
        st["n"] = _ints(_new_rows(c)) if c["ragged"] else None
    elif c["op"] == "accept":
        paths = _paths(c)
        st["count"] = _ints([len(p) for p in paths])
        st["path"] = _ints([p + [-1] * (c["most"] - len(p)) for p in paths])
    elif c["op"] == "fork":
        st["src"], st["new"] = _ints(_sources(c)), _ints([c["new"]] * b)
    elif own:
        st["saved"] = st["cache"].state.clone()
    return st


# ------------------------------------------------------------------------------------------------ the two forms

def run(st):
    c = st["case"]
    return _own(c, st) if own else _plain(c, st)


def _own(c, st):
    if c["op"] == "attn":
        return st["plan"].run(st["q"], st["k"][0], st["v"][0], st["table"], st["length"], out=st["out"], lse=st["lse"],
                              parents=st["parents"], q_len=st["q_len"], slopes=st["slopes"])
    cache = st["cache"]
    if c["op"] == "append":   # the rows stand behind the sequences' lengths until they are accepted
        cache.append(st["k_new"], st["v_new"], n=st["n"])
        return cache.k, cache.v
    if c["op"] == "accept":
        cache.length.copy_(st["length"])   # as before the step
        cache.accept(st["count"], st["path"])
        return cache.k, cache.v, cache.length
    if c["op"] == "fork":
        cache.select(st["src"])
        cache.reserve(st["new"])
        return cache.k, cache.v, cache.table, cache.length, cache.refs
    cache.state.copy_(st["saved"])         # as before the compaction
    cache.compact()
    return cache.k, cache.v, cache.table, cache.refs


def _plain(c, st):
    if c["op"] == "attn":
        return _plain_attention(c, st)
    k, v, table, page = st["k"], st["v"], st["table"].long(), c["page"]
    length = st["length"].long()
    rows_of = torch.arange(c["b"], device="cuda")[:, None]
    if c["op"] == "append":
        i = torch.arange(c["n"], device="cuda")[None].expand(c["b"], -1)
        at = length[:, None] + i
        pg, off = table[rows_of, (at // page).clamp(max=table.shape[1] - 1)], at % page
        if st["n"] is None:
            k[:, pg, off], v[:, pg, off] = st["k_new"], st["v_new"]
        else:
            ok = i < st["n"][:, None]
            k[:, pg[ok], off[ok]], v[:, pg[ok], off[ok]] = st["k_new"][:, ok], st["v_new"][:, ok]
        return k, v
    if c["op"] == "accept":
        j = torch.arange(c["most"], device="cuda")[None]
        dst = length[:, None] + j
        src = torch.where(j < st["count"][:, None], length[:, None] + st["path"], dst)   # other rows stay
        at = lambda x: (table[rows_of, x // page], x % page)   # noqa: E731
        (ps, os), (pd, od) = at(src), at(dst)
        ok = (j < st["count"][:, None])
        ps, os, pd, od = ps[ok], os[ok], pd[ok], od[ok]
        k[:, pd, od], v[:, pd, od] = k[:, ps, os], v[:, ps, os]
        return k, v, (length + st["count"]).to(torch.int32)
    pages = k.shape[1]
    slot = torch.arange(table.shape[1], device="cuda")[None]
    if c["op"] == "fork":
        src = st["src"].long()
        length, have = length[src], (length[src] + page - 1) // page
        table = torch.where(slot < have[:, None], table[src], -1)
        refs = torch.zeros(pages + 1, dtype=torch.long, device="cuda")
        refs.index_add_(0, torch.where(table < 0, pages, table).flatten(), torch.ones_like(table).flatten())
        # the page that the next token goes to is copied by all of its holders but the first
        tail = table[rows_of[:, 0], (length // page).clamp(max=table.shape[1] - 1)]
        partial = length % page > 0
        first = torch.full((pages + 1,), c["b"], dtype=torch.long, device="cuda")
        first.scatter_reduce_(0, torch.where(partial, tail, pages), rows_of[:, 0], "amin")
        copies = partial & (first[tail] != rows_of[:, 0])
        # new pages: the free ones from the lowest on, sequence after sequence
        want = (length + st["new"] + page - 1) // page
        need = (want - have).clamp(min=0) + copies
        start = need.cumsum(0) - need
        free = refs[:pages] == 0
        order = torch.full((pages + 1,), -1, dtype=torch.long, device="cuda")
        order.scatter_(0, torch.where(free, free.long().cumsum(0) - 1, pages), torch.arange(pages, device="cuda"))
        fresh = order[(start[:, None] + copies[:, None] + slot - have[:, None]).clamp(0, pages - 1)]
        table = torch.where((slot >= have[:, None]) & (slot < want[:, None]), fresh, table)
        dst = order[start.clamp(max=pages - 1)]
        table = torch.where(copies[:, None] & (slot == (length // page)[:, None]), dst[:, None], table)
        who = copies.nonzero()[:, 0]
        a, z, fill = tail[who], dst[who], torch.arange(page, device="cuda")[None] < (length % page)[who, None]
        for x in (k, v):
            x[:, z] = torch.where(fill[None, :, :, None, None], x[:, a], x[:, z])
        refs = torch.zeros(pages + 1, dtype=torch.long, device="cuda")
        refs.index_add_(0, torch.where(table < 0, pages, table).flatten(), torch.ones_like(table).flatten())
        i32 = torch.int32
        return k, v, table.to(i32), length.to(i32), refs[:pages].to(i32)
    # compact: the used pages with the highest numbers move into the free ones with the lowest, in order
    refs = torch.zeros(pages + 1, dtype=torch.long, device="cuda")
    refs.index_add_(0, torch.where(table < 0, pages, table).flatten(), torch.ones_like(table).flatten())
    refs = refs[:pages]
    page_id = torch.arange(pages, device="cuda")
    n_used = (refs > 0).sum()
    movers = ((refs > 0) & (page_id >= n_used)).nonzero()[:, 0]
    holes = ((refs == 0) & (page_id < n_used)).nonzero()[:, 0]
    k[:, holes], v[:, holes] = k[:, movers], v[:, movers]
    goes = page_id.clone()
    goes[movers] = holes
    after = torch.zeros_like(refs)
    after[goes[refs > 0]] = refs[refs > 0]
    table = torch.where(table < 0, -1, goes[table.clamp(min=0)])
    return k, v, table.to(torch.int32), after.to(torch.int32)


def _plain_attention(c, st):
    b, m, hq, hkv, page = c["b"], c["nodes"], c["hq"], c["hkv"], c["page"]
    G = hq // hkv
    table, ctx = st["table"].long().clamp(min=0), st["length"].long()
    k = st["k"][0][table].flatten(1, 2).float().transpose(1, 2)     # [b][hkv][keys][D]
    v = st["v"][0][table].flatten(1, 2).float().transpose(1, 2)
    q = st["q"].float().unflatten(2, (hkv, G)).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [b][hkv][G * m][D]
    s = (q @ k.transpose(2, 3)).unflatten(2, (G, m)) * (1.0 / math.sqrt(D))           # [b][hkv][G][m][keys]
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    key = torch.arange(k.shape[2], device="cuda")
    node = key[None] - ctx[:, None]                                  # [b][keys]: number of the draft, below 0 in the context
    i = torch.arange(m, device="cuda")
    if c["tree"]:   # reach[i][j]: j is i or an ancestor of it; paths of up to 64 nodes by squaring
        par = st["parents"].long()
        reach = (i[None, :, None] == i) | (par[:, :, None] == i)
        for _ in range(6):
            reach = (reach.float() @ reach.float()) > 0
    else:
        reach = (i[:, None] >= i).expand(b, m, m)
    depth = reach.sum(-1) - 1
    sees = torch.gather(reach, 2, node.clamp(0, m - 1)[:, None].expand(b, m, -1))    # [b][m][keys]
    sees = torch.where(node[:, None] < 0, True, sees & (node[:, None] < m))
    if c["alibi"]:
        at = torch.where(node < 0, key[None], ctx[:, None] + torch.gather(depth, 1, node.clamp(0, m - 1)))
        far = (ctx[:, None, None] + depth[:, :, None] - at[:, None]).float()
        s = s - st["slopes"].view(hkv, G)[None, :, :, None, None] * far[:, None, None]
    s = torch.where(sees[:, None, None], s, float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (G, m)) / total
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3).to(st["out"].dtype)
    lse = (top + torch.log(total))[..., 0].permute(0, 3, 1, 2).flatten(2, 3)
    if st["q_len"] is not None:   # rows of sequences with fewer tokens stay as they were
        there = (i[None] < st["q_len"][:, None])[..., None]
        o, lse = torch.where(there[..., None], o, st["out"]), torch.where(there, lse, st["lse"])
    return o, lse


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(c, seed):
    """Attention by its definition in 64 bits: one sequence and head at a time over its own keys, every row's keys found
    by a walk up the tree.  The other operators move values and compute none."""
    if c["op"] != "attn" or 4 * D * c["hq"] * c["nodes"] * sum(_lengths(c)) > 4e12:
        return None
    st = prepare(c, seed)
    b, m, hq, G = c["b"], c["nodes"], c["hq"], c["hq"] // c["hkv"]
    out = torch.zeros(b, m, hq, D, device="cuda", dtype=torch.float64)
    lse = torch.zeros(b, m, hq, device="cuda", dtype=torch.float64)
    for i, (n, rows) in enumerate(zip(_lengths(c), _new_rows(c))):
        par = _parents(c, i) if c["tree"] else list(range(-1, m - 1))
        lines = [_ancestors(par, x) for x in range(rows)]
        pos = torch.tensor([n + len(x) - 1 for x in lines], device="cuda")
        key_pos = torch.cat([torch.arange(n, device="cuda"), pos])
        hidden = torch.ones(rows, rows, dtype=torch.bool)
        for x, line in enumerate(lines):
            hidden[x, line] = False
        hidden = torch.cat([torch.zeros(rows, n, dtype=torch.bool, device="cuda"), hidden.cuda()], 1)
        ids = st["table"][i, :-(-(n + rows) // c["page"])].long()
        for g in range(c["hkv"]):
            k, v = (st[x][0, ids, :, g].flatten(0, 1)[:n + rows].double() for x in "kv")
            for h in range(g * G, (g + 1) * G):
                s = torch.einsum("qd,kd->qk", st["q"][i, :rows, h].double(), k).div_(math.sqrt(D))
                if c["cap"]:
                    s = s.div_(c["cap"]).tanh_().mul_(c["cap"])
                if c["alibi"]:
                    s -= st["slopes"][h].double() * (pos[:, None] - key_pos[None])
                s.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(s, dim=1)
                lse[i, :rows, h] = z
                out[i, :rows, h] = s.sub_(z[:, None]).exp_() @ v
    return out, lse
