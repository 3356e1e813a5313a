"""Performance cases of the operators around the decode path: rotary position tables and rotations, attention
over a dense KV cache (prompts and single tokens, with capped scores, distance biases, document and prefix
masks) and attention of a batch whose sequences share one long prefix.

Every case runs in two forms on the same inputs: the plain form (elementary torch operations in fp32, angles in
fp64) and, with own = True, the library's operators through the binding.  Shapes are those of the package's
workloads (8 or 32 query heads over 2 or 8 KV heads of 128 channels; 4K, 32K and 131K contexts) and odd ones.
"""
import math

import torch

own = False

D = 128   # head dimension of every workload of the package
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the (cos, sin) table of a cache that stretches a 32K model to 131K tokens: built once per model load
        {"name": "table_131k_parts", "op": "table", "rows": 131200, "rot": 128, "base": 500000.0, "scaling": "parts",
         "factor": 4.0, "orig": 32768},
        # a half-rotated head's table for a 4K context: latency of a small call
        {"name": "table_4k_ntk", "op": "table", "rows": 4160, "rot": 64, "base": 10000.0, "scaling": "ntk",
         "factor": 2.0, "orig": 2048},
        # one decode step of 16 sequences at their own positions: queries and keys of one layer
        {"name": "rope_decode_b16", "op": "rope", "b": 16, "s": 1, "hq": 32, "hkv": 8, "rot": 128, "inter": False,
         "inverse": False, "type": "bf16", "rows": 33024, "factor": 1.0},
        # one layer of a 32K prompt
        {"name": "rope_prompt_32k", "op": "rope", "b": 1, "s": 32768, "hq": 32, "hkv": 8, "rot": 128, "inter": False,
         "inverse": False, "type": "bf16", "rows": 33024, "factor": 1.0},
        # interleaved pairs over half of the head, four odd-length prompts, with a magnitude factor; the inverse
        # rotation, which is also the gradient
        {"name": "rope_inter_4099_back", "op": "rope", "b": 4, "s": 4099, "hq": 32, "hkv": 8, "rot": 64, "inter": True,
         "inverse": True, "type": "fp16", "rows": 8192, "factor": 1.125},
        # one token against a short cache: latency
        {"name": "attn_token_1k", "op": "attn", "b": 1, "sq": 1, "skv": 1040, "hq": 8, "hkv": 2, "type": "bf16",
         "cap": 0.0, "alibi": False, "docs": 0, "prefix": False, "ragged": False},
        # a decode step of 16 sequences of different lengths up to 32K + 256: memory bound
        {"name": "attn_tokens_b16_33k", "op": "attn", "b": 16, "sq": 1, "skv": 33024, "hq": 32, "hkv": 8,
         "type": "bf16", "cap": 0.0, "alibi": False, "docs": 0, "prefix": False, "ragged": True},
        # one layer of a 32K prompt: tensor-core bound
        {"name": "attn_prompt_32k", "op": "attn", "b": 1, "sq": 32768, "skv": 32768, "hq": 32, "hkv": 8,
         "type": "bf16", "cap": 0.0, "alibi": False, "docs": 0, "prefix": False, "ragged": False},
        # documents packed into two odd rows, capped scores
        {"name": "attn_docs_cap_4099", "op": "attn", "b": 2, "sq": 4099, "skv": 4099, "hq": 32, "hkv": 8,
         "type": "fp16", "cap": 30.0, "alibi": False, "docs": 9, "prefix": False, "ragged": False},
        # a padded batch of prefix-mask prompts with distance biases, one KV head per query head
        {"name": "attn_prefix_alibi_1500", "op": "attn", "b": 8, "sq": 1500, "skv": 1500, "hq": 8, "hkv": 8,
         "type": "bf16", "cap": 0.0, "alibi": True, "docs": 0, "prefix": True, "ragged": True},
        # a decode step of 16 sequences that share a 32K prompt, each with up to 256 tokens of its own
        {"name": "shared_b16_32k", "op": "shared", "b": 16, "sq": 1, "pre": 32768, "skv": 256, "hq": 32, "hkv": 8,
         "type": "bf16", "cap": 0.0, "alibi": False},
        # two drafted tokens of three sequences behind a short system prompt: latency
        {"name": "shared_b3_1000_draft2", "op": "shared", "b": 3, "sq": 2, "pre": 1000, "skv": 37, "hq": 8, "hkv": 2,
         "type": "fp16", "cap": 30.0, "alibi": False},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(8, 2), (32, 8), (8, 8), (16, 8), (32, 4), (4, 1)])


def draw(rng):
    op = rng.choice(["table", "rope", "rope", "attn", "attn", "attn", "tokens", "tokens", "shared", "shared"])
    typ = rng.choice(["bf16", "bf16", "fp16"])
    hq, hkv = _heads(rng)
    if op == "table":
        return {"op": "table", "rows": _log_int(rng, 2, 131200), "rot": 2 * rng.randint(2, 64),
                "base": rng.choice([10000.0, 500000.0, 1000000.0]),
                "scaling": rng.choice(["none", "linear", "ntk", "parts"]), "factor": rng.uniform(1.0, 16.0),
                "orig": _log_int(rng, 1024, 32768)}
    if op == "rope":
        s = _log_int(rng, 1, 16384)
        return {"op": "rope", "b": rng.randint(1, max(1, min(64, 32768 // s))), "s": s, "hq": hq, "hkv": hkv,
                "rot": rng.choice([128, 128, 64, 2 * rng.randint(1, 64)]), "inter": rng.random() < 0.5,
                "inverse": rng.random() < 0.3, "type": rng.choice(["bf16", "fp16", "fp32"]),
                "rows": s + _log_int(rng, 1, 32768), "factor": rng.choice([1.0, rng.uniform(0.5, 1.5)])}
    cap, alibi = rng.choice([0.0, 0.0, 30.0, 50.0]), rng.random() < 0.3
    if op == "attn":     # prompts, whole or the last chunk of a longer context
        skv = _log_int(rng, 2, 8192)
        sq = skv if rng.random() < 0.7 else rng.randint(1, skv)
        b = rng.randint(1, max(1, min(8, 16384 // skv)))
        kind = rng.choice(["causal", "docs", "prefix"])
        return {"op": "attn", "b": b, "sq": sq, "skv": skv, "hq": hq, "hkv": hkv, "type": typ, "cap": cap,
                "alibi": alibi, "docs": rng.randint(2, 12) if kind == "docs" else 0, "prefix": kind == "prefix",
                "ragged": rng.random() < 0.4}
    if op == "tokens":   # decode steps, sometimes with a few drafted tokens
        skv = _log_int(rng, 1, 131072)
        b = rng.randint(1, max(1, min(64, 262144 // skv)))
        sq = min(skv, rng.choice([1, 1, 1, 2, 4]))
        return {"op": "attn", "b": b, "sq": sq, "skv": skv, "hq": hq, "hkv": hkv, "type": typ, "cap": cap,
                "alibi": alibi, "docs": 0, "prefix": False, "ragged": rng.random() < 0.7}
    return {"op": "shared", "b": _log_int(rng, 1, 64), "sq": rng.choice([1, 1, 1, 2, 3]),
            "pre": _log_int(rng, 1, 65536), "skv": _log_int(rng, 4, 2048), "hq": hq, "hkv": hkv, "type": typ,
            "cap": cap, "alibi": alibi}


# ------------------------------------------------------------------------------------------------ lengths and masks
# (functions of the case alone, so that the work of a case is known without its inputs)

def _kv_lens(c):
    """Valid keys of every sequence of an attention case."""
    b, skv, sq = c["b"], c["skv"], c["sq"]
    if not c["ragged"]:
        return [skv] * b
    lens = [skv - (i * skv * 3) // (4 * b) for i in range(b)]   # between a quarter of the cache and all of it
    if b > 2 and sq > 1:
        lens[1] = 1                                             # a prompt of one token in a padded batch
    return [max(1, n) for n in lens]


def _q_lens(c):
    """Queries of every sequence: the last ones of its keys (a padded batch of prompts has fewer than sq)."""
    return [min(c["sq"], n) for n in _kv_lens(c)] if c["ragged"] else [c["sq"]] * c["b"]


def _doc_starts(c):
    """First tokens of the documents packed into a row of skv tokens."""
    n, s = c["docs"], c["skv"]
    return sorted({int(s * (i / n) ** 1.5) for i in range(n)})


def _prefix_lens(c):
    return [(n * (i + 1)) // (2 * c["b"] + 1) for i, n in enumerate(_kv_lens(c))]


def _own_lens(c):
    """Keys of its own of every sequence behind a shared prefix, the newest tokens included."""
    return [max(min(c["sq"], c["skv"]), c["skv"] - (i * c["skv"]) // c["b"]) for i in range(c["b"])]


def _pairs(c):
    """Visible (query, key) pairs of one query head, summed over the batch."""
    if c["op"] == "shared":
        return sum(c["sq"] * (c["pre"] + n) - sum(range(min(c["sq"], n))) for n in _own_lens(c))
    total = 0
    for i, (n, m) in enumerate(zip(_kv_lens(c), _q_lens(c))):
        first = n - m
        if c["docs"]:
            starts = [x for x in _doc_starts(c) if x < n] + [n]
            for lo, hi in zip(starts, starts[1:]):
                f = max(first, lo)
                if f < hi:
                    total += (f + 1 - lo + hi - lo) * (hi - f) // 2
        elif c["prefix"]:
            p = _prefix_lens(c)[i]
            inside = max(0, min(n, p) - first)
            total += inside * p + sum(range(max(first, p) + 1, n + 1))
        else:
            total += (first + 1 + n) * m // 2
    return total


def work(c):
    if c["op"] == "table":   # every entry written once; an angle, its reduction, a cosine and a sine per pair
        n = c["rows"] * (c["rot"] // 2)
        return {"bytes": 8 * n, "flops": 40 * n}
    if c["op"] == "rope":    # heads read and written once, each position's table row read once
        tok, size = c["b"] * c["s"], TYPES[c["type"]].itemsize
        heads = c["hq"] + c["hkv"]
        return {"bytes": tok * (2 * heads * D * size + 4) + 4 * c["rot"] * min(tok, c["rows"]),
                "flops": tok * heads * (c["rot"] // 2) * 6}
    rows = c["b"] * c["sq"] * c["hq"]
    if c["op"] == "shared":
        kv = 2 * c["hkv"] * D * 2 * (c["pre"] + sum(_own_lens(c)))
    else:
        kv = 2 * c["hkv"] * D * 2 * sum(_kv_lens(c))
        rows = sum(_q_lens(c)) * c["hq"]
    return {"bytes": kv + rows * (2 * D * 2 + 4), "flops": 4 * D * c["hq"] * _pairs(c)}


# ------------------------------------------------------------------------------------------------ inputs

def _theta(c):
    """Angle per position of every pair, in fp64 (the plain form's and the library's formulas agree)."""
    rot = c["rot"]
    i = torch.arange(rot // 2, dtype=torch.float64)
    base = c["base"]
    if c["scaling"] == "ntk":
        base = base * c["factor"] ** (rot / (rot - 2))
    th = base ** (-2.0 * i / rot)
    if c["scaling"] == "linear":
        th = th / c["factor"]
    if c["scaling"] == "parts":   # fast pairs keep their angle, slow ones are stretched, a ramp between
        turns = c["orig"] * th / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        th = keep * th + (1.0 - keep) * th / c["factor"]
    return th


def _heads_of(gen, *shape, typ, gain, plant=None):
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
    if plant is not None:
        x = x + gain * plant
    return x.to(TYPES[typ])


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": c}
    if c["op"] == "table":
        # a table is a function of its sizes; another seed is another base
        st["base"] = c["base"] * (1.0 + (seed % 997) / 997.0)
        st["out"] = torch.empty(c["rows"], c["rot"] // 2, 2, device="cuda", dtype=torch.float32)
        if own:
            from recoverable_quantized_kv_gb300 import binding
            binding.load()
        return st
    if c["op"] == "rope":
        b, s, typ = c["b"], c["s"], TYPES[c["type"]]
        st["q"] = torch.randn(b, s, c["hq"], D, generator=gen, device="cuda").to(typ)
        st["k"] = torch.randn(b, s, c["hkv"], D, generator=gen, device="cuda").to(typ)
        # every sequence continues somewhere else in the context
        first = torch.randint(0, c["rows"] - s + 1, (b, 1), generator=gen, device="cuda")
        st["pos"] = (first + torch.arange(s, device="cuda")[None]).to(torch.int32)
        ang = torch.arange(c["rows"], dtype=torch.float64)[:, None] * _theta(dict(c, base=10000.0, scaling="none"))
        st["table"] = torch.stack([ang.cos(), ang.sin()], dim=-1).float().cuda()
        st["oq"], st["ok"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        if own:
            from recoverable_quantized_kv_gb300 import binding
            st["rope"] = binding.Rope(st["table"])
        return st
    b, sq, skv, hq, hkv, typ = c["b"], c["sq"], c["skv"], c["hq"], c["hkv"], c["type"]
    # some windows of keys lie along a direction that the queries share, as retrieved passages do
    u = torch.randn(D, generator=gen, device="cuda")
    u = u / u.norm()
    st["q"] = _heads_of(gen, b, sq, hq, D, typ=typ, gain=4.0, plant=u)

    def keys(*shape):
        n = shape[-3]
        hit = (torch.rand((n + 31) // 32, generator=gen, device="cuda") < 0.05).repeat_interleave(32)[:n]
        return _heads_of(gen, *shape, typ=typ, gain=4.0, plant=hit[:, None, None] * u)

    st["k"] = keys(b, skv, hkv, D)
    st["v"] = _heads_of(gen, b, skv, hkv, D, typ=typ, gain=0.0)
    st["slopes"] = None
    if c["alibi"]:   # one slope per head, a geometric sequence
        st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda")
    st["out"] = torch.zeros_like(st["q"])
    st["lse"] = torch.zeros(b, sq, hq, device="cuda", dtype=torch.float32)
    i32 = {"device": "cuda", "dtype": torch.int32}
    if c["op"] == "shared":
        st["kp"], st["vp"] = keys(c["pre"], hkv, D), _heads_of(gen, c["pre"], hkv, D, typ=typ, gain=0.0)
        st["kv_len"] = torch.tensor(_own_lens(c), **i32)
        if own:
            from recoverable_quantized_kv_gb300 import binding
            st["plan"] = binding.PrefixAttention(b, sq, c["pre"], skv, hq, hkv, dtype=TYPES[typ], softcap=c["cap"])
        return st
    st["kv_len"] = torch.tensor(_kv_lens(c), **i32) if c["ragged"] else None
    st["q_len"] = torch.tensor(_q_lens(c), **i32) if c["ragged"] else None
    st["prefix_len"] = torch.tensor(_prefix_lens(c), **i32) if c["prefix"] else None
    st["doc_ids"] = None
    if c["docs"]:
        starts = torch.tensor(_doc_starts(c))
        ids = (torch.arange(skv)[:, None] >= starts[None]).sum(1)
        st["doc_ids"] = ids[None].expand(b, skv).contiguous().to(**i32)
    if own:
        from recoverable_quantized_kv_gb300 import binding
        st["plan"] = binding.Attention(b, sq, skv, hq, hkv, dtype=TYPES[typ], softcap=c["cap"])
    return st


# ------------------------------------------------------------------------------------------------ the two forms

def run(st):
    c = st["case"]
    return _own(c, st) if own else _plain(c, st)


def _own(c, st):
    from recoverable_quantized_kv_gb300 import binding
    if c["op"] == "table":
        return binding.rope_table(c["rows"], rot_dim=c["rot"], base=st["base"], scaling=c["scaling"],
                                  factor=c["factor"], orig_len=c["orig"], low=1.0, high=32.0, out=st["out"])
    if c["op"] == "rope":
        return st["rope"].apply(st["q"], st["k"], positions=st["pos"], interleaved=c["inter"], inverse=c["inverse"],
                                factor=c["factor"], q_out=st["oq"], k_out=st["ok"])
    if c["op"] == "shared":
        return st["plan"].run(st["q"], st["kp"], st["vp"], st["k"], st["v"], out=st["out"], lse=st["lse"],
                              slopes=st["slopes"], kv_len=st["kv_len"])
    return st["plan"].run(st["q"], st["k"], st["v"], out=st["out"], lse=st["lse"], slopes=st["slopes"],
                          q_len=st["q_len"], kv_len=st["kv_len"], prefix_len=st["prefix_len"],
                          doc_ids=st["doc_ids"])


def _softmax_rows(s, v):
    """Rows of scores (masked ones at -inf) against values: the output and the log-sum-exp, empty rows as 0, -inf."""
    m = s.amax(dim=-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(dim=-1, keepdim=True)
    o = (p @ v) / torch.where(l > 0, l, torch.ones_like(l))
    return o, (m + torch.log(l))[..., 0]


def _plain(c, st):
    if c["op"] == "table":
        th = _theta(dict(c, base=st["base"])).cuda()
        ang = torch.arange(c["rows"], device="cuda", dtype=torch.float64)[:, None] * th
        return torch.stack([ang.cos(), ang.sin()], dim=-1).float()
    if c["op"] == "rope":
        cs = st["table"][st["pos"].long()]                      # [b][s][rot / 2][2]
        cos, sin = cs[:, :, None, :, 0], cs[:, :, None, :, 1]
        if c["inverse"]:
            sin = -sin
        return tuple(_rotate(x, cos, sin, c).to(x.dtype) for x in (st["q"], st["k"]))
    b, sq, skv, hq, hkv = c["b"], c["sq"], c["skv"], c["hq"], c["hkv"]
    G = hq // hkv
    scale, cap = 1.0 / math.sqrt(D), c["cap"]
    out, lse = torch.zeros_like(st["q"]), torch.zeros_like(st["lse"])
    if c["op"] == "shared":
        lens, q_lens, pre = _own_lens(c), [sq] * b, c["pre"]
    else:
        lens, q_lens, pre = _kv_lens(c), _q_lens(c), 0
    for i in range(b):
        n, m = lens[i], q_lens[i]
        for g in range(hkv):
            k, v = st["k"][i, :n, g].float(), st["v"][i, :n, g].float()
            if pre:
                k, v = torch.cat([st["kp"][:, g].float(), k]), torch.cat([st["vp"][:, g].float(), v])
            step = max(1, min(m, (1 << 28) // (G * (pre + n))))
            for r in range(0, m, step):
                e = min(m, r + step)
                pos = torch.arange(pre + n - m + r, pre + n - m + e, device="cuda")
                seen = pre + n if c.get("prefix") else int(pre + n - m + e)
                key = torch.arange(seen, device="cuda")
                ok = key[None] <= pos[:, None]
                if c.get("prefix"):
                    ok = ok | (key[None] < st["prefix_len"][i])
                if c.get("docs"):
                    ok = ok & (st["doc_ids"][i][pos][:, None] == st["doc_ids"][i][key][None])
                q = st["q"][i, r:e, g * G:(g + 1) * G].float().transpose(0, 1)         # [G][rows][D]
                s = (q @ k[:seen].T) * scale
                if cap:
                    s = cap * torch.tanh(s / cap)
                if c["alibi"]:
                    s = s - st["slopes"][g * G:(g + 1) * G, None, None] * (pos[:, None] - key[None]).abs().float()
                s = torch.where(ok[None], s, float("-inf"))
                o, ls = _softmax_rows(s, v[:seen])
                out[i, r:e, g * G:(g + 1) * G] = o.transpose(0, 1).to(out.dtype)
                lse[i, r:e, g * G:(g + 1) * G] = ls.transpose(0, 1)
    return out, lse


def _rotate(x, cos, sin, c):
    r, x = c["rot"], x.float()
    if c["inter"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y * c["factor"], x[..., r:]], dim=-1)


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(c, seed):
    """The definitions in 64 bits: angles and rotations as complex numbers, attention one head at a time over all
    its keys with a log-softmax.  None where the products would take too long in fp64."""
    if c["op"] in ("attn", "shared"):
        keys = c["skv"] + c.get("pre", 0)
        if 4 * D * c["hq"] * c["b"] * c["sq"] * keys > 5e12 or 8 * c["sq"] * keys > 8e9:
            return None
    st = prepare(c, seed)
    if c["op"] == "table":
        angles, rot = [], c["rot"]
        for i in range(rot // 2):   # pair by pair, through logarithms
            log_base = math.log(st["base"]) + (math.log(c["factor"]) * rot / (rot - 2) if c["scaling"] == "ntk" else 0.0)
            th = math.exp(-2 * i * log_base / rot)
            share = 1.0 if c["scaling"] == "linear" else 0.0   # of the stretched angle
            if c["scaling"] == "parts":
                turns = c["orig"] * th / math.tau
                share = 1.0 if turns <= 1.0 else 0.0 if turns >= 32.0 else (32.0 - turns) / 31.0
            angles.append(th * (share / c["factor"] + 1.0 - share))
        pos = torch.arange(c["rows"], device="cuda", dtype=torch.float64)
        z = torch.polar(torch.ones((), device="cuda", dtype=torch.float64),
                        torch.outer(pos, torch.tensor(angles, device="cuda", dtype=torch.float64)))
        return torch.view_as_real(z)
    if c["op"] == "rope":
        z = torch.view_as_complex(st["table"].double().contiguous())[st["pos"].long()][:, :, None]
        z = (z.conj() if c["inverse"] else z) * c["factor"]
        outs = []
        for x in (st["q"], st["k"]):
            y, r = x.double().clone(), c["rot"]
            first, second = (slice(0, r, 2), slice(1, r, 2)) if c["inter"] else (slice(0, r // 2), slice(r // 2, r))
            w = torch.complex(y[..., first], y[..., second]) * z
            y[..., first], y[..., second] = w.real, w.imag
            outs.append(y)
        return tuple(outs)
    b, sq, hq = c["b"], c["sq"], c["hq"]
    out = torch.zeros(b, sq, hq, D, device="cuda", dtype=torch.float64)
    lse = torch.zeros(b, sq, hq, device="cuda", dtype=torch.float64)
    pre = c.get("pre", 0)
    for i in range(b):
        n = (_own_lens(c) if pre else _kv_lens(c))[i]
        m = sq if pre else _q_lens(c)[i]
        i_q = torch.arange(m, device="cuda")[:, None] + (pre + n - m)   # positions of the queries
        i_k = torch.arange(pre + n, device="cuda")[None]
        hidden = i_k > i_q
        if c.get("prefix"):
            hidden = hidden & (i_k >= _prefix_lens(c)[i])
        if c.get("docs"):
            starts = torch.tensor(_doc_starts(c), device="cuda")
            doc = torch.bucketize(torch.arange(pre + n, device="cuda"), starts, right=True)
            hidden = hidden | (doc[i_q[:, 0]][:, None] != doc[None])
        for h in range(hq):
            g = h * c["hkv"] // hq
            k, v = st["k"][i, :n, g].double(), st["v"][i, :n, g].double()
            if pre:
                k, v = torch.cat([st["kp"][:, g].double(), k]), torch.cat([st["vp"][:, g].double(), v])
            s = torch.einsum("qd,kd->qk", st["q"][i, :m, h].double(), k).div_(math.sqrt(D))
            if c["cap"]:
                s = s.div_(c["cap"]).tanh_().mul_(c["cap"])
            if c["alibi"]:
                s -= st["slopes"][h].double() * (i_q - i_k).abs()
            s.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(s, dim=1)
            lse[i, :m, h] = z
            out[i, :m, h] = s.sub_(z[:, None]).exp_() @ v
    return out, lse
