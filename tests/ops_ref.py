"""Plain 64-bit forms of the rotary and attention operators, and error bounds derived from the roundings the kernels
document.  Test infrastructure: shares no code with the library."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative


def visible(pos, n, causal=True, prefix=0, ids=None):
    """[rows][n] mask: key j visible to the row at position p."""
    key = torch.arange(n, device=pos.device)[None]
    p = pos[:, None]
    ok = (key <= p) | (key < prefix) if causal else torch.ones(len(pos), n, dtype=torch.bool, device=pos.device)
    if ids is not None:
        run = torch.cat([torch.zeros(1, dtype=torch.long, device=pos.device), (ids[1:n] != ids[:max(n, 1) - 1]).long().cumsum(0)])
        ok = ok & (p >= 0) & (run[pos.clamp(0)][:, None] == run[None, :n])
    return ok


def attention_rows(q, k, v, ok, pos, key_pos, scale, cap=0.0, slope=None, half=HALF[torch.bfloat16]):
    """One head: q [m][d], k, v [n][d] (any float type), ok [m][n].  Returns out, lse (fp64) and bounds on the
    kernel's errors in both."""
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:   # no keys at all: one that nothing sees
        k, v, ok, key_pos = k.new_zeros(1, k.shape[1]), v.new_zeros(1, v.shape[1]), ok.new_zeros(len(ok), 1), pos.new_zeros(1)
    n = k.shape[0]
    kz = torch.where(ok.any(0)[:, None], k, torch.zeros_like(k))   # a key that no row sees does not count
    s = q @ kz.T * scale
    if cap:
        s = cap * torch.tanh(s / cap)
    if slope is not None:
        s = s - slope * (pos[:, None] - key_pos[None]).abs()
    s = torch.where(ok, s, torch.full_like(s, -math.inf))
    m = s.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m) & (m < 0), torch.zeros_like(m), m)
    e = torch.where(ok, torch.exp(s - m), torch.zeros_like(s))
    l = e.sum(1)
    p = e / torch.where(l > 0, l, torch.ones_like(l))[:, None]
    if torch.isfinite(v).all():
        out, amp = p @ v, p @ v.abs()
    else:   # a masked value must not count, even as 0 * NaN: row by row
        out = torch.stack([(p[i][ok[i]][:, None] * v[ok[i]]).sum(0) for i in range(len(p))])
        amp = p @ torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))   # of the outputs that stay finite
    lse = m[:, 0] + torch.log(l)
    # fp32 logits: products of 128 channels summed (128 roundings of the running sum), scaled, exponentiated by a unit
    # with relative error 2^-22; a cap adds a reciprocal and an exponential of relative error 2^-22 to 2 cap; a bias one
    # rounding of its size
    mag = (q.abs() @ kz.abs().T * scale).amax().item()
    delta = 130 * 2.0 ** -24 * mag + 2.0 ** -21 + (8 * cap * 2.0 ** -22 if cap else 0.0)
    if slope is not None:
        delta += 4 * 2.0 ** -24 * float(slope) * float((pos[:, None] - key_pos[None]).abs().max())
    rows = half * (amp + out.abs())              # p rounded for the product, out rounded once
    rows = rows + (2 * delta + (n + 64) * 2.0 ** -24) * amp   # logits; fp32 sums of n terms
    if half == HALF[torch.float16]:              # probabilities below 2^-14 step by 2^-24, the row's largest is at least 1
        rows = rows + n * 2.0 ** -25 * torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v)).amax()
        rows = rows + 2.0 ** -25                 # and so do small outputs
    lerr = delta + (n / 128 + 64) * 2.0 ** -24 + 2.0 ** -22 * (1 + torch.where(torch.isfinite(lse), lse.abs(), 0 * l))
    return out, lse, rows, lerr


def attention(q, k, v, q_len=None, kv_len=None, prefix_len=None, doc_ids=None, slopes=None, causal=True, cap=0.0,
              scale=0.0, k_prefix=None, v_prefix=None):
    """Whole operator; returns dicts (b, h) -> (out, lse, out bound, lse bound) over the written rows.  With a shared prefix
    the keys are the joined ones."""
    B, sq, hq, d = q.shape
    hkv, G = k.shape[2], q.shape[2] // k.shape[2]
    scale = scale or 1.0 / math.sqrt(d)
    res = {}
    for b in range(B):
        n = k.shape[1] if kv_len is None else int(kv_len[b])
        m = sq if q_len is None else int(q_len[b])
        if m == 0:
            continue
        pre = 0 if k_prefix is None else k_prefix.shape[0]
        pos = torch.arange(m, device=q.device) + (pre + n - m)
        ids = None if doc_ids is None else doc_ids[b]
        ok = visible(pos, pre + n, causal, 0 if prefix_len is None else min(int(prefix_len[b]), n), ids)
        key_pos = torch.arange(pre + n, device=q.device)
        for h in range(hq):
            g = h // G
            kk, vv = k[b, :n, g], v[b, :n, g]
            if pre:
                kk, vv = torch.cat([k_prefix[:, g], kk]), torch.cat([v_prefix[:, g], vv])
            res[b, h] = attention_rows(q[b, :m, h], kk, vv, ok, pos, key_pos, scale, cap,
                                       None if slopes is None else slopes[h].double(), HALF[q.dtype])
    return res


def compare(out, lse, res, tag=""):
    """Every written row within its bound; non-finite values in the same places."""
    for (b, h), (o, ls, eo, el) in res.items():
        m = o.shape[0]
        got, gl = out[b, :m, h].double(), lse[b, :m, h].double()
        fin = torch.isfinite(o)
        assert torch.equal(torch.isfinite(got), fin), f"{tag} non-finite outputs differ at sequence {b} head {h}"
        bad = ((got - o).abs() > eo) & fin
        assert not bad.any(), (f"{tag} b={b} h={h}: error {(got - o).abs()[bad].max().item():.3e} against bound "
                               f"{eo[bad].min().item():.3e}, {int(bad.sum())} of {bad.numel()} at rows "
                               f"{bad.any(1).nonzero().flatten()[:8].tolist()}")
        fin = torch.isfinite(ls)
        assert torch.equal(gl[~fin].nan_to_num(nan=7.0), ls[~fin].nan_to_num(nan=7.0)), f"{tag} lse infinities b={b} h={h}"
        bad = ((gl - ls).abs() > el) & fin
        assert not bad.any(), f"{tag} lse b={b} h={h}: {(gl - ls).abs()[bad].max().item():.3e} > {el[bad].min().item():.3e}"
