"""The attention operators' definition in 64 bits, row by row over the visible keys alone, with bounds that are finite
wherever the result is.  Test infrastructure: shares no code with the library.

What a row does not see enters neither its result nor its bound, so an infinity or NaN that some rows see leaves the other
rows of the head checked."""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step of the output, relative


def row(q, k, v, pos, key_pos, scale, cap, slope, dtype):
    """q [d], k, v [n][d] of the visible keys, fp64.  Returns out, lse and the bounds on both."""
    n = k.shape[0]
    if n == 0:
        zero = q.new_zeros(v.shape[1])
        return zero, q.new_tensor(-math.inf), zero, q.new_tensor(0.0)
    raw = (k @ q) * scale
    s = cap * torch.tanh(raw / cap) if cap else raw
    far = (pos - key_pos).abs().double()
    if slope is not None:
        s = s - slope * far
    m = s.max()
    e = torch.exp(s - m)
    l = e.sum()
    p = e / l
    out = (p[:, None] * v).sum(0)
    lse = m + torch.log(l)
    # fp32 logits: 128 products summed in a running sum and scaled (130 roundings of the sum of magnitudes, at most of what
    # is left of it behind a cap: tanh is a contraction), the exponential's unit 2^-22 and two roundings of the exponent's
    # argument, whose size the logits bound; behind a cap the tanh's own error, 2^-19 of the logit or, below a cap of 64,
    # 8 * 2^-22 of the cap; a bias: six roundings of its largest term and twenty of its sums along 32 keys
    mag = ((k.abs() @ q.abs()) * scale)
    mag = mag[torch.isfinite(mag)].max() if torch.isfinite(mag).any() else q.new_tensor(0.0)
    top = s[torch.isfinite(s)].abs().max() if torch.isfinite(s).any() else q.new_tensor(0.0)
    delta = 130 * 2.0 ** -24 * mag + 2.0 ** -21 + 4 * 2.0 ** -24 * top
    if cap:
        delta = delta + torch.minimum(8 * 2.0 ** -22 * q.new_tensor(min(cap, 64.0)) + 2.0 ** -19 * top, q.new_tensor(2 * cap))
    if slope is not None:
        delta = delta + 2.0 ** -24 * abs(slope) * (6 * far.max() + 20 * 32)
    fin = torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))
    amp = (torch.where(torch.isfinite(p), p, torch.zeros_like(p))[:, None] * fin).sum(0)
    grow = torch.expm1(2 * delta.clamp(max=40))   # of a probability whose logit and whose sum are off by delta
    eo = HALF[dtype] * (amp + out.abs()) + (grow + (n + 64) * 2.0 ** -24) * amp
    if dtype == torch.float16:
        # p is held with the row's largest at 2^0 to 2^15 over a scale that leaves it at least 2^7 above 1: small
        # probabilities step by 2^-24 * 2^-7 of the largest, and small outputs by 2^-24
        eo = eo + n * 2.0 ** -32 * fin.max() + 2.0 ** -25
    el = delta + (n / 128 + 64) * 2.0 ** -24 + 2.0 ** -22 * (1 + torch.where(torch.isfinite(lse), lse.abs(), 0 * l))
    return out, lse, eo, el


def check(out, lse, q, k, v, tag="", rows=None, q_len=None, kv_len=None, prefix_len=None, doc_ids=None, slopes=None,
          causal=True, cap=0.0, scale=0.0, k_prefix=None, v_prefix=None):
    """Every row (or the listed ones) of every sequence and head within its bound, non-finite values in the same places."""
    B, sq, hq, d = q.shape
    G = hq // k.shape[2]
    scale = scale or 1.0 / math.sqrt(d)
    pre = 0 if k_prefix is None else k_prefix.shape[0]
    for b in range(B):
        n = k.shape[1] if kv_len is None else int(kv_len[b])
        m = sq if q_len is None else int(q_len[b])
        run = None
        if doc_ids is not None:
            ids = doc_ids[b, :n]
            run = torch.cat([ids.new_zeros(min(n, 1)), (ids[1:] != ids[:-1]).to(ids.dtype)]).cumsum(0)
        for h in range(hq):
            kk, vv = k[b, :n, h // G], v[b, :n, h // G]
            if pre:
                kk, vv = torch.cat([k_prefix[:, h // G], kk]), torch.cat([v_prefix[:, h // G], vv])
            kk, vv = kk.double(), vv.double()
            keys = torch.arange(pre + n, device=q.device)
            for i in (range(m) if rows is None else rows):
                p = pre + n - m + i
                ok = torch.ones_like(keys, dtype=torch.bool)
                if causal:
                    ok = keys <= p
                    if prefix_len is not None:
                        ok = ok | (keys < min(int(prefix_len[b]), n))
                if run is not None:
                    ok = ok & (run == run[p] if p >= 0 else False)
                o, ls, eo, el = row(q[b, i, h].double(), kk[ok], vv[ok], p, keys[ok], scale, cap,
                                    None if slopes is None else float(slopes[h]), q.dtype)
                got, gl = out[b, i, h].double(), lse[b, i, h].double()
                where = f"{tag} sequence {b} head {h} row {i}"
                fin = torch.isfinite(o)
                assert torch.isfinite(eo[fin]).all() and (not torch.isfinite(ls) or torch.isfinite(el)), f"no bound: {where}"
                assert torch.equal(torch.isfinite(got), fin), f"non-finite outputs: {where}"
                err = (got - o).abs()[fin]
                assert (err <= eo[fin]).all(), f"{where}: error {err.max().item():.3e}, bound {eo[fin].max().item():.3e}"
                if torch.isfinite(ls):
                    assert (gl - ls).abs() <= el, f"{where}: lse {gl.item()} for {ls.item()}, bound {el.item():.3e}"
                else:
                    assert torch.equal(gl.nan_to_num(nan=7.0), ls.nan_to_num(nan=7.0)), f"{where}: lse {gl.item()} for {ls.item()}"
