"""Rotary tables and rotations against their formulas in 64 bits, and a run of them with the attention operators and the
cache, as a decoder uses them."""
import math

import numpy as np
import pytest
import torch

import ops_ref as R
from recoverable_quantized_kv_gb300 import binding, synth

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def theta(rot, base=10000.0, scaling="none", factor=1.0, orig=0, low=1.0, high=32.0):
    """Angles per position, pair by pair, from the documented formulas."""
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
        th = b ** (-2.0 * i / rot)
        if scaling == "linear":
            th /= factor
        if scaling == "parts":
            keep = min(1.0, max(0.0, (orig * th / (2 * math.pi) - low) / (high - low)))
            th = keep * th + (1 - keep) * th / factor
        out.append(th)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


@pytest.mark.parametrize("rows,first,kw", [
    (1, 0, dict(rot_dim=2)), (7, 3, dict(rot_dim=6, base=500000.0)), (33024, 0, dict(base=500000.0)),
    (1000, 131072, dict(base=1000000.0, scaling="linear", factor=8.0)),
    (500, 2 ** 31 - 500, dict()), (4160, 0, dict(rot_dim=64, scaling="ntk", factor=2.5)),
    (9999, 1, dict(scaling="parts", factor=4.0, orig_len=8192)),
    (4097, 0, dict(rot_dim=512, scaling="parts", factor=16.0, orig_len=4096, low=1.0, high=4.0)),
    (300, 0, dict(scaling="linear", factor=0.125)), (64, 5, dict(rot_dim=4, base=0.5))])
def test_table(lib, rows, first, kw):
    """Every entry within 2^-23 of the exact angle's; fp64 angles of position 2^31 are exact to 2^-22 of a radian, which is
    what their bound adds there."""
    t = binding.rope_table(rows, first=first, **kw)
    rot = kw.get("rot_dim", 128)
    a = {"orig" if k == "orig_len" else k: v for k, v in kw.items() if k != "rot_dim"}
    th = theta(rot, **a)
    assert torch.allclose(torch.tensor(binding.rope_angles(**kw), dtype=torch.float64, device="cuda"), th, rtol=1e-14)
    pos = torch.arange(first, first + rows, dtype=torch.float64, device="cuda")
    ang = pos[:, None] * th
    want = torch.stack([ang.cos(), ang.sin()], -1)
    # the angle per position is held to 2^-53 relative on both sides, and the product rounds once in fp64
    tol = 2.0 ** -23 + 3 * 2.0 ** -53 * ang.abs().max().item()
    assert (t.double() - want).abs().max().item() <= tol


def test_table_is_the_one_the_cache_takes(lib):
    want = torch.from_numpy(synth.rope_table(5000, 500000.0)).cuda()
    assert (binding.rope_table(5000, base=500000.0) - want).abs().max().item() <= 2.0 ** -23 + 2.0 ** -24


def apply_ref(x, table, pos, inter, inverse, factor):
    cs = table.double()[pos.long()][:, :, None]
    z = torch.complex(cs[..., 0], -cs[..., 1] if inverse else cs[..., 1]) * factor
    r = 2 * table.shape[1]
    y = x.double().clone()
    a, b = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, r // 2), slice(r // 2, r))
    w = torch.complex(y[..., a], y[..., b]) * z
    y[..., a], y[..., b] = w.real, w.imag
    # products of two fp32 numbers (one of them a factored cosine), each rounded, summed with a rounding
    mag = torch.zeros_like(y)
    m = (x.double()[..., a].abs() + x.double()[..., b].abs()) * abs(factor)
    mag[..., a], mag[..., b] = m, m
    return y, R.HALF[x.dtype] * y.abs() + 3 * 2.0 ** -24 * mag + (2.0 ** -25 if x.dtype == FP else 0.0)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot,d", [(128, 128), (64, 128), (2, 2), (6, 10), (128, 130), (96, 128), (512, 1024), (34, 128)])
def test_apply(lib, dtype, inter, rot, d):
    B, s, hq, hk = 3, 5, 6, 2
    g = torch.Generator(device="cuda").manual_seed(rot + d)
    q = torch.randn(B, s, hq, d, generator=g, device="cuda").to(dtype)
    k = torch.randn(B, s, hk, d, generator=g, device="cuda").to(dtype)
    rope = binding.Rope(binding.rope_table(300, rot_dim=rot))
    pos = torch.randint(0, 300, (B, s), generator=g, device="cuda", dtype=torch.int32)
    pos[0, 0], pos[1, 1] = 299, 0
    for inverse, factor in ((False, 1.0), (True, 1.25)):
        qo, ko = rope.apply(q, k, positions=pos, interleaved=inter, inverse=inverse, factor=factor)
        for got, x in ((qo, q), (ko, k)):
            want, tol = apply_ref(x, rope.table, pos, inter, inverse, factor)
            assert torch.all((got.double() - want).abs() <= tol)
            assert torch.equal(got[..., rot:], x[..., rot:])
    rope.check()


@pytest.mark.parametrize("tokens", [1, 2, 4099])
def test_default_positions_and_lengths(lib, tokens):
    rope = binding.Rope(binding.rope_table(8192))
    q = torch.randn(1, tokens, 4, 128, device="cuda").to(BF)
    qo, ko = rope.apply(q, pos0=37)
    assert ko is None
    pos = (37 + torch.arange(tokens, device="cuda"))[None]
    want, tol = apply_ref(q, rope.table, pos, False, False, 1.0)
    assert torch.all((qo.double() - want).abs() <= tol)


def test_strides_and_in_place(lib):
    """Inside a fused projection, head-major, broadcast inputs, an odd offset that rules out wide loads; in place."""
    B, s, hq, hk, d = 2, 33, 4, 2, 128
    rope = binding.Rope(binding.rope_table(s))
    fused = torch.randn(B, s, hq + 2 * hk, d, device="cuda").to(BF)
    before = fused.clone()
    q, k = fused[:, :, :hq], fused[:, :, hq:hq + hk]
    want = rope.apply(q.contiguous(), k.contiguous())
    hm = torch.empty(B, hq, s, d, dtype=BF, device="cuda").transpose(1, 2)
    got = rope.apply(q, k, q_out=hm)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rope.apply(q, k, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(fused[:, :, hq + hk:], before[:, :, hq + hk:])
    flat = torch.randn(1 + B * s * hq * d, device="cuda").to(BF)
    odd = flat[1:].view(B, s, hq, d)
    w, tol = apply_ref(odd, rope.table, torch.arange(s, device="cuda")[None].expand(B, s), False, False, 1.0)
    assert torch.all((rope.apply(odd)[0].double() - w).abs() <= tol)
    one = torch.randn(1, 1, 1, d, device="cuda").to(BF).expand(B, s, hq, d)
    w, tol = apply_ref(one, rope.table, torch.arange(s, device="cuda")[None].expand(B, s), False, False, 1.0)
    assert torch.all((rope.apply(one)[0].double() - w).abs() <= tol)


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot,d,tokens,hq", [(74, 128, 3, 40), (10, 1024, 2, 9), (2, 8, 5, 3), (126, 128, 400, 7)])
def test_pairs_off_the_vectors(lib, dtype, inter, rot, d, tokens, hq):
    """Heads on 16 bytes whose pairs are not: head-major in, in place, a position outside the table, a head count that is
    no multiple of a block's."""
    rope = binding.Rope(binding.rope_table(500, rot_dim=rot))
    g = torch.Generator(device="cuda").manual_seed(rot + tokens)
    q = torch.randn(2, hq, tokens, d, generator=g, device="cuda").to(dtype).transpose(1, 2)
    k = torch.randn(2, tokens, 2, d, generator=g, device="cuda").to(dtype)
    pos = torch.randint(0, 500, (2, tokens), generator=g, device="cuda", dtype=torch.int32)
    wants = [apply_ref(x, rope.table, pos, inter, False, 0.75) for x in (q, k)]
    outs = rope.apply(q, k, positions=pos, interleaved=inter, factor=0.75)
    for got, x, (want, tol) in zip(outs, (q, k), wants):
        assert torch.all((got.double() - want).abs() <= tol) and torch.equal(got[..., rot:], x[..., rot:])
    pos[1, 1] = 500
    before = q.clone(), k.clone()
    rope.apply(q, k, positions=pos, interleaved=inter, factor=0.75, q_out=q, k_out=k)
    for x, b, got in zip((q, k), before, outs):
        assert torch.equal(x[1, 1], b[1, 1]) and torch.equal(x[0], got[0]) and torch.equal(x[1, 2:], got[1, 2:])
    with pytest.raises(binding.QEvictError):
        rope.check()


def test_positions_outside_the_table(lib):
    """The token is not written and the status word says so; the other tokens are."""
    rope = binding.Rope(binding.rope_table(16))
    q = torch.randn(1, 4, 2, 128, device="cuda").to(BF)
    out = torch.full_like(q, 9.0)
    rope.apply(q, positions=torch.tensor([[3, 16, -1, 15]], dtype=torch.int32, device="cuda"), q_out=out)
    with pytest.raises(binding.QEvictError) as e:
        rope.check()
    assert e.value.status == binding.EDEVICE
    rope.check()
    assert torch.all(out[0, 1:3] == 9.0)
    want, tol = apply_ref(q, rope.table, torch.tensor([[3, 0, 0, 15]], device="cuda"), False, False, 1.0)
    ok = (out.double() - want).abs() <= tol
    assert ok[0, 0].all() and ok[0, 3].all()


@pytest.mark.parametrize("inter", [False, True])
def test_gradient(lib, inter):
    """The inverse call is the gradient: against the transposed rotation by autograd in fp64 and against central
    differences of the kernel itself (linear, so a step of 1 is exact up to fp32 roundings of values below 8)."""
    s, rot, d, f = 5, 12, 16, 1.25
    rope = binding.Rope(binding.rope_table(64, rot_dim=rot))
    x = torch.randn(1, s, 1, d, device="cuda", dtype=F32)
    w = torch.randn(1, s, 1, d, device="cuda", dtype=F32)
    grad = rope.apply(w, pos0=9, interleaved=inter, inverse=True, factor=f)[0]
    grad = torch.cat([grad[..., :rot], w[..., rot:]], -1)
    xd = x.double().requires_grad_()
    cs = rope.table.double()[9:9 + s][None, :, None]
    a, b = (xd[..., 0:rot:2], xd[..., 1:rot:2]) if inter else (xd[..., :rot // 2], xd[..., rot // 2:rot])
    y1, y2 = f * (a * cs[..., 0] - b * cs[..., 1]), f * (b * cs[..., 0] + a * cs[..., 1])
    y = torch.stack([y1, y2], -1).flatten(-2) if inter else torch.cat([y1, y2], -1)
    (torch.cat([y, xd[..., rot:]], -1) * w.double()).sum().backward()
    assert (grad.double() - xd.grad).abs().max().item() <= 3 * 2.0 ** -24 * 2 * f * w.abs().max().item() + 2.0 ** -23
    for c in (0, 3, rot - 1, d - 1):
        e = torch.zeros_like(x)
        e[..., c] = 1.0
        up = rope.apply(x + e, pos0=9, interleaved=inter, factor=f)[0]
        dn = rope.apply(x - e, pos0=9, interleaved=inter, factor=f)[0]
        num = (((up - dn) / 2).double() * w.double()).sum(-1)
        # each of 16 outputs carries three fp32 roundings of values below 8, weighted by |w|
        tol = 3 * 2.0 ** -24 * 8 * w.abs().sum(-1).max().item() + 2.0 ** -22
        assert (num - grad[..., c].double()).abs().max().item() <= tol


def test_capture(lib):
    rope = binding.Rope(binding.rope_table(100))
    q, pos = torch.randn(2, 1, 4, 128, device="cuda").to(BF), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    rope.apply(q, positions=pos, q_out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.apply(q, positions=pos, q_out=out)
    for p in (5, 99):
        pos.fill_(p)
        g.replay()
        want, tol = apply_ref(q, rope.table, pos, False, False, 1.0)
        assert torch.all((out.double() - want).abs() <= tol)


def test_a_decoder_layer_run(lib):
    """Table, rotation, prompt attention, cache prefill, then decode steps of rotated tokens: a cache whose budget keeps
    every window Full gives what attention over the dense cache gives; the prompt shared by the batch too."""
    wl = synth.workload("tiny_4k", batch=2, prompt_len=700, steps=8, budget_num=400, n_plant=0)
    cfg = binding.make_config(wl, rope=1)
    B, P, steps = wl.batch, wl.prompt_len, 7
    table = binding.rope_table(wl.max_len, base=500000.0)
    rope, cache = binding.Rope(table), binding.Cache(cfg)
    cache.set_rope_table(table)
    g = torch.Generator(device="cuda").manual_seed(3)
    mk = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)   # noqa: E731
    k, v = (mk(1, wl.max_len, wl.h_kv, 128).expand(B, -1, -1, -1).contiguous() for _ in range(2))
    for b in range(1, B):   # the prompt is common, the tokens behind it are not
        k[b, P:], v[b, P:] = mk(wl.max_len - P, wl.h_kv, 128), mk(wl.max_len - P, wl.h_kv, 128)
    q = mk(B, wl.max_len, wl.h_q, 128)
    q[:] = q[:1]
    q, k = rope.apply(q, k, q_out=q, k_out=k)
    prompt = binding.Attention(B, P, P, wl.h_q, wl.h_kv)
    po, pl = prompt.run(q[:, :P], k[:, :P], v[:, :P])
    R.compare(po, pl, R.attention(q[:, :P], k[:, :P], v[:, :P]), "prompt")
    qp, kp, vp = (x[:, :P].contiguous() for x in (q, k, v))
    cache.prefill_route(0, kp, vp, q_prompt=qp)
    dense = binding.Attention(B, 1, wl.max_len, wl.h_q, wl.h_kv)
    shared = binding.PrefixAttention(B, 1, P, wl.max_len - P, wl.h_q, wl.h_kv)
    for t in range(P, P + steps):
        qt, kt, vt = (x[:, t].contiguous() for x in (q, k, v))
        out = torch.empty_like(qt)
        cache.decode_step(0, qt, kt, vt, out)
        n = torch.full((B,), t + 1, dtype=torch.int32, device="cuda")
        ref = R.attention(q[:, t:t + 1], k, v, kv_len=[t + 1] * B)
        do, dl = dense.run(q[:, t:t + 1], k, v, kv_len=n)
        so, sl = shared.run(q[:, t:t + 1], k[0, :P], v[0, :P], k[:, P:], v[:, P:], kv_len=n - P)
        R.compare(do, dl, ref, "dense")
        R.compare(so, sl, ref, "shared")
        # the cache's own tolerance is 2e-2 (bf16 outputs and probabilities)
        assert (out.float() - do[:, 0].float()).abs().max().item() <= 2e-2
    cache.check()
    prompt.check()
    dense.check()
    shared.check()
    rope.check()
