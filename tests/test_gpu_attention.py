"""Attention over a dense KV cache and behind a shared prefix, against the definition in 64 bits."""
import math

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


def run_case(B, sq, skv, hq, hkv, dtype=BF, causal=True, cap=0.0, scale=0.0, slopes=False, seed=1, gain=1.5, **arrays):
    q, k, v = rnd(B, sq, hq, 128, seed=seed, dtype=dtype, gain=gain), rnd(B, skv, hkv, 128, seed=seed + 1, dtype=dtype), \
        rnd(B, skv, hkv, 128, seed=seed + 2, dtype=dtype)
    sl = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda") if slopes else None
    plan = binding.Attention(B, sq, skv, hq, hkv, dtype=dtype, causal=causal, softcap=cap, scale=scale)
    out, lse = plan.run(q, k, v, slopes=sl, **arrays)
    plan.check()
    R.compare(out, lse, R.attention(q, k, v, slopes=sl, causal=causal, cap=cap, scale=scale, **arrays))
    return plan, (q, k, v, out, lse)


@pytest.mark.parametrize("sq,skv", [(1, 1), (1, 2), (1, 127), (1, 128), (1, 129), (2, 300), (1, 5000), (5, 517), (64, 64),
                                    (127, 127), (128, 128), (129, 129), (256, 256), (300, 300), (1000, 1000),
                                    (33, 4100), (700, 1500)])
@pytest.mark.parametrize("hq,hkv,dtype", [(8, 2, BF), (4, 4, FP)])
def test_causal_lengths(lib, sq, skv, hq, hkv, dtype):
    run_case(2, sq, skv, hq, hkv, dtype)


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8, 16, 33, 128])
@pytest.mark.parametrize("sq", [1, 7, 200])
def test_head_groups(lib, G, sq):
    run_case(1, sq, 260, 2 * G, 2, BF)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cap,slopes,causal,scale", [(30.0, False, True, 0.0), (0.0, True, True, 0.0), (5.0, True, True, 0.25),
                                                     (0.0, False, False, 0.0), (2.0, False, False, 1.0),
                                                     (0.0, True, False, 0.03)])
@pytest.mark.parametrize("sq,skv", [(1, 700), (400, 400), (50, 1300)])
def test_scores_capped_biased_scaled(lib, dtype, cap, slopes, causal, scale, sq, skv):
    run_case(2, sq, skv, 8, 2, dtype, causal=causal, cap=cap, slopes=slopes, scale=scale)


@pytest.mark.parametrize("cap", [100.0, 24.0, 14.0, 8.0, 2.0])
@pytest.mark.parametrize("sq,skv", [(300, 300), (1, 700)])
def test_caps_from_barely_felt_to_tight(lib, cap, sq, skv):
    """Logits of deviation 1.5, about 5 at most among the 1024 of a warp's step: the caps put them on either side of 0.25 and 0.6
    of the cap, or on both within one row."""
    run_case(1, sq, skv, 4, 2, cap=cap, seed=13)


def test_capped_scores_far_beyond_the_cap(lib):
    """Logits of hundreds against a cap of 3: tanh at its ends, both signs."""
    run_case(1, 130, 260, 4, 2, BF, cap=3.0, gain=300.0)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_large_logits_move_the_running_max(lib, dtype):
    """Peaked rows whose maxima grow along the keys in both directions: the running max is moved and the sums rescaled."""
    B, s, hq, hkv = 1, 900, 4, 1
    q, k, v = rnd(B, s, hq, 128, dtype=dtype), rnd(B, s, hkv, 128, seed=2, dtype=dtype), rnd(B, s, hkv, 128, seed=3, dtype=dtype)
    ramp = torch.linspace(0, 6, s, device="cuda")[None, :, None, None]
    for kk in (k * ramp, k * ramp.flip(1)):
        kk = kk.to(dtype)
        plan = binding.Attention(B, s, s, hq, hkv, dtype=dtype)
        out, lse = plan.run(q * 2, kk, v)
        plan.check()
        R.compare(out, lse, R.attention(q * 2, kk, v))


@pytest.mark.parametrize("sq", [1, 3, 260])
def test_ragged_lengths_and_rows_behind_them(lib, sq):
    """A padded batch: rows behind a sequence's queries keep what they held; a sequence without keys gives 0 and -inf;
    one without queries writes nothing."""
    B, skv = 6, 500
    kv = [500, 1, 257, 0, 128, 300]
    ql = [min(sq, n) if n else sq for n in kv]
    ql[4] = 0
    q, k, v = rnd(B, sq, 8, 128), rnd(B, skv, 2, 128, seed=2), rnd(B, skv, 2, 128, seed=3)
    plan = binding.Attention(B, sq, skv, 8, 2)
    out, lse = torch.full_like(q, 7.0), torch.full((B, sq, 8), 7.0, device="cuda")
    plan.run(q, k, v, out=out, lse=lse, q_len=i32(ql), kv_len=i32(kv))
    plan.check()
    R.compare(out, lse, R.attention(q, k, v, q_len=ql, kv_len=kv))
    for b in range(B):
        assert torch.all(out[b, ql[b]:] == 7.0) and torch.all(lse[b, ql[b]:] == 7.0)
    assert torch.all(out[3, :ql[3]] == 0) and torch.all(lse[3, :ql[3]] == -math.inf)


def test_many_sequences_of_all_lengths(lib):
    """More sequences than a warp has lanes, empty and short ones between long ones, so that shares of the key tiles begin and
    end anywhere; and more units of work than SMs."""
    g = torch.Generator().manual_seed(5)
    B, skv = 70, 1500
    kv = [int(x) for x in torch.randint(0, skv + 1, (B,), generator=g)]
    kv[0], kv[33], kv[34], kv[69] = 0, 0, 1, skv
    q, k, v = rnd(B, 1, 8, 128), rnd(B, skv, 2, 128, seed=2), rnd(B, skv, 2, 128, seed=3)
    plan = binding.Attention(B, 1, skv, 8, 2)
    out, lse = plan.run(q, k, v, kv_len=i32(kv))
    plan.check()
    R.compare(out, lse, R.attention(q, k, v, kv_len=kv))
    assert torch.all(out[0] == 0) and torch.all(lse[33] == -math.inf)
    run_case(40, 70, 200, 16, 8, FP)          # 320 units of one pair of row tiles each


@pytest.mark.parametrize("sq,skv", [(200, 9000), (33, 20000), (300, 40000)])
def test_last_chunk_of_a_long_context(lib, sq, skv):
    """Few rows against many keys: pairs of row tiles, and an odd last one, cut into parts."""
    run_case(1, sq, skv, 8, 2, BF)
    run_case(2, sq, skv, 4, 4, FP, kv_len=i32([skv - 77, sq]), cap=15.0)


def test_more_queries_than_keys(lib):
    """Causal queries before position 0 see nothing."""
    B, sq, skv = 2, 70, 90
    q, k, v = rnd(B, sq, 4, 128), rnd(B, skv, 2, 128, seed=2), rnd(B, skv, 2, 128, seed=3)
    plan = binding.Attention(B, sq, skv, 4, 2)
    out, lse = plan.run(q, k, v, kv_len=i32([20, 90]))
    plan.check()
    R.compare(out, lse, R.attention(q, k, v, kv_len=[20, 90]))
    assert torch.all(out[0, :50] == 0) and torch.all(lse[0, :50] == -math.inf)


@pytest.mark.parametrize("sq,skv", [(600, 600), (200, 600), (1, 600)])
@pytest.mark.parametrize("causal", [True, False])
def test_documents(lib, sq, skv, causal):
    """Runs of equal ids, ids that return later in another document, documents of one token, ends inside a tile."""
    ids = []
    for n, x in [(1, 5), (130, 2), (1, 2 ** 31 - 1), (127, 2), (128, -7), (3, 0), (210, 9)]:
        ids += [x] * n
    ids = torch.tensor([ids, [4] * 600], dtype=torch.int32, device="cuda")
    run_case(2, sq, skv, 8, 2, BF, causal=causal, doc_ids=ids)


@pytest.mark.parametrize("n", [1, 1000, 1024, 1025, 5000])
def test_documents_in_long_rows(lib, n):
    """The scan over document ids at sizes around its 1024 pieces: alternating single tokens, then one run."""
    ids = torch.arange(n, device="cuda") % 2
    ids[n // 2:] = 3
    run_case(1, min(n, 40), n, 4, 4, BF, doc_ids=ids[None].to(torch.int32))


@pytest.mark.parametrize("prefix", [[0, 0], [1, 64], [300, 300], [128, 299], [77, 1000]])
def test_prefix_mask(lib, prefix):
    run_case(2, 300, 300, 8, 2, FP, prefix_len=i32(prefix))


def test_prefix_mask_with_documents_lengths_bias_and_cap(lib):
    ids = (torch.arange(400, device="cuda") // 150)[None].expand(3, 400).contiguous().to(torch.int32)
    run_case(3, 400, 400, 4, 2, BF, cap=20.0, slopes=True, doc_ids=ids, prefix_len=i32([200, 10, 390]), kv_len=i32([400, 333, 2]),
             q_len=i32([400, 100, 2]))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_masked_places_may_hold_anything(lib, dtype, bad):
    """Keys and values behind a sequence's end, of later tokens and of other documents hold infinities or NaN: rows that do
    not see them are unchanged to the bound, rows that see them get what the definition gives."""
    B, s = 2, 300
    q, k, v = rnd(B, s, 4, 128, dtype=dtype), rnd(B, s, 2, 128, seed=2, dtype=dtype), rnd(B, s, 2, 128, seed=3, dtype=dtype)
    k[0, 250:] = bad
    v[0, 250:] = bad
    plan = binding.Attention(B, s, s, 4, 2, dtype=dtype)
    kv, ql = [250, 300], [250, 300]
    out, lse = plan.run(q, k, v, kv_len=i32(kv), q_len=i32(ql))
    R.compare(out, lse, R.attention(q, k, v, kv_len=kv, q_len=ql), "behind the end")
    v[1, 200, 0, 5] = bad         # visible to rows from 200 on, in one KV head and channel
    out, lse = plan.run(q, k, v, kv_len=i32(kv), q_len=i32(ql))
    assert torch.isfinite(out[1, :200].float()).all()
    R.compare(out, lse, R.attention(q, k, v, kv_len=kv, q_len=ql), "a later value")
    ids = torch.zeros(B, s, dtype=torch.int32, device="cuda")
    ids[:, 140:] = 1
    v[1, 100] = bad
    out, lse = plan.run(q, k, v, kv_len=i32(kv), q_len=i32(ql), doc_ids=ids)
    R.compare(out, lse, R.attention(q, k, v, kv_len=kv, q_len=ql, doc_ids=ids), "another document")
    one = binding.Attention(B, 1, s, 4, 2, dtype=dtype)   # single tokens, the values visible or behind the end
    out, lse = one.run(q[:, :1], k, v, kv_len=i32([250, 150]))
    R.compare(out, lse, R.attention(q[:, :1], k, v, kv_len=[250, 150]), "single tokens")
    plan.check()
    one.check()


def test_a_later_nan_in_a_long_prompt(lib):
    """The rows that share a tile with a later value that is not finite are worked out again over all their keys."""
    s, at = 8192, 7000
    q, k, v = rnd(1, s, 4, 128), rnd(1, s, 2, 128, seed=2), rnd(1, s, 2, 128, seed=3)
    clean = binding.Attention(1, s, s, 4, 2)
    want, want_lse = clean.run(q, k, v)
    v[0, at, 1, 17] = math.nan
    plan = binding.Attention(1, s, s, 4, 2)
    out, lse = plan.run(q, k, v)
    plan.check()
    assert torch.equal(out[:, :, :2], want[:, :, :2])            # the other KV head
    assert torch.isnan(out[0, at:, 2:, 17]).all()
    keep = [c for c in range(128) if c != 17]
    rows = torch.arange(at - 130, at + 130, device="cuda")
    for h in (2, 3):
        ok = R.visible(rows, s)
        vv = v[0, :, 1].clone()
        vv[at, 17] = 0
        o, ls, eo, el = R.attention_rows(q[0, rows, h], k[0, :, 1], vv, ok, rows, torch.arange(s, device="cuda"), 1 / math.sqrt(128))
        assert torch.all((out[0, rows, h].double() - o).abs()[:, keep] <= eo[:, keep])
        assert torch.all((out[0, rows, h].double() - o).abs()[:130] <= eo[:130])
        assert torch.all((lse[0, rows, h].double() - ls).abs() <= el)


@pytest.mark.parametrize("slopes", [False, True])
def test_masked_places_with_capped_scores(lib, slopes):
    """Keys behind the end and of later tokens hold NaN next to visible ones; infinite scores reach the cap."""
    B, s = 2, 260
    q, k, v = rnd(B, s, 4, 128), rnd(B, s, 2, 128, seed=2), rnd(B, s, 2, 128, seed=3)
    k[0, 131:], v[0, 131:] = math.nan, math.inf
    k[1, 201], v[1, 201] = math.nan, -math.inf
    q[1, 7] = 1e38       # products overflow to infinities of both signs
    sl = torch.tensor([0.5, 0.25, 0.125, 0.0], device="cuda") if slopes else None
    plan = binding.Attention(B, s, s, 4, 2, softcap=25.0)
    out, lse = plan.run(q, k, v, slopes=sl, kv_len=i32([131, 201]), q_len=i32([131, 201]))
    plan.check()
    assert torch.isfinite(out[0, :131].float()).all() and torch.isfinite(lse[1, :201]).all()
    qq = q.clone()
    qq[1, 7] = 0
    ref = R.attention(qq, k, v, slopes=sl, cap=25.0, kv_len=[131, 201], q_len=[131, 201])
    keep = [i for i in range(201) if i != 7]
    for (b, h), (o, ls, eo, el) in ref.items():
        rows = torch.tensor(keep if b else range(131), device="cuda")
        assert torch.all((out[b, rows, h].double() - o[rows]).abs() <= eo[rows])
        assert torch.all((lse[b, rows, h].double() - ls[rows]).abs() <= el[rows] if torch.is_tensor(el) else el)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_visible_values_of_vanishing_weight_propagate(lib, bad):
    """A bias of 1 a key leaves keys 3000 back a weight of 0 in fp32; 0 times an infinity is NaN, in whichever part it lies."""
    for sq, skv, at in ((1, 6000, 10), (1, 6000, 2990), (3, 700, 5)):
        q, k, v = rnd(2, sq, 4, 128), rnd(2, skv, 2, 128, seed=2), rnd(2, skv, 2, 128, seed=3)
        v[1, at, 0, 9] = bad
        sl = torch.ones(4, device="cuda")
        plan = binding.Attention(2, sq, skv, 4, 2)
        out, lse = plan.run(q, k, v, slopes=sl)
        plan.check()
        assert not torch.isfinite(out[1, :, :2, 9]).any()
        R.compare(out, lse, R.attention(q, k, v, slopes=sl))


@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_visible_nan_scores_propagate(lib, cap):
    q, k, v = rnd(1, 4, 2, 128), rnd(1, 300, 1, 128, seed=2), rnd(1, 300, 1, 128, seed=3)
    q[0, 1, 0] = math.nan
    plan = binding.Attention(1, 4, 300, 2, 1, softcap=cap)
    out, lse = plan.run(q, k, v)
    assert torch.isnan(out[0, 1, 0]).all() and torch.isnan(lse[0, 1, 0])
    keep = [0, 2, 3]
    assert torch.isfinite(out[0, keep].float()).all() and torch.isfinite(out[0, 1, 1].float()).all()


def test_strides(lib):
    """Queries, keys and values inside one fused projection, a head-major cache, an output inside a wider tensor, one
    cache for the whole batch."""
    B, s, hq, hkv = 2, 200, 4, 2
    fused = rnd(B, s, hq + 2 * hkv, 128, seed=9)
    q, k, v = fused[:, :, :hq], fused[:, :, hq:hq + hkv], fused[:, :, hq + hkv:]
    wide = torch.zeros(B, s, hq, 256, dtype=BF, device="cuda")
    plan = binding.Attention(B, s, s, hq, hkv)
    out, lse = plan.run(q, k, v, out=wide[..., 128:])
    R.compare(out, lse, R.attention(q, k, v), "fused")
    assert torch.all(wide[..., :128] == 0)
    kh, vh = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    out2, _ = plan.run(q.contiguous(), kh, vh)
    assert torch.equal(out2, out.contiguous())
    ke, ve = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
    assert ke.stride(0) == 0
    out3, lse3 = plan.run(q, ke, ve)
    R.compare(out3, lse3, R.attention(q, ke, ve), "one cache")
    plan.check()


def test_cache_offsets_past_32_bits(lib):
    """One layer's view of a token-major cache of 32 layers x 131072 tokens (2^32 elements)."""
    n, layers, hkv = 131072, 32, 8
    cache = torch.empty(n, layers, hkv, 128, dtype=BF, device="cuda")
    k = cache[None, :, layers - 1]
    k.copy_(rnd(1, n, hkv, 128, seed=4))
    assert k.stride(1) * n > 2 ** 31
    v = rnd(1, n, hkv, 128, seed=5)
    q = rnd(1, 1, 32, 128, seed=6)
    plan = binding.Attention(1, 1, n, 32, hkv)
    out, lse = plan.run(q, k, v)
    plan.check()
    R.compare(out, lse, R.attention(q, k, v))


def test_long_prompt_rows(lib):
    """A 32K prompt of the 32-head shape: the first, last and odd rows of every head against the definition."""
    s, hq, hkv = 32768, 32, 8
    q, k, v = rnd(1, s, hq, 128), rnd(1, s, hkv, 128, seed=2), rnd(1, s, hkv, 128, seed=3)
    plan = binding.Attention(1, s, s, hq, hkv)
    out, lse = plan.run(q, k, v)
    plan.check()
    rows = torch.tensor([0, 1, 127, 128, 4095, 4096, 10001, 20000, 32766, 32767], device="cuda")
    for h in range(hq):
        ok = R.visible(rows, s)
        o, ls, eo, el = R.attention_rows(q[0, rows, h], k[0, :, h // 4], v[0, :, h // 4], ok, rows,
                                         torch.arange(s, device="cuda"), 1 / math.sqrt(128))
        assert torch.all((out[0, rows, h].double() - o).abs() <= eo) and torch.all((lse[0, rows, h].double() - ls).abs() <= el)


def test_same_results_on_every_run(lib):
    for sq, skv in ((1, 9000), (500, 500)):
        q, k, v = rnd(3, sq, 8, 128), rnd(3, skv, 2, 128, seed=2), rnd(3, skv, 2, 128, seed=3)
        plan = binding.Attention(3, sq, skv, 8, 2)
        first = [t.clone() for t in plan.run(q, k, v)]
        for _ in range(3):
            again = plan.run(q, k, v)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_lengths_out_of_range_are_clamped_and_reported(lib):
    q, k, v = rnd(2, 1, 4, 128), rnd(2, 100, 2, 128, seed=2), rnd(2, 100, 2, 128, seed=3)
    plan = binding.Attention(2, 1, 100, 4, 2)
    out, lse = plan.run(q, k, v, kv_len=i32([5000, -3]))
    with pytest.raises(binding.QEvictError) as e:
        plan.check()
    assert e.value.status == binding.EDEVICE
    plan.check()                                  # reported once
    R.compare(out, lse, R.attention(q, k, v, kv_len=[100, 0]))


def test_a_stream_given_by_the_caller(lib):
    """Inputs made on the current stream, the call on another that waits for it, new outputs read after a wait back."""
    side = torch.cuda.Stream()
    q, k, v = rnd(2, 40, 8, 128), rnd(2, 3000, 2, 128, seed=2), rnd(2, 3000, 2, 128, seed=3)
    plan = binding.Attention(2, 40, 3000, 8, 2)
    side.wait_stream(torch.cuda.current_stream())
    out, lse = plan.run(q, k, v, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    R.compare(out, lse, R.attention(q, k, v))
    plan.check(stream=side)


@pytest.mark.parametrize("sq", [1, 600])
def test_a_plan_made_while_its_stream_is_busy(lib, sq):
    """A plan made behind queued work, in memory that holds other bits, and used at once on a stream that waits for nothing."""
    side = torch.cuda.Stream()
    q, k, v = rnd(2, sq, 8, 128), rnd(2, 600, 2, 128, seed=2), rnd(2, 600, 2, 128, seed=3)
    torch.cuda.synchronize()
    torch.full((binding.Attention(2, sq, 600, 8, 2).work.numel(),), 255, dtype=torch.uint8, device="cuda")
    big = torch.ones(1 << 28, device="cuda")
    for _ in range(20):
        big.mul_(1.0)
    plan = binding.Attention(2, sq, 600, 8, 2)
    out, lse = plan.run(q, k, v, stream=side)
    plan.check(stream=side)
    R.compare(out, lse, R.attention(q, k, v))


def test_an_error_leaves_a_usable_plan(lib):
    """The count of units given out starts anew after a reported error."""
    q, k, v = rnd(2, 600, 8, 128), rnd(2, 600, 2, 128, seed=2), rnd(2, 600, 2, 128, seed=3)
    plan = binding.Attention(2, 600, 600, 8, 2)
    plan.run(q, k, v)
    plan.work[:4] = torch.tensor([1, 0, 0, 0], dtype=torch.uint8)        # a wait that ran out
    plan.work[128:132] = torch.tensor([3, 0, 0, 0], dtype=torch.uint8)   # and left a count
    with pytest.raises(binding.QEvictError):
        plan.check()
    assert not plan.work[:256].any()
    R.compare(*plan.run(q, k, v), R.attention(q, k, v))
    plan.check()


def test_captured_plan_made_in_the_capture(lib):
    q, k, v = rnd(2, 300, 8, 128), rnd(2, 300, 2, 128, seed=2), rnd(2, 300, 2, 128, seed=3)
    binding.Attention(2, 300, 300, 8, 2).run(q, k, v)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = binding.Attention(2, 300, 300, 8, 2)
        out, lse = plan.run(q, k, v)
    for _ in range(3):
        graph.replay()
    R.compare(out, lse, R.attention(q, k, v))
    plan.check()


def test_zero_logits_under_the_smallest_cap(lib):
    """tanh(0) stays 0 where the powers of scale / cap are largest: a mean of the visible values."""
    q, k, v = torch.zeros(1, 200, 4, 128, dtype=BF, device="cuda"), rnd(1, 200, 2, 128, seed=2), rnd(1, 200, 2, 128, seed=3)
    for cap in (2.0 ** -14, 2.0 ** 99):
        plan = binding.Attention(1, 200, 200, 4, 2, softcap=cap, scale=1.0)
        out, lse = plan.run(q, k, v)
        plan.check()
        R.compare(out, lse, R.attention(q, k, v, scale=1.0, cap=cap))


def test_bias_at_positions_past_fp32_integers(lib):
    """A token at position 2^24 + 4097 and zero keys: the logits are -slope |p - j|, lse = -log(1 - exp(-slope)) up to
    exp(-slope 2^24).  A distance that was off by one key would move lse by the slope, 0.5."""
    n, slope = 2 ** 24 + 4098, 0.5
    kv = torch.zeros(1, n, 1, 128, dtype=BF, device="cuda")
    plan = binding.Attention(1, 1, n, 1, 1)
    out, lse = plan.run(rnd(1, 1, 1, 128), kv, kv, slopes=torch.tensor([slope], device="cuda"))
    plan.check()
    assert not out.any()
    # Terms of 32 keys at a time stay below 32 in log2 units, whose half step is 2^-20: 16 sums of the bias along the keys,
    # four more roundings, and the exponential's and logarithm's 2^-22 each: less than 21 * 2^-20.
    assert abs(lse.item() + math.log(1 - math.exp(-slope))) <= 21 * 2.0 ** -20


def test_plans_of_one_workspace_size_do_not_share(lib):
    """Calls of different shapes in turn on one stream, each plan with its own workspace, results unchanged."""
    plans = []
    for sq, skv in ((1, 5000), (600, 600), (1, 700), (100, 9000)):
        q, k, v = rnd(2, sq, 8, 128), rnd(2, skv, 2, 128, seed=2), rnd(2, skv, 2, 128, seed=3)
        plan = binding.Attention(2, sq, skv, 8, 2)
        plans.append((plan, q, k, v, plan.run(q, k, v)))
    again = [p.run(q, k, v) for p, q, k, v, _ in plans for _ in range(2)]
    for n, (p, q, k, v, first) in enumerate(plans):
        for a in again[2 * n:2 * n + 2]:
            assert torch.equal(a[0], first[0]) and torch.equal(a[1], first[1])


def test_graph_replay_and_another_stream(lib):
    """Captured with device lengths that change between replays; two plans replayed on two streams at once."""
    B, skv = 4, 3000
    graphs = []
    for n in range(2):
        st = {"q": rnd(B, 1, 8, 128, seed=n), "k": rnd(B, skv, 2, 128, seed=10 + n), "v": rnd(B, skv, 2, 128, seed=20 + n)}
        st["len"] = i32([skv] * B)
        st["plan"] = binding.Attention(B, 1, skv, 8, 2)
        st["out"], st["lse"] = torch.zeros_like(st["q"]), torch.zeros(B, 1, 8, device="cuda")
        args = dict(out=st["out"], lse=st["lse"], kv_len=st["len"])
        st["stream"] = torch.cuda.Stream()
        st["stream"].wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st["stream"]):
            st["plan"].run(st["q"], st["k"], st["v"], **args)
        st["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(st["graph"], stream=st["stream"]):
            st["plan"].run(st["q"], st["k"], st["v"], **args)
        graphs.append(st)
    torch.cuda.synchronize()
    for lens in ([3000, 1, 128, 2999], [0, 700, 129, 5]):
        for st in graphs:
            with torch.cuda.stream(st["stream"]):
                st["len"].copy_(i32(lens))
                for _ in range(3):
                    st["graph"].replay()
        torch.cuda.synchronize()
        for st in graphs:
            st["plan"].check()
            R.compare(st["out"], st["lse"], R.attention(st["q"], st["k"], st["v"], kv_len=lens))


# ------------------------------------------------------------------------------------------------ shared prefix

def run_prefix(B, sq, pre, skv, hq, hkv, dtype=BF, cap=0.0, slopes=False, lens=None, seed=1):
    q = rnd(B, sq, hq, 128, seed=seed, dtype=dtype, gain=1.5)
    kp, vp = rnd(pre, hkv, 128, seed=seed + 1, dtype=dtype), rnd(pre, hkv, 128, seed=seed + 2, dtype=dtype)
    k, v = rnd(B, skv, hkv, 128, seed=seed + 3, dtype=dtype), rnd(B, skv, hkv, 128, seed=seed + 4, dtype=dtype)
    sl = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device="cuda") if slopes else None
    plan = binding.PrefixAttention(B, sq, pre, skv, hq, hkv, dtype=dtype, softcap=cap)
    out, lse = plan.run(q, kp, vp, k, v, slopes=sl, kv_len=None if lens is None else i32(lens))
    plan.check()
    R.compare(out, lse, R.attention(q, k, v, kv_len=lens, slopes=sl, cap=cap, k_prefix=kp, v_prefix=vp))


@pytest.mark.parametrize("B", [1, 3, 32, 33, 70])
@pytest.mark.parametrize("pre", [1, 128, 1000])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_shared_prefix(lib, B, pre, dtype):
    run_prefix(B, 1, pre, 40, 8, 2, dtype, lens=[1 + (i * 7) % 40 for i in range(B)])


@pytest.mark.parametrize("sq", [1, 2, 3, 32])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (6, 2)])
def test_shared_prefix_drafted_tokens(lib, sq, hq, hkv):
    run_prefix(5, sq, 333, 50, hq, hkv, lens=[50, sq, 40, sq + 1, 33])


@pytest.mark.parametrize("cap,slopes", [(30.0, False), (0.0, True), (10.0, True)])
def test_shared_prefix_capped_and_biased(lib, cap, slopes):
    run_prefix(7, 2, 700, 300, 8, 2, cap=cap, slopes=slopes, lens=[2, 300, 129, 5, 17, 128, 256])


def test_shared_prefix_at_decode_size(lib):
    """16 sequences of the 32-head shape behind a 32K prompt; and some without own keys yet."""
    run_prefix(16, 1, 32768, 256, 32, 8, lens=[1 + 17 * i for i in range(16)])
    run_prefix(4, 1, 2000, 8, 8, 2, lens=[0, 1, 8, 0])


@pytest.mark.parametrize("sq,pre", [(2, 4000), (5, 256), (30, 20), (32, 1), (16, 129)])
@pytest.mark.parametrize("cap,slopes", [(0.0, False), (30.0, True)])
def test_shared_prefix_queries_inside_the_prefix(lib, sq, pre, cap, slopes):
    """Fewer own keys than queries: the first queries sit inside the prefix, or before it, and see it up to themselves."""
    run_prefix(4, sq, pre, 40, 8, 2, cap=cap, slopes=slopes, lens=[0, 1, sq - 1, sq])
    run_prefix(3, sq, pre, 1, 8, 2, cap=cap, slopes=slopes)


def test_shared_prefix_values_seen_by_some_queries(lib):
    """Infinities in the prefix's last keys, which only the later queries see."""
    q, kp, vp = rnd(2, 6, 8, 128), rnd(300, 2, 128, seed=2), rnd(300, 2, 128, seed=3)
    k, v = rnd(2, 10, 2, 128, seed=4), rnd(2, 10, 2, 128, seed=5)
    vp[297, 0, 5] = math.inf
    kp[299, 1, 7] = math.nan
    plan = binding.PrefixAttention(2, 6, 300, 10, 8, 2)
    out, lse = plan.run(q, kp, vp, k, v, kv_len=i32([1, 10]))
    plan.check()
    R.compare(out, lse, R.attention(q, k, v, kv_len=[1, 10], k_prefix=kp, v_prefix=vp))


def test_shared_prefix_garbage_behind_own_keys(lib):
    B, pre, skv = 3, 200, 64
    q, kp, vp = rnd(B, 1, 8, 128), rnd(pre, 2, 128, seed=2), rnd(pre, 2, 128, seed=3)
    k, v = rnd(B, skv, 2, 128, seed=4), rnd(B, skv, 2, 128, seed=5)
    lens = [10, 64, 1]
    for b, n in enumerate(lens):
        k[b, n:] = math.nan
        v[b, n:] = math.nan
    plan = binding.PrefixAttention(B, 1, pre, skv, 8, 2)
    out, lse = plan.run(q, kp, vp, k, v, kv_len=i32(lens))
    plan.check()
    R.compare(out, lse, R.attention(q, k, v, kv_len=lens, k_prefix=kp, v_prefix=vp))


def test_shared_prefix_equals_joined_attention(lib):
    """The same keys through qevict_attn: within two of the output's half steps plus the probabilities'."""
    B, pre, skv = 4, 500, 60
    q, kp, vp = rnd(B, 1, 8, 128), rnd(pre, 2, 128, seed=2), rnd(pre, 2, 128, seed=3)
    k, v = rnd(B, skv, 2, 128, seed=4), rnd(B, skv, 2, 128, seed=5)
    out, lse = binding.PrefixAttention(B, 1, pre, skv, 8, 2).run(q, kp, vp, k, v)
    joined = [torch.cat([p[None].expand(B, -1, -1, -1), x], dim=1) for p, x in ((kp, k), (vp, v))]
    ref = R.attention(q, *joined)
    R.compare(out, lse, ref)
    out2, lse2 = binding.Attention(B, 1, pre + skv, 8, 2).run(q, *joined)
    R.compare(out2, lse2, ref)
