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


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cap", [64.0, 1000.0, 1e5])
@pytest.mark.parametrize("sq,skv", [(1, 700), (200, 200)])
def test_large_caps_keep_small_logits(lib, dtype, cap, sq, skv):
    """Heads whose logits reach past the cap beside heads of ordinary ones, in one tile: the ordinary ones keep their digits."""
    q, k, v = rnd(1, sq, 4, 128, dtype=dtype), rnd(1, skv, 1, 128, seed=2, dtype=dtype), rnd(1, skv, 1, 128, seed=3, dtype=dtype)
    q *= 0.1
    q[:, :, 0] *= cap / 4.5      # logits of deviation 11.3 * 0.1, and a quarter of the cap
    plan = binding.Attention(1, sq, skv, 4, 1, dtype=dtype, softcap=cap, scale=1.0)
    out, lse = plan.run(q, k, v)
    plan.check()
    S.check(out, lse, q, k, v, cap=cap, scale=1.0, rows=[0] if sq == 1 else [0, 1, 31, 32, 63, 100, 199])


@pytest.mark.parametrize("top", [2.0 ** 20, 2.0 ** 33, 2.0 ** 40])
@pytest.mark.parametrize("cap", [2.0 ** 61, 2.0 ** 70, 2.0 ** 90, 2.0 ** 99])
@pytest.mark.parametrize("sq", [1, 300])
def test_caps_near_the_largest(lib, top, cap, sq):
    """One key of every row's product is 128 top^2, far above the others: the row is that key's value."""
    q, k, v = rnd(1, sq, 4, 128), rnd(1, 300, 2, 128, seed=2), rnd(1, 300, 2, 128, seed=3)
    q.fill_(top)
    k[0, 0] = top
    plan = binding.Attention(1, sq, 300, 4, 2, softcap=cap, scale=1.0)
    out, lse = plan.run(q, k, v)
    plan.check()
    S.check(out, lse, q, k, v, cap=cap, scale=1.0, rows=range(0, sq, 37))
    assert torch.equal(out[0, -1].view(2, 2, 128), v[0, 0][:, None].expand(2, 2, 128))


@pytest.mark.parametrize("cap,scale", [(20.0, 0.0), (64.0, 0.0), (2000.0, 0.0), (3e4, 0.05), (1e6, 0.0), (1e9, 0.0),
                                       (2.0 ** 40, 1.0), (2.0 ** 99, 1.0), (50.0, 1e-4), (50.0, 1e-9), (2.0 ** -13, 1.0)])
@pytest.mark.parametrize("skv", [1, 200])
def test_capped_logits_over_the_whole_range_of_caps(lib, cap, scale, skv):
    """Rows of products from -1.5 to 1.5 times cap / scale against one key (behind it keys of the same rows that none sees): lse is
    the capped logit."""
    n, real = 1000, scale or 1 / math.sqrt(128)
    top = cap / real
    q, k = torch.zeros(1, n, 1, 128, dtype=BF, device="cuda"), torch.zeros(1, skv, 1, 128, dtype=BF, device="cuda")
    b = 2.0 ** round(math.log2(top) / 2)
    q[0, :, 0, 5] = (torch.linspace(-1.5, 1.5, n, device="cuda", dtype=torch.float64) * (top / b)).to(BF)
    k[..., 5] = b
    plan = binding.Attention(1, n, skv, 1, 1, causal=False, softcap=cap, scale=scale)
    out, lse = plan.run(q, k, torch.ones_like(k), kv_len=i32([1]))
    plan.check()
    want = cap * torch.tanh(q[0, :, 0, 5].double() * b * (torch.tensor(scale or 0.0, dtype=torch.float32).double().item() or real) / cap)
    # scale / cap, its product and the logarithm's two conversions are rounded (2^-22), tanh is off by up to 2^-20 of itself or, up
    # to a cap of 64, by 8 * 2^-22 of the cap
    tol = 2.0 ** -19 * want.abs() + 8 * 2.0 ** -22 * min(cap, 64.0)
    assert ((lse[0, :, 0].double() - want).abs() <= tol).all()
    # the one weight is 2^e, e the rounding of a maximum up to 10^6 (2^-4 there): rounded to bf16 against an unrounded sum, and
    # the output once, half a step each
    assert ((out.float() - 1).abs() <= 2 * S.HALF[BF]).all()


@pytest.mark.parametrize("dtype,size", [(FP, 1000), (FP, 5000), (FP, 6001), (FP, 12004), (FP, 60000), (BF, 8064), (BF, 20096), (BF, 24064),
                                        (BF, 1e15)])
@pytest.mark.parametrize("sq,skv", [(1, 500), (300, 300), (20, 9000)])
@pytest.mark.parametrize("slopes", [False, True])
def test_logits_whose_last_digit_is_large(lib, dtype, size, sq, skv, slopes):
    """One key's logit is 10^7 and more, where fp32 numbers lie whole powers of two apart: the row is that key's value."""
    q, k, v = rnd(1, sq, 4, 128, dtype=dtype), rnd(1, skv, 2, 128, seed=2, dtype=dtype), rnd(1, skv, 2, 128, seed=3, dtype=dtype)
    q.fill_(size)
    k.mul_(1e-3)
    k[0, 0] = size
    sl = torch.tensor([0.5, 0.25, 0.125, 0.0], device="cuda") if slopes else None
    plan = binding.Attention(1, sq, skv, 4, 2, dtype=dtype)
    out, lse = plan.run(q, k, v, slopes=sl)
    plan.check()
    assert torch.equal(out[0].view(sq, 2, 2, 128), v[0, 0][None, :, None].expand(sq, 2, 2, 128))
    want = 128 * q[0, 0, 0, 0].double() ** 2 / math.sqrt(128)
    # the product's running sum (128 roundings), its scale (2), the exponent's base and the logarithm's way back (3)
    assert ((lse.double() - want).abs() <= 133 * 2.0 ** -24 * want + (0 if sl is None else 0.5 * skv)).all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_large_logits_of_both_signs(lib, dtype):
    """Rows of every magnitude from 1 to 10^10 in one tile, with equal keys at the top: the mean of their values."""
    s = 200
    q, k, v = rnd(1, s, 2, 128, dtype=dtype), rnd(1, s, 1, 128, seed=2, dtype=dtype), rnd(1, s, 1, 128, seed=3, dtype=dtype)
    q[0] = (torch.logspace(0, 4.5, s, device="cuda")[:, None, None] * torch.ones(2, 128, device="cuda")).to(dtype)
    k[:] = -300.0
    k[0, 0:9:4] = 300.0
    plan = binding.Attention(1, s, s, 2, 1, dtype=dtype)
    out, lse = plan.run(q, k, v)
    plan.check()
    for i in range(s):
        top = v[0, 0:min(i, 8) + 1:4, 0].double()
        # weights of 1 / 1, 1 / 2 or 1 / 3, rounded once each, and the output once
        assert ((out[0, i].double() - top.mean(0)).abs() <= S.HALF[dtype] * (top.abs().mean(0) + top.mean(0).abs()) + 2.0 ** -22).all()


def test_logits_from_far_below_to_far_above(lib):
    """Tiles of logits of -10^9, 10^9, -10^7, 0 in every order along the keys: the largest that a row sees decides."""
    s, size = 640, 10000.0
    for dtype in (BF, FP):
        q, k, v = rnd(1, s, 2, 128, dtype=dtype), rnd(1, s, 1, 128, seed=2, dtype=dtype), rnd(1, s, 1, 128, seed=3, dtype=dtype)
        q.fill_(size)
        for order in ((0, 1, 2, 3, 2), (1, 0, 3, 2, 0), (2, 0, 2, 0, 3), (3, 2, 0, 2, 1), (0, 2, 0, 2, 0)):
            level = torch.tensor([-1e4, 1e4, -1e2, 0.0], device="cuda")[torch.tensor(order, device="cuda").repeat_interleave(128)]
            k[0, :, 0] = level[:, None].to(dtype)
            plan = binding.Attention(1, s, s, 2, 1, dtype=dtype)
            out, lse = plan.run(q, k, v)
            plan.check()
            for i in range(0, s, 61):
                vv = v[0, :i + 1, 0][level[:i + 1] == level[:i + 1].max()].double()
                tol = S.HALF[dtype] * (vv.abs().mean(0) + vv.mean(0).abs()) + (len(vv) + 64) * 2.0 ** -24 * vv.abs().mean(0) + 2.0 ** -24
                assert ((out[0, i].double() - vv.mean(0)).abs() <= tol).all(), (order, i)


@pytest.mark.parametrize("dtype,size", [(FP, 300), (FP, 1000), (FP, 6001), (FP, 60000), (BF, 300), (BF, 20096), (BF, 1e15)])
@pytest.mark.parametrize("sq,skv", [(1, 300), (300, 300), (7, 9000), (200, 9000)])
@pytest.mark.parametrize("one", [None, 0, -1])
def test_logits_far_below_zero(lib, dtype, size, sq, skv, one):
    """Every key's logit is -10^6 and less: the mean of the visible values; one key of logit 0 among them: that key's value."""
    q, k, v = rnd(1, sq, 4, 128, dtype=dtype), rnd(1, skv, 2, 128, seed=2, dtype=dtype), rnd(1, skv, 2, 128, seed=3, dtype=dtype)
    q.fill_(size)
    k.fill_(-size)
    if one is not None:
        k[0, one] = 0
    plan = binding.Attention(1, sq, skv, 4, 2, dtype=dtype)
    out, lse = plan.run(q, k, v)
    plan.check()
    want = -128 * q[0, 0, 0, 0].double() ** 2 / math.sqrt(128)
    for i in sorted({0, sq // 2, sq - 1}):
        n = skv - sq + i + 1
        hit = one is not None and (one == 0 or i == sq - 1)
        for h in range(4):
            vv = v[0, one if one == 0 else skv - 1, h // 2][None].double() if hit else v[0, :n, h // 2].double()
            # equal weights, each rounded by half a step, and the output; n sums; parts' sums of weights, log2 n of them lost
            # behind a maximum of -10^6 and less are not: parts of equal maxima weigh by their sums
            tol = S.HALF[dtype] * (vv.abs().mean(0) + vv.mean(0).abs()) + (n + 64) * 2.0 ** -24 * vv.abs().mean(0) + 2.0 ** -24
            assert ((out[0, i, h].double() - vv.mean(0)).abs() <= tol).all(), (i, h)
            if hit:
                assert abs(lse[0, i, h].item()) <= 2.0 ** -20
            else:
                assert abs(lse[0, i, h].item() - want.item() - math.log(n)) <= 140 * 2.0 ** -24 * abs(want.item())


# ------------------------------------------------------------------------------------------------ weights far below the largest

def sink(dtype, skv, hkv, bits, at):
    """Keys whose logit is 0 and one, at `at`, whose logit is bits * ln 2 and whose value is 0; the other values near 1."""
    k, v = torch.zeros(1, skv, hkv, 128, dtype=dtype, device="cuda"), 1 + rnd(1, skv, hkv, 128, seed=3, dtype=dtype, gain=0.25)
    k[0, at, :, 0] = bits * math.log(2)
    v[0, at] = 0
    return k, v


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bits", [20.0, 24.5, 25.5, 28.0])
@pytest.mark.parametrize("sq,skv", [(1, 60000), (1, 900), (300, 4096), (20, 60000)])
def test_many_small_weights_beside_a_large_one(lib, dtype, bits, sq, skv):
    """The last tokens see one key of weight 1 and thousands of weight 2^-bits, which together make the output."""
    q = torch.zeros(1, sq, 4, 128, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    k, v = sink(dtype, skv, 2, bits, skv - sq)
    plan = binding.Attention(1, sq, skv, 4, 2, dtype=dtype, scale=1.0)
    out, lse = plan.run(q, k, v)
    plan.check()
    S.check(out, lse, q, k, v, scale=1.0, rows=sorted({0, sq // 2, sq - 1}))
    assert (out[0, -1].float() > 0).all()


@pytest.mark.parametrize("bits", [20.0, 25.5])
def test_many_small_weights_behind_a_shared_prefix(lib, bits):
    q = torch.zeros(3, 1, 4, 128, dtype=FP, device="cuda")
    q[..., 0] = 1.0
    kp, vp = (x[0] for x in sink(FP, 20000, 2, bits, 19990))
    k, v = torch.zeros(3, 8, 2, 128, dtype=FP, device="cuda"), torch.ones(3, 8, 2, 128, dtype=FP, device="cuda")
    plan = binding.PrefixAttention(3, 1, 20000, 8, 4, 2, dtype=FP, scale=1.0)
    out, lse = plan.run(q, kp, vp, k, v)
    plan.check()
    S.check(out, lse, q, k, v, scale=1.0, k_prefix=kp, v_prefix=vp)


# ------------------------------------------------------------------------------------------------ plans

def test_a_report_leaves_the_count_of_units_alone(lib):
    """Only a wait that ran out leaves the count undone.  A clamped length does not, and a call on another stream may be drawing
    from the count while the word is read."""
    q, k, v = rnd(2, 600, 8, 128), rnd(2, 600, 2, 128, seed=2), rnd(2, 600, 2, 128, seed=3)
    plan = binding.Attention(2, 600, 600, 8, 2)
    plan.run(q, k, v, kv_len=i32([601, 600]))
    plan.work[128:132] = torch.tensor([3, 0, 0, 0], dtype=torch.uint8)   # as if a call were under way
    with pytest.raises(binding.QEvictError) as e:
        plan.check()
    assert e.value.status == binding.EDEVICE
    assert e.value.word == 8 and plan.work[128].item() == 3 and not plan.work[:4].any()


def test_a_status_is_reported_once(lib):
    """Reported once, then clean."""
    plan = binding.Attention(1, 1, 100, 4, 2)
    rope = binding.Rope(binding.rope_table(16))
    for word, check in ((plan.work[:4], plan.check), (rope.status.view(torch.uint8)[:4], rope.check)):
        check()
        word[0] = 8
        with pytest.raises(binding.QEvictError):
            check()
        assert not word.any()
        check()


@pytest.mark.parametrize("given", [False, True])
def test_a_plan_dropped_while_its_call_runs(lib, given):
    """A plan made on one stream and used on another, as the current one or by name: its workspace is not handed to the first
    stream while the call runs."""
    side = torch.cuda.Stream()
    q, k, v = rnd(2, 1, 8, 128), rnd(2, 3000, 2, 128, seed=2), rnd(2, 3000, 2, 128, seed=3)
    table = binding.rope_table(4000)
    torch.cuda.synchronize()
    for make in (lambda: binding.Attention(2, 1, 3000, 8, 2), lambda: binding.PrefixAttention(2, 1, 3000, 3000, 8, 2),
                 lambda: binding.Rope(table)):
        plan = make()
        own = plan.status if isinstance(plan, binding.Rope) else plan.work
        at, size = own.data_ptr(), own.numel() * own.element_size()
        args = {"Attention": (q, k, v), "PrefixAttention": (q, k[0], v[0], k, v), "Rope": (q, k[:, :1])}[type(plan).__name__]
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)   # about 0.1 s
            outs = plan.run(*args, stream=side if given else None) if hasattr(plan, "run") else \
                plan.apply(*args, stream=side if given else None)
        del plan, own
        others = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert at not in [x.data_ptr() for x in others]
        torch.cuda.synchronize()
        del outs, others


def test_gradients_are_refused(lib):
    """No graph is recorded, so tensors that ask for one are refused; under no_grad, and detached, they are taken."""
    q, k, v = rnd(1, 2, 4, 128), rnd(1, 9, 2, 128, seed=2), rnd(1, 9, 2, 128, seed=3)
    plan, step = binding.Attention(1, 2, 9, 4, 2), binding.PrefixAttention(1, 2, 9, 9, 4, 2)
    rope = binding.Rope(binding.rope_table(16))
    sl = torch.ones(4, device="cuda")
    calls = {"q": lambda: plan.run(q, k, v), "k": lambda: plan.run(q, k, v), "v": lambda: step.run(q, k[0], v[0], k, v),
             "slopes": lambda: plan.run(q, k, v, slopes=sl), "rope": lambda: rope.apply(q, k[:, :2])}
    for name, call in calls.items():
        t = {"q": q, "k": k, "v": v, "slopes": sl, "rope": k}[name]
        want = call()
        t.requires_grad_()
        with pytest.raises(binding.QEvictError) as e:
            call()
        assert e.value.status == binding.EINVAL
        with torch.no_grad():
            got = call()
        t.requires_grad_(False)
        assert all(torch.equal(x, y) for x, y in zip(want, got))


# ------------------------------------------------------------------------------------------------ infinities and NaN that some rows see

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("cap,slopes", [(0.0, False), (20.0, False), (0.0, True), (2.0, True)])
def test_keys_that_some_rows_see(lib, dtype, bad, cap, slopes):
    """A later token's key, one of another document and one behind the end hold infinities or NaN: the rows that do not see it
    keep their bounds."""
    s, n = 300, [270, 300]
    q, k, v = rnd(2, s, 4, 128, dtype=dtype), rnd(2, s, 2, 128, seed=2, dtype=dtype), rnd(2, s, 2, 128, seed=3, dtype=dtype)
    k[0, 200, 0, 3], k[1, 129, 1, 77], k[0, 270:], v[0, 270:] = bad, bad, bad, bad
    sl = torch.tensor([0.5, 0.25, 0.125, 0.0], device="cuda") if slopes else None
    arrays = dict(slopes=sl, kv_len=i32(n), q_len=i32(n))
    plan = binding.Attention(2, s, s, 4, 2, dtype=dtype, softcap=cap)
    some = [0, 1, 63, 127, 128, 129, 130, 199, 200, 201, 269]
    out, lse = plan.run(q, k, v, **arrays)
    S.check(out, lse, q, k, v, "later", rows=some, cap=cap, **arrays)
    ids = torch.zeros(2, s, dtype=torch.int32, device="cuda")
    ids[0, 150:], ids[1, 130:] = 1, 2
    out, lse = plan.run(q, k, v, doc_ids=ids, **arrays)
    S.check(out, lse, q, k, v, "documents", rows=some, cap=cap, doc_ids=ids, **arrays)
    pl = i32([250, 40])
    out, lse = plan.run(q, k, v, prefix_len=pl, **arrays)
    S.check(out, lse, q, k, v, "prefix", rows=some, cap=cap, prefix_len=pl, **arrays)
    full = binding.Attention(2, 7, s, 4, 2, dtype=dtype, causal=False, softcap=cap)
    out, lse = full.run(q[:, :7], k, v, slopes=sl, kv_len=i32([200, 129]))
    S.check(out, lse, q[:, :7], k, v, "not causal", causal=False, cap=cap, slopes=sl, kv_len=[200, 129])
    plan.check()
    full.check()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("cap,slopes", [(0.0, False), (20.0, False), (0.0, True)])
def test_shared_prefix_keys_and_values_that_some_queries_see(lib, dtype, cap, slopes):
    """The prefix's last keys and values, and own ones of later drafted tokens, hold infinities or NaN."""
    q, kp, vp = rnd(2, 6, 8, 128, dtype=dtype), rnd(300, 2, 128, seed=2, dtype=dtype), rnd(300, 2, 128, seed=3, dtype=dtype)
    k, v = rnd(2, 10, 2, 128, seed=4, dtype=dtype), rnd(2, 10, 2, 128, seed=5, dtype=dtype)
    vp[297, 0, 5] = math.inf
    kp[299, 1, 7] = math.nan
    sl = torch.tensor([2.0 ** -h for h in range(8)], device="cuda") if slopes else None
    plan = binding.PrefixAttention(2, 6, 300, 10, 8, 2, dtype=dtype, softcap=cap)
    for lens in ([1, 10], [0, 3]):
        out, lse = plan.run(q, kp, vp, k, v, slopes=sl, kv_len=i32(lens))
        S.check(out, lse, q, k, v, str(lens), cap=cap, slopes=sl, kv_len=lens, k_prefix=kp, v_prefix=vp)
    kp, vp = rnd(300, 2, 128, seed=2, dtype=dtype), rnd(300, 2, 128, seed=3, dtype=dtype)
    k[1, 7, 0, 9], v[0, 9, 1, 3] = -math.inf, math.nan
    out, lse = plan.run(q, kp, vp, k, v, slopes=sl)
    S.check(out, lse, q, k, v, "own", cap=cap, slopes=sl, k_prefix=kp, v_prefix=vp)
    plan.check()
