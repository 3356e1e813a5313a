"""Calls whose host thread has not used the GPU before: the first thing that it does is the call, with outputs at hand."""
import threading

import pytest
import torch

from oracle import qevict_oracle as O
from recoverable_quantized_kv_gb300 import binding, synth
from test_gpu_paged_attention import BF, i32, rnd

pytestmark = pytest.mark.gpu


def in_a_thread(call):
    failed = []

    def run():
        try:
            call()
        except BaseException as e:   # noqa: BLE001
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join(120)
    assert not t.is_alive()
    if failed:
        raise failed[0]


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("kind", ["dense", "prefix", "paged"])
def test_attention(lib, kind, stream):
    q, lse = rnd(2, 3, 4, 128), torch.zeros(2, 3, 4, device="cuda")
    if kind == "dense":
        kv, plan = rnd(2, 300, 2, 128), binding.Attention(2, 3, 300, 4, 2)
        args = (q, kv, kv)
    elif kind == "prefix":
        kv, pre, plan = rnd(2, 40, 2, 128), rnd(300, 2, 128), binding.PrefixAttention(2, 3, 300, 40, 4, 2)
        args = (q, pre, pre, kv, kv)
    else:
        kv, plan = rnd(12, 16, 2, 128), binding.PagedAttention(2, 3, 12, 16, 6, 4, 2)
        args = (q, kv, kv, i32([[0, 1, 2, 3, 4, 5], [6, 7, 8, 9, 10, 11]]), i32([5, 60]))
    want, want_lse = plan.run(*args)
    out, side = torch.zeros_like(q), torch.cuda.Stream() if stream else None
    torch.cuda.synchronize()
    in_a_thread(lambda: plan.run(*args, out=out, lse=lse, stream=side))
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_rotations_and_pages(lib):
    rope, q = binding.Rope(binding.rope_table(64)), rnd(1, 20, 2, 128)
    out, cache = torch.zeros_like(q), binding.PagedCache(1, 8, 16, 2, 1, 4)
    want, _ = rope.apply(q)
    rows = rnd(1, 20, 2, 128)
    torch.cuda.synchronize()
    in_a_thread(lambda: rope.apply(q, q_out=out))
    in_a_thread(lambda: cache.reserve(20))
    in_a_thread(lambda: cache.append(rows, rows, layer=0))
    in_a_thread(cache.compact)
    in_a_thread(cache.check)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(cache.k[0, :2].flatten(0, 1)[:20], rows[0])


def test_prefill_scores(lib):
    wl = synth.workload("tiny_4k", prompt_len=1200, n_plant=4)
    cache, ins = binding.Cache(binding.make_config(wl)), synth.prompt_inputs(wl, 0, 0)
    q, k, npw = ins["q"][None].cuda(), ins["k"][None].cuda(), O.prompt_windows(O.Config.from_obj(wl))
    want, got = (torch.zeros(1, npw, device="cuda") for _ in range(2))
    cache.prefill_scores(q, k, want)
    torch.cuda.synchronize()
    in_a_thread(lambda: cache.prefill_scores(q, k, got))
    cache.check()
    assert torch.equal(got, want) and bool(want.any())
