"""Refusals of the rotary and attention operators that need no GPU: no gradient is recorded, sizes whose products leave 64
bits are refused."""
import ctypes

import pytest
import torch

from recoverable_quantized_kv_gb300 import binding as B


@pytest.mark.parametrize("name", ["q", "k", "v", "slopes", "k_prefix", "v_prefix"])
def test_inputs_that_require_a_gradient(name):
    """Refused before anything else is looked at (these are CPU tensors, refused for that otherwise)."""
    t = {n: torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16) for n in ("q", "k", "v")}
    t.update(k_prefix=torch.zeros(3, 4, 128, dtype=torch.bfloat16), v_prefix=torch.zeros(3, 4, 128, dtype=torch.bfloat16),
             slopes=torch.zeros(4))
    t[name].requires_grad_()
    attn, step, rope = (object.__new__(c) for c in (B.Attention, B.PrefixAttention, B.Rope))
    rope.index = attn.index = step.index = 0
    step.desc = attn.desc = None
    calls = [lambda: step.run(t["q"], t["k_prefix"], t["v_prefix"], t["k"], t["v"], slopes=t["slopes"])]
    if "prefix" not in name:
        calls.append(lambda: attn.run(t["q"], t["k"], t["v"], slopes=t["slopes"]))
    if name in ("q", "k"):
        calls.append(lambda: rope.apply(t["q"], t["k"]))
    for call in calls:
        with pytest.raises(B.QEvictError, match="no gradient is recorded") as e:
            call()
        assert e.value.status == B.EINVAL
        with torch.no_grad(), pytest.raises(Exception) as e:
            call()
        assert "gradient" not in str(e.value)
