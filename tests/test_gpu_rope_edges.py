"""Rotary tables at positions and angles where the phase needs more than fp64 holds."""
import math
from decimal import Decimal, getcontext

import pytest
import torch

from recoverable_quantized_kv_gb300 import binding

pytestmark = pytest.mark.gpu
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


def exact_entry(pos, theta):
    """cos and sin of pos * theta, the fp64 theta taken as it is: reduced in 90 digits, then below pi in fp64."""
    turns = Decimal(pos) * Decimal(theta) / (2 * PI)
    a = float((turns - turns.to_integral_value()) * 2 * PI)
    return math.cos(a), math.sin(a)


@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(base=0.77 ** -64), dict(base=0.9 ** -64, rot_dim=64),
                                dict(scaling="linear", factor=0.125), dict(scaling="linear", factor=1e-6),
                                dict(scaling="linear", factor=2.0 ** -39, rot_dim=32), dict(base=1e-9, rot_dim=8),
                                dict(scaling="parts", factor=16.0, orig_len=8192), dict(scaling="ntk", factor=8.0)])
@pytest.mark.parametrize("first", [0, 131000, 2 ** 24 - 3, 2 ** 29, 2 ** 31 - 7])
def test_table_holds_its_bound_everywhere(lib, kw, first):
    """Within 2^-23 of position * theta_i, for every accepted position and angles up to 2^40."""
    getcontext().prec = 90
    th = binding.rope_angles(**kw)
    assert max(th) <= 2.0 ** 40
    got = binding.rope_table(7, first=first, **kw).cpu().double()
    want = torch.tensor([[exact_entry(first + r, t) for t in th] for r in range(7)], dtype=torch.float64)
    assert (got - want).abs().max().item() <= 2.0 ** -23
