"""Sizes and counts of the paged cache that are no whole numbers: refused, not cut off (no GPU needed)."""
import pytest
import torch

from recoverable_quantized_kv_gb300 import binding as B
from test_pages_paths import host_cache


@pytest.mark.parametrize("n", [16.5, float("nan"), float("inf"), "16", None, [16], torch.tensor(1.5), torch.tensor([1, 2])])
def test_sizes(n):
    with pytest.raises(B.QEvictError) as e:
        B._sizes("PagedCache", page=n)
    assert e.value.status == B.EINVAL


def test_whole_numbers_of_other_types():
    import numpy as np
    assert B._sizes("x", a=np.int64(3), b=True, c=torch.tensor(7), d=-2 ** 31, e=16.0) == (3, 1, 7, -2 ** 31, 16)


@pytest.mark.parametrize("new", [1.5, float("nan"), None, "1"])
def test_reserve(new):
    calls = []
    with pytest.raises(B.QEvictError):
        host_cache(calls).reserve(new)
    assert not calls


@pytest.mark.parametrize("layer", [0.5, 1.5, "0", 2, -1, 2 ** 32])
def test_layers(monkeypatch, layer):
    monkeypatch.setattr(B, "_tensor", lambda *a, **kw: None)   # (which wants tensors on a GPU)
    calls, x = [], torch.zeros(3, 4, 2, 128, dtype=torch.bfloat16)
    c = host_cache(calls)
    c.shape, c.dtype, c.device, c._rows = (2, 10, 16, 2, 128), x.dtype, x.device, {}
    with pytest.raises(B.QEvictError):
        c.append(x, x, layer=layer)
    assert not calls
