"""Norm with rotation into the cache at the documented largest call: 2^29 rows of heads (needs an MI355X).

Inputs are one row seen from every token, so that only the outputs take memory.
"""
import pytest
import torch

import quantized_linear_layers_fp4_amd as fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def test_largest_write_into_the_cache():
    """fp32, 2^24 tokens of 1 + 31 heads of 128: the last tokens' keys and values reach their slots, and every query is made."""
    n, hkv, d = 1 << 24, 31, 128
    x = torch.randn(1, 1 + 2 * hkv, d, device=DEV)
    q, k, v = (t.expand(n, -1, -1) for t in x.split([1, hkv, hkv], 1))
    slots = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    last = torch.tensor([0, 1, n // 2 + 3, n - 17, n - 2, n - 1], device=DEV)
    slots[last] = torch.arange(6, device=DEV, dtype=torch.int32) + 3
    a, b = fp4.kv4_cache(1, 16, hkv, d), fp4.kv4_cache(1, 16, hkv, d)
    got = fp4.kv4_norm_rope(a, q, k, v, slots)
    want = fp4.kv4_norm_rope(b, *(t[:6].contiguous() for t in (q, k, v)), slots[last].contiguous())
    assert bool((got == want[0]).all()) and torch.equal(a.data, b.data) and int(a.data.count_nonzero()) > 0
