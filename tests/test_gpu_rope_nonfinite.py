"""Norm and rotation: an infinity or a NaN, of a row, a gradient or a weight, stays in the columns that the formula takes
it to (needs an MI355X).

Nothing is compared with a tolerance: a column that the spoiled value does not belong to keeps, bit for bit, what it is without
it, and a column that is neither normed nor rotated is the input's.
"""
import pytest
import torch

import quantized_linear_layers_fp4_amd as fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
INF, NAN = float("inf"), float("nan")
# few rows, rows whose last lanes hold nothing, and as many as runs of heads take, the last run with fewer
SIZES = [(5, 3, 2, 64, 32), (9, 2, 1, 40, 16), (3, 2, 2, 256, 112), (4, 4, 1, 128, 0), (33000, 7, 1, 64, 16), (33000, 9, 3, 64, 0)]


def same(a, b):
    return bool(((a == b) & (a.signbit() == b.signbit()) | a.isnan() & b.isnan()).all())


def setup(n, hq, hkv, d, rot, dt):
    g = torch.Generator(device=DEV).manual_seed(n + d)
    q, k = (torch.randn(n, h, d, generator=g, device=DEV).to(dt) for h in (hq, hkv))
    if not rot:
        return q, k, dict(table=None, positions=None)
    return q, k, dict(table=fp4.rope_table(4000, rot), positions=(torch.arange(n, device=DEV) % 4000).int())


def partner(col, rot, il):
    if col >= rot:
        return col
    return col ^ 1 if il else (col + rot // 2) % rot


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,rot", SIZES)
def test_without_the_norm(n, hq, hkv, d, rot, il, dt):
    """Columns past the rotated ones are the input's, whatever it holds; a pair's values reach the pair alone."""
    q, k, how = setup(n, hq, hkv, d, rot, dt)
    how.update(eps=None, interleaved=il)
    for x in (q, k):
        x[n // 2, 0, d - 3] = -0.0
    places = [(0, 0, d - 1, INF), (n - 1, -1, rot, -INF), (n // 2, 0, d - 2, NAN), (n - 1, 0, d - 8, INF)]
    if rot:
        places += [(1, 0, 0, INF), (2, -1, rot - 1, NAN)]

    def run(q, k):
        return (*fp4.qk_norm_rope(q, k, **how), *fp4.qk_norm_rope_backward(q, k, q, k, **how)[:2])
    base = run(q, k)
    q2, k2 = q.clone(), k.clone()
    for x in (q2, k2):
        for t, h, c, v in places:
            x[t, h, c] = v
    for got, was, x in zip(run(q2, k2), base, (q2, k2, q2, k2)):
        assert same(got[..., rot:], x[..., rot:])
        keep = torch.ones(got.shape, dtype=torch.bool, device=DEV)
        for t, h, c, _ in places:
            keep[t, h, c] = keep[t, h, partner(c, rot, il)] = False
        assert same(got[keep], was[keep])
        for t, h, c, _ in places:
            assert not bool(got[t, h, c].isfinite())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("col,value", [(0, INF), (5, NAN), (-1, -INF)])
@pytest.mark.parametrize("n,hq,hkv,d,rot", SIZES)
def test_weights(n, hq, hkv, d, rot, col, value, il, dt):
    """A weight's value reaches its column and the one that this is paired with."""
    q, k, how = setup(n, hq, hkv, d, rot, dt)
    how.update(interleaved=il)
    w = [1 + 0.25 * torch.randn(d, generator=torch.Generator(device=DEV).manual_seed(i), device=DEV) for i in range(2)]
    base = fp4.qk_norm_rope(q, k, q_weight=w[0], k_weight=w[1], **how)
    col %= d
    w[0][col] = w[1][col] = value
    keep = [c for c in range(d) if c not in (col, partner(col, rot, il))]
    for got, was in zip(fp4.qk_norm_rope(q, k, q_weight=w[0], k_weight=w[1], **how), base):
        assert same(got[..., keep], was[..., keep])
        assert not bool(got[..., col].isfinite().any())


@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("n", [5, 17000])
@pytest.mark.parametrize("rot", [0, 32])
def test_write_into_the_cache(rot, n, il):
    """The serving form's queries, and the tokens that it marks, are those of the norm, then kv4_write."""
    q, k, how = setup(n, 8, 2, 128, rot, torch.bfloat16)
    how.update(eps=None, interleaved=il)
    for x in (q, k):
        x[0, 0, 127], x[n - 1, 1, rot], x[n // 2, 0, 126] = INF, -INF, NAN
    pages = -(-n // 64)
    slots = torch.arange(n, device=DEV)
    a, b = fp4.kv4_cache(pages, 64, 2, 128), fp4.kv4_cache(pages, 64, 2, 128)
    qo, ko = fp4.qk_norm_rope(q, k, **how)
    fp4.kv4_write(a, ko, k, slots)
    got = fp4.kv4_norm_rope(b, q, k, k, slots, **how)
    assert same(got, qo) and same(got[..., rot:], q[..., rot:]) and torch.equal(a.data, b.data)
