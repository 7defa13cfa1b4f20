"""Norm with rotation where a workgroup goes through runs of heads, and its weights' gradients row by row (needs an MI355X).

Runs: bf16 calls of ceil(n / (256 / lanes)) * heads >= 8192 (forward) and 4096 (gradients, cache), fp32 half of that, `lanes` being
d / 8 rounded up to a power of two; the sizes here reach them, with a last run of fewer heads and a last workgroup of
fewer tokens, and gradients of more items than workgroups.

Tolerances, with u = 2^-24: values as in test_gpu_rope.py (16 u of the terms' magnitudes for queries, 1.01 u for keys, 80 u r (H + |x r| D)
for gradients, then the type's rounding).  A weight's gradient: each term g x r is within 17 u (g 4u, x r 12u, the product u), and it takes part in at
most one addition for each row that its lane group goes through, 8 for the exchanges and the waves, then one for each 64th row of
partial sums and 64 more.  At most 1024 workgroups share ceil(n / (256 / lanes)) * heads rows of lane groups about evenly, in whole runs of
4: below that number / 500 + 8 rows a lane group.
"""
import pytest
import torch

import quantized_linear_layers_fp4_amd as fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
DTS = dict(argvalues=[torch.bfloat16, torch.float32], ids=["bf16", "fp32"])


def lanes(d):
    return 4 if d <= 32 else 8 if d <= 64 else 16 if d <= 128 else 32


def setup(n, hq, hkv, d, rot, dt):
    g = torch.Generator(device=DEV).manual_seed(n + hq)
    x = torch.randn(n, hq + 2 * hkv, d, generator=g, device=DEV).to(dt)
    dq, dk = (torch.randn(n, h, d, generator=g, device=DEV).to(dt) for h in (hq, hkv))
    w = [(1 + 0.5 * torch.randn(d, generator=g, device=DEV)).to(dt) for _ in range(2)]
    pos = torch.randint(0, 3001, (n,), generator=g, device=DEV).int()
    pos[::11] = -1
    return x, dq, dk, w, fp4.rope_table(3001, rot), pos


def turned(y, tab, pos, il, sign, absolute=False):
    """y in 64 bits with its first columns turned; or of magnitudes, added."""
    rot = tab.shape[1]
    c, s = (t[:, None] for t in tab[pos.clamp(min=0).long()].double().chunk(2, 1))
    i = torch.arange(rot // 2, device=DEV)
    p, q = (2 * i, 2 * i + 1) if il else (i, i + rot // 2)
    out = y.clone()
    a, b = y[..., p], y[..., q]
    if absolute:
        out[..., p], out[..., q] = a * c.abs() + b * s.abs(), b * c.abs() + a * s.abs()
    else:
        out[..., p], out[..., q] = a * c - sign * b * s, b * c + sign * a * s
    out[pos < 0] = 0
    return out


def reference(x, dy, w, tab, pos, il, eps):
    x, dy, w = x.double(), dy.double(), w.double()
    r = (x.square().mean(2, keepdim=True) + eps).rsqrt()
    y, ym = turned(x * r * w, tab, pos, il, 1), turned((x * r * w).abs(), tab, pos, il, 1, True)
    g, G = turned(dy, tab, pos, il, -1), turned(dy.abs(), tab, pos, il, -1, True)
    xr = x * r
    h, H = g * w, G * w.abs()
    r = torch.where((pos < 0)[:, None, None], 0, r)
    dx = r * (h - xr * (h * xr).mean(2, keepdim=True))
    dxm = r * (H + xr.abs() * (H * xr.abs()).mean(2, keepdim=True))
    return y, ym, dx, dxm, (g * xr).sum((0, 1)), (G * xr.abs()).sum((0, 1))


def close(got, want, tol):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("dt", **DTS)
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,rot", [
    (3, 8189, 11, 32, 32), (32773, 7, 1, 64, 32), (17, 4500, 5, 128, 128), (16389, 9, 3, 80, 16), (8201, 5, 3, 256, 240),
    (2100, 9, 3, 64, 64), (1300, 8, 2, 128, 128)])
def test_runs_of_heads(n, hq, hkv, d, rot, il, dt):
    x, dq, dk, w, tab, pos = setup(n, hq, hkv, d, rot, dt)
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    how = dict(table=tab, positions=pos, q_weight=w[0], k_weight=w[1], eps=1e-6, interleaved=il)
    outs = fp4.qk_norm_rope(q, k, **how)
    grads = fp4.qk_norm_rope_backward(dq, dk, q, k, **how)
    half = torch.finfo(dt).eps / 2 * (1 + 2.0 ** -8)
    groups = -(-n // (256 // lanes(d))) * (hq + hkv)
    chain = groups / 500 + 8 + 8 + 16 + 64
    for i, (a, dy) in enumerate(((q, dq), (k, dk))):
        y, ym, dx, dxm, dw, dwm = reference(a, dy, w[i], tab, pos, il, 1e-6)
        close(outs[i], y, y.abs() * half + (16 if i == 0 else 1.01) * U * ym + 1e-37)
        close(grads[i], dx, dx.abs() * half + 80 * U * dxm + 1e-37)
        close(grads[2 + i], dw, (chain + 17) * U * dwm + 1e-37)


@pytest.mark.parametrize("dt", **DTS)
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d", [(1, 3, 1, 64), (33, 5, 2, 128), (3, 8189, 11, 32), (17, 4500, 5, 128), (32773, 7, 1, 64), (2100, 9, 3, 64),
                                        (8201, 5, 3, 256)])
def test_weights_gradients_of_one_row(n, hq, hkv, d, il, dt):
    """A gradient in one row: the weight's is that row's, once, whichever it is, and no other row gets one."""
    x, _, _, w, tab, _ = setup(n, hq, hkv, d, 32, dt)
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    pos = (torch.arange(n, device=DEV) % 3001).int()
    how = dict(table=tab, positions=pos, q_weight=w[0], k_weight=w[1], eps=1e-6, interleaved=il)
    for t, hf in ((n - 1, 1.0), (0, 0.0), (n - 1, 0.0), (n // 2, 0.5), (max(n - 2, 0), 0.75), (n // 3, 1.0)):
        dq, dk = torch.zeros(n, hq, d, device=DEV, dtype=dt), torch.zeros(n, hkv, d, device=DEV, dtype=dt)
        at = [int(hf * (h - 1)) for h in (hq, hkv)]
        for dy, h in ((dq, at[0]), (dk, at[1])):
            dy[t, h] = torch.randn(d, generator=torch.Generator(device=DEV).manual_seed(t + h), device=DEV).to(dt)
        grads = fp4.qk_norm_rope_backward(dq, dk, q, k, **how)
        for i, (a, dy, h) in enumerate(((q, dq, at[0]), (k, dk, at[1]))):
            _, _, dx, dxm, dw, dwm = reference(a[t:t + 1, h:h + 1], dy[t:t + 1, h:h + 1], w[i], tab, pos[t:t + 1], il, 1e-6)
            close(grads[2 + i], dw, 17 * U * dwm + 1e-37)
            row = grads[i][t:t + 1, h:h + 1]
            close(row, dx, dx.abs() * torch.finfo(dt).eps / 2 * (1 + 2.0 ** -8) + 80 * U * dxm + 1e-37)
            assert int(grads[i].count_nonzero()) == int(row.count_nonzero())


@pytest.mark.parametrize("dt", **DTS)
@pytest.mark.parametrize("n,hq,hkv,d", [(3, 8189, 11, 64), (8201, 7, 3, 128), (16389, 6, 5, 64)])
def test_runs_into_the_cache(n, hq, hkv, d, dt):
    """The write into the cache by runs of heads is the norm, then kv4_write, bit for bit."""
    x, _, _, w, tab, pos = setup(n, hq, hkv, d, 48, dt)
    q, k, v = x.split([hq, hkv, hkv], 1)
    pages = -(-n // 32) + 1
    slots = torch.randperm(pages * 32, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))[:n]
    a, b = fp4.kv4_cache(pages, 32, hkv, d), fp4.kv4_cache(pages, 32, hkv, d)
    qo, ko = fp4.qk_norm_rope(q, k, tab, pos, *w)
    fp4.kv4_write(a, ko, v, slots)
    assert torch.equal(fp4.kv4_norm_rope(b, q, k, v, slots, tab, pos, *w), qo) and torch.equal(a.data, b.data)
