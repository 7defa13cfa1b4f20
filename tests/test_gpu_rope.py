"""Norm of queries and keys with rotation, its gradients and its write into the 4-bit cache, against 64 bits (needs an MI355X).

Tolerances, with u = 2^-24 and M the sum of the magnitudes of a value's two terms times r:
  queries    the products with the weight (u each), two more and the sum (2u), the row's sum of squares (8 in a chain, 5 by
             pairs, halved by the root: 7u), the root (2u), the last product (u): below 16 u M, then the type's rounding
  keys       rounded to fp32 (u), then to the type
  gradients  with H = |w| times the magnitudes of the rotated gradient and D = sum H |x r| / d: g 4u, h u, x r 12u, the dot
             product (8 + 5 + 1 + 17)u D, the last three operations: below 80 u r (H + |x r| D)
  weights    one addition a row in the worst case: (rows + 100) u times the sum of magnitudes
"""
import numpy as np
import pytest
import torch

import quantized_linear_layers_fp4_amd as fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24


def half(dt):
    return torch.finfo(dt).eps / 2


def f64(t):
    return t.detach().cpu().double().numpy()


def angles(max_pos, rot, base=10000.0, factor=1.0):
    a = np.arange(max_pos)[:, None] / factor * base ** (-2.0 * np.arange(rot // 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1)


def turn(y, cos, sin, il):
    """y (n, h, d) with its first columns turned; cos, sin (n, rot / 2)."""
    rot = 2 * cos.shape[1]
    i = np.arange(rot // 2)
    p, q = (2 * i, 2 * i + 1) if il else (i, i + rot // 2)
    out = y.copy()
    c, s = cos[:, None], sin[:, None]
    out[..., p], out[..., q] = y[..., p] * c - y[..., q] * s, y[..., q] * c + y[..., p] * s
    return out


class Ref:
    def __init__(self, x, w, tab, pos, eps, il):
        self.x, self.w = f64(x), np.ones(x.shape[2]) if w is None else f64(w)
        self.norm, self.il = eps is not None, il
        n = x.shape[0]
        if tab is None:
            self.c = self.s = np.zeros((n, 0))
            self.pad = np.zeros(n, bool)
        else:
            t, p = f64(tab), np.asarray(pos)
            rows = t[np.clip(p, 0, len(t) - 1)]
            rows[p >= len(t)] = np.nan
            self.pad = p < 0
            self.c, self.s = rows[:, :rows.shape[1] // 2], rows[:, rows.shape[1] // 2:]
        with np.errstate(invalid="ignore", divide="ignore"):
            self.r = 1 / np.sqrt((self.x ** 2).mean(2, keepdims=True) + eps) if self.norm else np.ones(self.x.shape[:2] + (1,))

    def forward(self):
        """(y, M)."""
        with np.errstate(invalid="ignore"):
            y = self.x * self.r * self.w
            out, mag = turn(y, self.c, self.s, self.il), turn(np.abs(y), np.abs(self.c), -np.abs(self.s), self.il)
            p = turn(np.abs(y), np.abs(self.c), np.abs(self.s), self.il)
        out[self.pad] = 0
        return out, np.maximum(np.abs(mag), np.abs(p))

    def backward(self, dy):
        """(dx, its bound's magnitude, dw, its magnitudes' sum)."""
        dy = f64(dy)
        g = turn(dy, self.c, -self.s, self.il)
        G = np.maximum(np.abs(turn(np.abs(dy), np.abs(self.c), -np.abs(self.s), self.il)),
                       np.abs(turn(np.abs(dy), np.abs(self.c), np.abs(self.s), self.il)))
        g[self.pad], G[self.pad] = 0, 0
        if not self.norm:
            return g, G, None, None
        xr = self.x * self.r
        xr[self.pad] = 0
        h, H = g * self.w, G * np.abs(self.w)
        r = np.where(self.pad[:, None, None], 0, self.r)
        dx = r * (h - xr * (h * xr).mean(2, keepdims=True))
        return dx, r * (H + np.abs(xr) * (H * np.abs(xr)).mean(2, keepdims=True)), (g * xr).sum((0, 1)), (G * np.abs(xr)).sum((0, 1))


def inputs(n, hq, hkv, d, dt, seed=0, weights=True, odd=True):
    """Views of a fused projection's rows (from an odd element on), weights, gradients like the outputs."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, (hq + 2 * hkv) * d + 3, generator=g)
    x[:, ::29] *= 20.0
    x = x.to(dt).to(DEV)[:, 1 if odd else 0:][:, :(hq + 2 * hkv) * d]
    x = x.unflatten(1, (hq + 2 * hkv, d))
    w = [(1 + torch.randn(d, generator=g)).to(dt).to(DEV) if weights else None for _ in range(2)]
    dq, dk = (torch.randn(n, h, d, generator=g).to(dt).to(DEV) for h in (hq, hkv))
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], w, dq, dk


def close(got, want, tol):
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN in other places"
    with np.errstate(invalid="ignore"):
        bad = np.abs(got - want) > tol
    assert not bad.any(), float((np.abs(got - want) / tol)[bad].max())


def check(q, k, w, dq, dk, tab, pos, eps, il):
    how = dict(table=tab, positions=pos, q_weight=w[0], k_weight=w[1], eps=eps, interleaved=il)
    dt = q.dtype
    p = None if pos is None else pos.cpu().numpy()
    outs = fp4.qk_norm_rope(q, k, **how)
    grads = fp4.qk_norm_rope_backward(dq, dk, q, k, **how)
    for i, (x, wt, dy) in enumerate(((q, w[0], dq), (k, w[1], dk))):
        if x is None:
            assert outs[i] is None and grads[i] is None and grads[2 + i] is None
            continue
        ref = Ref(x, wt, tab, p, eps, il)
        y, mag = ref.forward()
        tiny = 1e-37 if dt == torch.float32 else 1e-38
        close(outs[i], y, np.abs(y) * half(dt) * (1 + 2.0 ** -8) + (16 if i == 0 else 1.01) * U * mag + tiny)
        dx, dmag, dw, wmag = ref.backward(dy)
        close(grads[i], dx, np.abs(dx) * half(dt) * (1 + 2.0 ** -8) + 80 * U * dmag + tiny)
        if wt is None:
            assert grads[2 + i] is None
        else:
            assert grads[2 + i].dtype == torch.float32
            close(grads[2 + i], dw, (x.shape[0] * x.shape[1] + 100) * U * wmag + 1e-37)
    return outs, grads


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,rot", [
    (1, 1, 1, 64, 64), (3, 5, 1, 128, 128), (17, 4, 4, 32, 16), (33, 3, 2, 40, 32), (9, 6, 3, 80, 80), (65, 2, 1, 96, 16),
    (7, 3, 1, 200, 112), (20, 2, 2, 256, 256), (5, 1, 1, 136, 128), (1300, 8, 2, 128, 128), (2100, 9, 3, 64, 32),
    (700, 7, 5, 256, 240)])
def test_sizes(n, hq, hkv, d, rot, il, dt):
    q, k, _, w, dq, dk = inputs(n, hq, hkv, d, DT[dt])
    tab = fp4.rope_table(5000, rot)
    pos = torch.randint(0, 5000, (n,), generator=torch.Generator().manual_seed(n)).int().to(DEV)
    check(q, k, w, dq, dk, tab, pos, 1e-6, il)


@pytest.mark.parametrize("n", [5, 1500])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_parts_left_out(n, dt):
    """No weights, no norm, no rotation, no keys, one weight, weights of the other type."""
    q, k, _, w, dq, dk = inputs(n, 8, 2, 64, DT[dt], seed=3)
    tab, pos = fp4.rope_table(2000, 64), torch.arange(n, device=DEV, dtype=torch.int32)
    check(q, k, (None, None), dq, dk, tab, pos, 1e-5, False)
    check(q, k, (None, None), dq, dk, tab, pos, None, True)
    check(q, k, w, dq, dk, None, None, 1e-5, False)
    check(q, None, (w[0], None), dq, None, tab, pos, 1e-6, False)
    check(q, k, (None, w[1]), dq, dk, tab, pos, 1e-6, False)
    other = torch.float32 if dt == "bf16" else torch.bfloat16
    check(q, k, [x.to(other) for x in w], dq, dk, tab, pos, 1e-6, True)


@pytest.mark.parametrize("n", [40, 3000])
def test_padding_and_far_positions(n):
    """Negative positions: zeros out, nothing to the gradients, whatever the rows hold; positions past the table: NaN in
    the columns that turn."""
    q, k, _, w, dq, dk = inputs(n, 8, 2, 128, torch.bfloat16, seed=5)
    tab = fp4.rope_table(100, 64)
    pos = (torch.arange(n) % 100).int()
    pos[::7] = -1
    pos[3] = -2 ** 31
    base, grads = check(q, k, w, dq, dk, tab, pos.to(DEV), 1e-6, False)
    q2, k2, dq2 = q.clone(), k.clone(), dq.clone()
    q2[::7], k2[7], dq2[14] = float("nan"), float("inf"), float("nan")
    out, g2 = fp4.qk_norm_rope(q2, k2, tab, pos.to(DEV), *w), fp4.qk_norm_rope_backward(dq2, dk, q2, k2, tab, pos.to(DEV), *w)
    assert all(torch.equal(a, b) for a, b in zip(out + g2, base + grads))
    pos[10], pos[20] = 100, 2 ** 31 - 1
    out = fp4.qk_norm_rope(q, k, tab, pos.to(DEV), *w)
    for a, b in zip(out, base):
        for t in (10, 20):
            assert bool(a[t, :, :64].isnan().all()) and torch.equal(a[t, :, 64:], b[t, :, 64:])
        keep = [t for t in range(n) if t not in (10, 20)]
        assert torch.equal(a[keep], b[keep])


@pytest.mark.parametrize("n", [6, 2000])
def test_values_at_the_range_ends(n):
    """fp32 rows whose squares pass fp32's range, zero rows, tiny rows without eps; rows with NaN or infinity are NaN and no
    other is touched."""
    q, k, _, w, dq, dk = inputs(n, 8, 2, 64, torch.float32, seed=7)
    q, k = q.contiguous(), k.contiguous()
    tab, pos = fp4.rope_table(2100, 64), torch.arange(n, device=DEV, dtype=torch.int32)
    q[0] *= 1e30
    q[1] *= 1e-30
    q[2] = 0
    k[3] *= 1e33
    k[4] *= 1e-33
    dq[1] *= 1e-25  # the row's r is 1e30: its gradient stays a number
    dk[4] *= 1e-28
    check(q[3:], k[:3].repeat(2, 1, 1)[:n - 3] if n < 10 else k[3:], w, dq[3:], dk[3:], tab, pos[3:], 1e-6, False)
    check(q, k, w, dq, dk, tab, pos, 1e-6, True)
    q[2] = 1
    check(q, k, w, dq, dk, tab, pos, 0.0, False)
    base = fp4.qk_norm_rope(q, k, tab, pos, *w)
    q[1, 3, 5], k[2, 0, 9] = float("nan"), float("-inf")
    out = fp4.qk_norm_rope(q, k, tab, pos, *w)
    assert bool(out[0][1, 3].isnan().all()) and bool(out[1][2, 0].isnan().all())
    for a, b, at in ((out[0], base[0], (1, 3)), (out[1], base[1], (2, 0))):
        a[at] = b[at]
        assert torch.equal(a, b)


def test_gradients_by_differences():
    """(f(x + e v) - f(x - e v)) / 2e against <grad, v>: with e = 2^-6 of values near 1 the third derivative's part is below
    e^2 and fp32's rounding of f, summed, below 2^-20 of its magnitude over e."""
    torch.manual_seed(0)
    n, hq, hkv, d = 12, 3, 2, 64
    q, k, dq, dk = (torch.randn(n, h, d, device=DEV) for h in (hq, hkv, hq, hkv))
    w = [1 + 0.1 * torch.randn(d, device=DEV) for _ in range(2)]
    tab, pos = fp4.rope_table(64, 64), torch.arange(n, device=DEV, dtype=torch.int32)
    grads = fp4.qk_norm_rope_backward(dq, dk, q, k, tab, pos, *w)

    def f(q, k, wq, wk):
        a, b = fp4.qk_norm_rope(q, k, tab, pos, wq, wk)
        return float((a.double() * dq.double()).sum() + (b.double() * dk.double()).sum())
    args = [q, k, *w]
    for i in range(4):
        v = torch.randn_like(args[i])
        e = 2.0 ** -6
        up, down = ([x + s * e * v if j == i else x for j, x in enumerate(args)] for s in (1, -1))
        got, want = (f(*up) - f(*down)) / (2 * e), float((grads[i].double() * v.double()).sum())
        size = float((grads[i].double() * v.double()).abs().sum())
        assert abs(got - want) <= 4 * e * e * size + 2.0 ** -18 * float(dq.abs().sum() + dk.abs().sum()) / e / 64, (i, got, want)


@pytest.mark.parametrize("n", [7, 2500])
def test_gradients_into_the_projections(n):
    """out: views into the fused projection's gradient; what lies between them stays."""
    hq, hkv, d = 8, 2, 64
    q, k, _, w, dq, dk = inputs(n, hq, hkv, d, torch.bfloat16)
    tab, pos = fp4.rope_table(4096, 32), torch.arange(n, device=DEV, dtype=torch.int32)
    want = fp4.qk_norm_rope_backward(dq, dk, q, k, tab, pos, *w)
    full = torch.full((n, (hq + 2 * hkv) * d + 1), 7.0, dtype=torch.bfloat16, device=DEV)
    v = full[:, 1:].unflatten(1, (hq + 2 * hkv, d))
    got = fp4.qk_norm_rope_backward(dq, dk, q, k, tab, pos, *w, out=(v[:, :hq], v[:, hq:hq + hkv]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((full[:, 0] == 7).all()) and bool((v[:, hq + hkv:] == 7).all()) and got[0].data_ptr() == v.data_ptr()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,rot,page", [(1, 4, 1, 64, 64, 16), (5, 5, 5, 128, 128, 16), (33, 6, 3, 128, 32, 64),
                                                 (100, 8, 2, 64, 16, 32), (3001, 8, 2, 128, 128, 128), (2500, 6, 6, 64, 64, 16)])
def test_write_into_the_cache(n, hq, hkv, d, rot, page, il, dt):
    """The fused write is the norm, then kv4_write, bit for bit; slots of no page are skipped, int32 ones too, and
    rows with a NaN are marked."""
    q, k, v, w, _, _ = inputs(n, hq, hkv, d, DT[dt], seed=n, odd=n != 33)
    k, v = k.clone(), v.clone()
    k[n // 2, 0, 3], v[n // 3, hkv - 1, 9] = float("nan"), float("inf")
    tab, pos = fp4.rope_table(8000, rot), torch.arange(n, device=DEV, dtype=torch.int32) * 2
    if n > 2:
        pos[1] = -1
    pages = -(-n // page) + 2
    g = torch.Generator().manual_seed(1)
    slots = torch.randperm(pages * page, generator=g)[:n] if n < 50 else torch.arange(n) + 3
    if n > 2:
        slots[0], slots[2] = -1, pages * page
    slots = slots.to(DEV)
    a, b = fp4.kv4_cache(pages, page, hkv, d), fp4.kv4_cache(pages, page, hkv, d)
    how = dict(table=tab, positions=pos, q_weight=w[0], k_weight=w[1], interleaved=il)
    qo, ko = fp4.qk_norm_rope(q, k, **how)
    fp4.kv4_write(a, ko, v, slots)
    for s in (slots, slots.int()):
        b.data.zero_()
        assert torch.equal(fp4.kv4_norm_rope(b, q, k, v, s, **how), qo)
        assert torch.equal(a.data, b.data)
    fp4.kv4_write(a, k, v, slots)
    fp4.kv4_norm_rope(b, q, k, v, slots, eps=None)
    assert torch.equal(a.data, b.data)


def test_table():
    for max_pos, rot, base, factor in ((1, 16, 10000.0, 1.0), (70001, 64, 10000.0, 1.0), (131072, 128, 500000.0, 8.0), (300, 240, 1e6, 0.5)):
        t = f64(fp4.rope_table(max_pos, rot, base, factor))
        rows = np.unique(np.r_[0, max_pos - 1, np.arange(0, max_pos, 997)])
        want = angles(max_pos, rot, base, factor)[rows]
        # the angle is known to 4 roundings of 64 bits (a power, two quotients, a product) in both, then one to fp32
        tol = np.abs(want) * U + 8 * 2.0 ** -53 * (rows[:, None] / factor) + 2.0 ** -52
        assert (np.abs(t[rows] - want) <= tol).all()


def test_repeated_streamed_and_captured():
    n = 2048
    q, k, v, w, dq, dk = inputs(n, 8, 2, 128, torch.bfloat16)
    tab, pos = fp4.rope_table(4096, 128), torch.arange(n, device=DEV, dtype=torch.int32)
    c = fp4.kv4_cache(n // 64, 64, 2, 128)
    slots = torch.arange(n, device=DEV)

    def run():
        return (*fp4.qk_norm_rope(q, k, tab, pos, *w), *fp4.qk_norm_rope_backward(dq, dk, q, k, tab, pos, *w),
                fp4.kv4_norm_rope(c, q, k, v, slots, tab, pos, *w))
    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for shift in (0, 5, 1):
        pos.copy_(torch.arange(n, device=DEV) + shift)
        g.replay()
        torch.cuda.synchronize()
        kept = c.data.clone()
        eager = run()
        assert all(torch.equal(a, b) for a, b in zip(eager, got)) and torch.equal(kept, c.data)


def test_refusals():
    q, k, v, w, dq, dk = inputs(4, 2, 1, 64, torch.bfloat16)
    tab, pos = fp4.rope_table(16, 64), torch.arange(4, device=DEV, dtype=torch.int32)
    c, slots = fp4.kv4_cache(2, 16, 1, 64), torch.arange(4, device=DEV)
    assert fp4.qk_norm_rope(q[:0], k[:0], tab, pos[:0])[0].shape == (0, 2, 64)
    assert float(fp4.qk_norm_rope_backward(dq[:0], dk[:0], q[:0], k[:0], tab, pos[:0], *w)[2].abs().sum()) == 0
    for args, kw, err in (
            ((q, k.float(), tab, pos), {}, TypeError), ((q, k, tab), {}, ValueError), ((q, k, tab, pos.long()), {}, ValueError),
            ((q, k, tab.double(), pos), {}, ValueError), ((q, k, tab, pos[:3]), {}, ValueError), ((q, k[:3], tab, pos), {}, ValueError),
            ((q, k[..., :32], tab, pos), {}, ValueError), ((q.transpose(1, 2), k, tab, pos), {}, ValueError), ((q[0], k, tab, pos), {}, ValueError),
            ((q, k, tab[:, :8].contiguous(), pos), {}, ValueError), ((q, k, tab[:, :24].contiguous(), pos), {}, fp4.Fp4Error),
            ((q[..., :16], k[..., :16], tab[:, :16].contiguous(), pos), {}, fp4.Fp4Error), ((q[:, :0], k, tab, pos), {}, ValueError),
            ((q[..., :32], k[..., :32], tab, pos), {}, fp4.Fp4Error), ((q.half(), k.half(), tab, pos), {}, TypeError),
            ((q, k, tab, pos, w[0][:60]), {}, ValueError), ((q, k, tab, pos, w[0], w[1].float()), {}, TypeError),
            ((q, k, tab, pos, w[0]), dict(eps=None), ValueError), ((q, k, tab, pos), dict(eps=-1e-6), ValueError),
            ((q, k, tab, pos), dict(eps=float("nan")), ValueError), ((q, None, tab, pos, None, w[1]), {}, ValueError)):
        with pytest.raises(err):
            fp4.qk_norm_rope(*args, **kw)
    for args, kw in (((dq[:, :1], dk, q, k), {}), ((dq, None, q, k), {}), ((dq, dk, q, None), {}),
                     ((dq, dk, q, k), dict(out=(dq[:3], None)))):
        with pytest.raises(ValueError):
            fp4.qk_norm_rope_backward(*args, tab, pos, **kw)
    with pytest.raises(ValueError):
        fp4.kv4_norm_rope(c, q, k, v[:3], slots, tab, pos)
    with pytest.raises(ValueError):
        fp4.kv4_norm_rope(c, q, q, q, slots, tab, pos)
    with pytest.raises(TypeError):
        fp4.kv4_norm_rope(c, q, k, v, slots.float(), tab, pos)
    with pytest.raises(fp4.Fp4Error):
        fp4.rope_table(10, 24)
