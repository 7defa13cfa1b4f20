"""The 4-bit key/value cache and its attention against 64-bit references (needs an MI355X).

Cache values are compared exactly.  Attention: a score's error is that of d additions (2^-23 each; twice that and
a margin of 2^-15 are allowed, of the magnitudes' sum) and of the base change; the output adds P's rounding to bf16 (2^-8), the score error as a factor, and its own rounding.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import quantized_linear_layers_fp4_amd as fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def kv(n, h, d, seed, dt=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    k, v = torch.randn(n, h, d, generator=g), torch.randn(n, h, d, generator=g)
    k[:, :, ::37] *= 8.0
    v[::3] *= 2.0 ** -9
    return k.to(dt), v.to(dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,h,page", [(1, 1, 16), (17, 3, 16), (33, 8, 64), (260, 5, 128), (40, 2, 1024)])
def test_write_read(n, h, page, d, dt):
    pages = -(-n // page) + 2
    k, v = kv(n, h, d, 1, DT[dt])
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2))[:n].to(DEV)
    c = fp4.kv4_cache(pages, page, h, d)
    fp4.kv4_write(c, k.to(DEV), v.to(DEV), slots)
    for out in (torch.float32, torch.bfloat16):
        a, b = fp4.kv4_read(c, slots, out_dtype=out)
        assert np.array_equal(f64(a), ref.cache_values(f64(k))) and np.array_equal(f64(b), ref.cache_values(f64(v)))
    a, _ = fp4.kv4_read(c, slots.int().flip(0).contiguous())
    assert np.array_equal(f64(a), ref.cache_values(f64(k))[::-1])
    other = torch.tensor([s for s in range(pages * page) if s not in set(slots.tolist())], device=DEV)
    assert float(fp4.kv4_read(c, other)[0].abs().sum()) == 0  # nothing else was touched


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("start", [0, 1, 4, 7])
def test_long_write_read(start, d):
    """A prompt long enough for four tokens a lane: runs of slots that begin anywhere, gaps, repeats out of
    the cache, a NaN, and an odd end."""
    n, h, page = 8195, 2 if d == 128 else 4, 32
    pages = 300
    k, v = kv(n, h, d, 5)
    k[40, 0, 3], v[4097, 1, 9] = float("nan"), float("inf")
    slots = torch.arange(n) + start
    slots[1000:1013] += 2 ** 40
    slots[2001] = -5
    slots[3000:3004] = torch.tensor([9503, 9502, 9501, 9500])
    c = fp4.kv4_cache(pages, page, h, d)
    for s in (slots, slots.clamp(max=2 ** 31 - 1).int()):
        c.data.zero_()
        fp4.kv4_write(c, k.to(DEV), v.to(DEV), s.to(DEV))
        a, b = (f64(t) for t in fp4.kv4_read(c, s.to(DEV), out_dtype=torch.float32))
        wk, wv = (ref.cache_values(np.where(np.isfinite(f64(t)), f64(t), 0)) for t in (k, v))
        gone = (slots < 0) | (slots >= pages * page)
        for got, want in ((a, wk), (b, wv)):
            want[40, 0], want[4097, 1], want[gone.numpy()] = np.nan, np.nan, 0
            assert np.array_equal(got, want, equal_nan=True)
        left = fp4.kv4_read(c, torch.tensor([x for x in range(pages * page) if x not in set(slots.tolist())], device=DEV))
        assert float(left[0].abs().sum()) == 0 and float(left[1].abs().sum()) == 0


def test_write_borders_strides_and_bad_slots():
    d = 64
    k = torch.zeros(8, 2, d)
    k[0, 0, :4] = torch.tensor([7.0, 6.5, 0.25, -0.75])
    k[1, 0, 0], k[1, 0, 1] = 7.01, -5.0
    k[2, 0, 0] = 1e-45
    k[3, 0, 40] = -1e37
    k[4, 1] = torch.linspace(-6, 6, d)
    v = torch.randn(8, 2, d)
    c = fp4.kv4_cache(2, 16, 2, d)
    slots = torch.tensor([3, -1, 31, 32, 0, 5, 1 << 40, 9], device=DEV)
    wide = torch.zeros(8, 3 * 2 * d + 2)
    wide[:, 1:1 + 2 * d], wide[:, 1 + 4 * d:1 + 6 * d] = k.view(8, -1), v.view(8, -1)
    wide = wide.to(DEV)  # the fused projection's output: q | k | v rows, from an odd element on
    fp4.kv4_write(c, wide[:, 1:1 + 2 * d].view(8, 2, d), wide[:, 1 + 4 * d:1 + 6 * d].view(8, 2, d), slots)
    a, b = fp4.kv4_read(c, slots, out_dtype=torch.float32)
    ok = [0, 2, 4, 5, 7]
    wk, wv = ref.cache_values(f64(k)), ref.cache_values(f64(v))
    wk[[1, 3, 6]], wv[[1, 3, 6]] = 0, 0
    assert np.array_equal(f64(a), wk) and np.array_equal(f64(b), wv) and ok
    assert int(fp4.kv4_read(c, torch.arange(32, device=DEV))[1].abs().sum(dim=(1, 2)).ne(0).sum()) == 5


def test_write_nonfinite():
    k, v = kv(6, 2, 128, 3)
    k[1, 0, 5], v[2, 1, 100], k[4, 1, 0] = float("nan"), float("inf"), float("-inf")
    c = fp4.kv4_cache(1, 16, 2, 128)
    s = torch.arange(6, device=DEV)
    fp4.kv4_write(c, k.to(DEV), v.to(DEV), s)
    a, b = (f64(t) for t in fp4.kv4_read(c, s))
    bad = np.zeros((6, 2), bool)
    bad[[1, 2, 4], [0, 1, 1]] = True
    fin = lambda t: np.where(np.isfinite(f64(t)), f64(t), 0)  # noqa: E731
    for got, src in ((a, k), (b, v)):
        assert np.isnan(got[bad]).all() and np.array_equal(got[~bad], ref.cache_values(fin(src))[~bad])


class Case:
    """Sequences of given lengths and query counts in a shuffled paged cache."""

    def __init__(self, lens, qlens, hq, hkv, d, page, seed=0, width=None, kmul=1.0):
        g = torch.Generator().manual_seed(seed)
        b = len(lens)
        self.width = width or max(1, -(-max(lens) // page))
        self.pages = b * self.width + 3
        self.table = torch.randperm(self.pages, generator=g)[:b * self.width].view(b, self.width).int()
        self.cache = fp4.kv4_cache(self.pages, page, hkv, d)
        self.k, self.v = [], []
        for i, n in enumerate(lens):
            k, v = kv(max(n, 1), hkv, d, seed + 10 + i)
            k = k * kmul
            t = torch.arange(n)
            fp4.kv4_write(self.cache, k[:n].to(DEV), v[:n].to(DEV),
                          (self.table[i, (t // page)].long() * page + t % page).to(DEV))
            self.k.append(ref.cache_values(f64(k))[:n])
            self.v.append(ref.cache_values(f64(v))[:n])
        self.lens, self.starts = lens, [0]
        for q in qlens:
            self.starts.append(self.starts[-1] + q)
        self.max_q = max(max(qlens), 1)
        self.q = (torch.randn(self.starts[-1], hq, d, generator=g) * 1.5).bfloat16()
        self.d, self.page = d, page

    def run(self, window=0, **kw):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        args = dict(q_start=i32(self.starts), max_q=self.max_q, window=window, return_lse=True)
        args.update(kw)
        return fp4.kv4_attention(args.pop("q", self.q.to(DEV)), self.cache, args.pop("pages", self.table.to(DEV)),
                                 args.pop("lens", i32(self.lens)), **args)

    def check(self, window=0, **kw):
        o, lse = self.run(window, **kw)
        scale = kw.get("scale") or self.d ** -0.5
        want, wl, omag, smag = ref.attention(f64(self.q), self.k, self.v, self.lens, self.starts, window, scale)
        ds = smag * (32 * 2.0 ** -20 + self.d * 2.0 ** -23) + 2.0 ** -21  # of a score
        none = np.isneginf(wl)
        o, lse = f64(o), f64(lse)
        assert np.array_equal(np.isneginf(lse), none) and (o[none] == 0).all()
        with np.errstate(invalid="ignore"):
            err = np.where(none, 0, np.abs(lse - wl))
            assert (err <= np.where(none, 1, ds + 2.0 ** -21 * (1 + np.abs(wl)))).all(), float(err.max())
        tol = omag * (2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -16) + np.abs(want) * 2.0 ** -8 + 1e-30
        err = np.abs(o - want)
        assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 2), (15, 3), (32, 1)])
def test_single_tokens(hq, hkv, page, d):
    Case([1, 0, 31, 32, 33, 127, 128, 129, 500], [1] * 9, hq, hkv, d, page).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 1, 33, 200])
def test_windows_and_drafts(window, d):
    """Several queries a sequence, more queries than tokens (rows that see nothing), none at all."""
    Case([700, 5, 3, 64, 300, 0], [5, 5, 7, 1, 0, 2], 10, 2, d, 32).check(window)


@pytest.mark.parametrize("lens,qlens,hq,hkv,page", [
    ([200, 333], [200, 100], 8, 2, 16), ([129], [129], 4, 4, 64), ([1000, 64, 40], [70, 64, 17], 5, 1, 128),
    ([513], [65], 32, 32, 16), ([90], [300], 2, 1, 32)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 50])
def test_chunks(lens, qlens, hq, hkv, page, d, window):
    Case(lens, qlens, hq, hkv, d, page).check(window)


@pytest.mark.parametrize("d", [64, 128])
def test_long_split(d):
    Case([20001, 9999], [1, 3], 8, 2, d, 64).check()
    Case([20001], [1], 8, 2, d, 64).check(window=5000)


def test_scale_and_large_scores():
    """Scores of hundreds: one token takes all the weight; and a scale of zero: the mean."""
    Case([300, 77], [1, 1], 4, 2, 128, 16, kmul=40.0).check()
    c = Case([300], [2], 4, 2, 64, 16)
    o, lse = c.run(scale=0.0)
    for j in range(2):
        mean = c.v[0][:299 + j].mean(0)
        assert np.abs(f64(o)[j].reshape(2, 2, 64) - mean[:, None]).max() <= 2.0 ** -8 * (np.abs(c.v[0]).mean(0).max() * 2)
        assert np.abs(f64(lse)[j] - np.log(299 + j)).max() < 1e-5


@pytest.mark.parametrize("qlens", [[1, 1], [40, 100]])
def test_nonfinite_and_stale_tokens(qlens):
    """A poisoned token makes the rows that see it NaN and no other; tokens past the length or before the
    window are not read into any row, whatever they hold."""
    lens, page = [150, 260], 32
    c = Case(lens, qlens, 4, 2, 128, page, width=9)
    base = c.run(window=120)
    bad = torch.full((1, 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    bad[:, 1] = 1.0
    slot = lambda i, t: torch.tensor([int(c.table[i, t // page]) * page + t % page], device=DEV)  # noqa: E731
    for i, n in enumerate(lens):
        fp4.kv4_write(c.cache, bad, bad, slot(i, n))                             # past the length
        if n - qlens[i] >= 120:                                                  # before every window
            fp4.kv4_write(c.cache, bad, bad, slot(i, n - qlens[i] - 120))
    o, lse = c.run(window=120)
    assert torch.equal(o, base[0]) and torch.equal(lse, base[1])
    t = lens[1] - 1 - qlens[1] // 2
    fp4.kv4_write(c.cache, bad, bad, slot(1, t))
    o, lse = (f64(x) for x in c.run(window=120))
    pos = np.arange(c.starts[2]) - c.starts[1] + lens[1] - qlens[1]
    sees = (np.arange(c.starts[2]) >= c.starts[1]) & (pos >= t) & (pos < t + 120)
    assert np.isnan(o[sees][:, :2]).all() and np.isnan(lse[sees][:, :2]).all()
    rest = np.isfinite(o).all(axis=2)
    assert rest[~sees].all() and rest[:, 2:].reshape(len(sees), -1)[:, :0].all()
    assert np.array_equal(o[~sees], f64(base[0])[~sees])


def test_bad_pages_are_masked():
    """Page indices outside the cache hide their tokens; the others are as before."""
    for qlens in ([1, 1], [60, 60]):
        c = Case([160, 128], qlens, 4, 2, 128, 32)
        table = c.table.clone()
        table[0, 1], table[0, 3], table[1, 0] = -1, c.pages, 2 ** 31 - 1
        o, lse = c.run(pages=table.to(DEV))
        keep = [np.r_[0:32, 64:96, 128:160], np.r_[32:128]]
        for i in range(2):
            for j in range(qlens[i]):
                pos = c.lens[i] - qlens[i] + j
                see = keep[i][keep[i] <= pos]
                w, wl, mag, _ = ref.attention(f64(c.q)[[c.starts[i] + j]], [c.k[i][see]], [c.v[i][see]], [len(see)],
                                              [0, 1], 0, 128 ** -0.5)
                row = c.starts[i] + j
                assert np.abs(f64(o)[row] - w[0]).max() <= 2.0 ** -6 * mag.max()
                assert np.abs(f64(lse)[row] - wl[0]).max() <= 1e-3


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_largest_finite_values(dt):
    """Values next to the type's largest read back finite, and as tokens that a row does not see they
    leave it as it was."""
    big = torch.finfo(DT[dt]).max
    for qlens in ([3], [50]):
        c = Case([90], qlens, 4, 2, 128, 32, width=4)
        base = c.run(window=40)
        x = torch.full((2, 2, 128), big, dtype=DT[dt])
        x[1] = -x[1]
        slots = torch.tensor([int(c.table[0, 2]) * 32 + 27, int(c.table[0, 0]) * 32], device=DEV)  # tokens 91 and 0
        fp4.kv4_write(c.cache, x.to(DEV), x.to(DEV), slots)
        for t in fp4.kv4_read(c.cache, slots, out_dtype=torch.float32):
            assert np.array_equal(f64(t), np.copysign(3 * 2.0 ** 126, f64(x)))
        o, lse = c.run(window=40)
        rows = slice(1, None) if qlens == [50] else slice(0, None)  # of 50, the first query's window ends at token 1
        assert torch.equal(o[rows], base[0][rows]) and torch.equal(lse[rows], base[1][rows])


@pytest.mark.parametrize("qlens", [[2, 1], [30, 41]])
@pytest.mark.parametrize("d", [64, 128])
def test_negative_scale(qlens, d):
    Case([150, 333], qlens, 6, 2, d, 16).check(scale=-0.07)


def test_more_queries_than_stated():
    """A sequence with more queries than max_q: the first max_q are computed, nothing else is written."""
    for qlens, mq in (([9, 2], 3), ([80, 40], 40)):
        c = Case([200, 120], qlens, 4, 2, 64, 16)
        want = c.run()
        ws = torch.zeros(fp4.kv4_attention_workspace(c.q.to(DEV), c.cache, c.table.to(DEV), mq).numel() + 65536,
                         dtype=torch.uint8, device=DEV)
        n = ws.numel() - 65536
        o, lse = c.run(max_q=mq, ws=ws[:n])
        rows = torch.cat([torch.arange(mq), torch.arange(c.starts[1], c.starts[1] + min(mq, qlens[1]))])
        assert torch.allclose(o[rows].float(), want[0][rows].float(), atol=2.0 ** -5, rtol=2.0 ** -6)
        assert torch.allclose(lse[rows], want[1][rows], atol=1e-4)
        assert int(ws[n:].max()) == 0


def test_q_strides_and_defaults():
    """Queries inside the fused projection's rows; no q_start; a wider table; no lse."""
    c = Case([100, 3, 64], [1, 1, 1], 8, 2, 64, 16)
    o, lse = c.run()
    wide = torch.zeros(3, 12 * 64 + 1, dtype=torch.bfloat16, device=DEV)
    wide[:, 1:1 + 512] = c.q.to(DEV).view(3, -1)
    table = torch.full((3, c.width + 5), -7, dtype=torch.int32, device=DEV)
    table[:, :c.width] = c.table.to(DEV)
    got = c.run(q=wide[:, 1:1 + 512].view(3, 8, 64), pages=table[:, :c.width], q_start=None, max_q=1, return_lse=False)
    assert torch.equal(got, o)


def test_repeated_streamed_and_captured():
    c = Case([3000, 777], [1, 1], 8, 2, 128, 64)
    ws = fp4.kv4_attention_workspace(c.q.to(DEV), c.cache, c.table.to(DEV), c.max_q)
    o, lse = c.run(ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, lse2 = c.run()
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    q, table, lens = c.q.to(DEV), c.table.to(DEV), torch.tensor(c.lens, dtype=torch.int32, device=DEV)
    call = lambda: fp4.kv4_attention(q, c.cache, table, lens, return_lse=True, ws=ws)  # noqa: E731
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        og, lg = call()
    for n in (3000, 1, 2500):
        lens[0] = n
        g.replay()
        torch.cuda.synchronize()
        want = call()
        assert torch.equal(og, want[0]) and torch.equal(lg, want[1])


def test_refusals():
    c = Case([10], [1], 4, 2, 64, 16)
    q, t, n = c.q.to(DEV), c.table.to(DEV), torch.tensor([10], dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        fp4.kv4_attention(q.float(), c.cache, t, n)
    for args in ((q[:, :3], t, n), (q[..., :32], t, n), (q, t.long(), n), (q, t, n.long()), (torch.cat([q, q]), t, n)):
        with pytest.raises(ValueError):
            fp4.kv4_attention(args[0], c.cache, args[1], args[2])
    k = torch.zeros(3, 2, 64, device=DEV)
    with pytest.raises(ValueError):
        fp4.kv4_write(c.cache, k[:, :1], k, torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(TypeError):
        fp4.kv4_write(c.cache, k, k.bfloat16(), torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(TypeError):
        fp4.kv4_write(c.cache, k, k, torch.zeros(3, device=DEV))
    e = torch.zeros(0, dtype=torch.int64, device=DEV)
    fp4.kv4_write(c.cache, k[:0], k[:0], e)
    assert fp4.kv4_read(c.cache, e)[0].shape == (0, 2, 64)
    assert fp4.kv4_attention(q[:0], c.cache, t[:0], n[:0]).shape == (0, 4, 64)
