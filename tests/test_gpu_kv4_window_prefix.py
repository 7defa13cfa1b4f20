"""Attention over the 4-bit cache with sinks beside a window, and over pages that a batch shares (needs an MI355X).

Against 64-bit references; a score's error is that of d additions (2^-23 each, twice that and a margin of 2^-15 of the magnitudes'
sum) and of the base change, the output adds P's rounding to bf16 (2^-8), the score error as a factor, and its own rounding.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import quantized_linear_layers_fp4_amd as fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def kv(n, h, d, seed):
    g = torch.Generator().manual_seed(seed)
    k, v = torch.randn(n, h, d, generator=g), torch.randn(n, h, d, generator=g)
    k[:, :, ::37] *= 8.0
    return k.bfloat16(), v.bfloat16()


class Case:
    """Sequences in a shuffled paged cache, `shared` first pages in common; page entries may be taken out."""

    def __init__(self, lens, qlens, hq, hkv, d, page, shared=0, width=None, seed=0, tail=0, kmul=1.0):
        g = torch.Generator().manual_seed(seed)
        b = len(lens)
        self.width = width or max(shared, 1, -(-max(lens) // page))
        own = self.width - shared
        self.pages = shared + b * own + 3
        order = torch.randperm(self.pages, generator=g)
        self.table = torch.cat([order[:shared].expand(b, shared), order[shared:shared + b * own].view(b, own)], 1).int().contiguous()
        self.cache = fp4.kv4_cache(self.pages, page, hkv, d)
        k, v = kv(self.pages * page, hkv, d, seed + 1)
        k = k * kmul
        fp4.kv4_write(self.cache, k.to(DEV), v.to(DEV), torch.arange(self.pages * page, device=DEV))
        self.kc, self.vc = (torch.from_numpy(ref.cache_values(f64(x))).to(DEV) for x in (k, v))
        self.lens, self.starts = list(lens), [0]
        for q in qlens:
            self.starts.append(self.starts[-1] + q)
        self.max_q = max(max(qlens), 1)
        self.q = (torch.randn(self.starts[-1] + tail, hq, d, generator=g) * 1.5).bfloat16()
        self.d, self.page, self.shared, self.hkv = d, page, shared, hkv

    def run(self, **kw):
        args = dict(q_start=i32(self.starts), max_q=self.max_q, shared=self.shared, return_lse=True)
        args.update(kw)
        return fp4.kv4_attention(args.pop("q", self.q.to(DEV)), self.cache, args.pop("pages", self.table.to(DEV)),
                                 args.pop("lens", i32(self.lens)), **args)

    def want(self, window=0, sinks=0, scale=None, max_q=None):
        """o, lse and the magnitudes behind them."""
        nq, hq, d = self.q.shape
        q, table = self.q.to(DEV).double(), self.table.to(DEV).long()
        scale = d ** -0.5 if scale is None else scale
        z = lambda *n: torch.zeros(*n, dtype=torch.float64, device=DEV)  # noqa: E731
        o, lse, omag, smag = z(nq, hq, d), z(nq, hq) - np.inf, z(nq, hq, d), z(nq, hq)
        g = hq // self.hkv
        for i, n in enumerate(self.lens):
            t = torch.arange(min(max(n, 0), self.width * self.page), device=DEV)
            pg = table[i, t // self.page]
            pg = torch.where(t < self.shared * self.page, table[0, t // self.page], pg)
            ql = self.starts[i + 1] - self.starts[i]
            m = min(ql, max_q or self.max_q)
            rows = slice(self.starts[i], self.starts[i] + m)
            pos = max(n, 0) - ql + torch.arange(m, device=DEV)
            see = (t <= pos[:, None]) & (pg >= 0) & (pg < self.pages)
            if window:
                see &= (t > pos[:, None] - window) | (t < sinks)
            slot = pg.clamp(0, self.pages - 1) * self.page + t % self.page
            some = see.any(1)
            if m == 0 or t.numel() == 0:
                continue
            for h in range(self.hkv):
                hs = slice(h * g, h * g + g)
                kk, vv, qq = self.kc[slot, h], self.vc[slot, h], q[rows, hs].reshape(-1, d)
                hide = ~see.repeat_interleave(g, 0)
                s = (qq @ kk.t() * scale).masked_fill(hide, -np.inf)
                zz = torch.logsumexp(s, 1)
                p = torch.exp(s - torch.where(zz == -np.inf, torch.zeros_like(zz), zz)[:, None])
                lse[rows, hs] = torch.where(some[:, None], zz.view(m, g), lse[rows, hs])
                o[rows, hs], omag[rows, hs] = (p @ vv).view(m, g, d), (p @ vv.abs()).view(m, g, d)
                smag[rows, hs] = (qq.abs() @ kk.abs().t() * abs(scale)).masked_fill(hide, 0).amax(1).view(m, g)
        return tuple(x.cpu().numpy() for x in (o, lse, omag, smag))

    def check(self, window=0, sinks=0, scale=None, max_q=None, **kw):
        if window or sinks:
            kw.update(window=window, sinks=sinks)
        if max_q:
            kw.update(max_q=max_q)
        o, lse = (f64(x) for x in self.run(scale=scale, **kw))
        want, wl, omag, smag = self.want(window, sinks, scale, max_q)
        ds = smag * (32 * 2.0 ** -20 + self.d * 2.0 ** -23) + 2.0 ** -21
        none = np.isneginf(wl)
        assert np.array_equal(np.isneginf(lse), none) and (o[none] == 0).all()
        with np.errstate(invalid="ignore"):
            err = np.where(none, 0, np.abs(lse - wl))
            assert (err <= np.where(none, 1, ds + 2.0 ** -21 * (1 + np.abs(wl)))).all(), float(np.nanmax(err))
        tol = omag * (2.0 ** -8 + 2 * ds[..., None] + 2.0 ** -16) + np.abs(want) * 2.0 ** -8 + 1e-30
        err = np.abs(o - want)
        assert (err <= tol).all(), float((err / tol).max())


# ----------------------------------------------------------------------------------------- a window with sinks
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("window,sinks", [(1, 1), (33, 4), (50, 64), (100, 31), (64, 500), (2000, 7), (2 ** 31 - 1, 3), (1, 2 ** 31 - 1)])
def test_sinks_of_single_tokens(window, sinks, page, d):
    Case([1, 0, 31, 65, 97, 128, 129, 500, 333], [1] * 9, 8, 2, d, page).check(window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,qlens,hq,hkv,page", [
    ([700, 5, 3, 64, 300, 0], [5, 5, 7, 1, 0, 2], 10, 2, 32), ([200, 333], [200, 100], 8, 2, 16), ([1000, 64, 40], [70, 64, 17], 5, 1, 128),
    ([700], [65], 16, 16, 16), ([500], [300], 2, 1, 32), ([90], [300], 2, 1, 32)])
@pytest.mark.parametrize("window,sinks", [(50, 3), (130, 100), (7, 65)])
def test_sinks_of_chunks(lens, qlens, hq, hkv, page, window, sinks, d):
    Case(lens, qlens, hq, hkv, d, page).check(window, sinks)


@pytest.mark.parametrize("d", [64, 128])
def test_sinks_far_on(d):
    """Long contexts: split along both parts of the axis; many sequences in one split each."""
    Case([20001, 9999], [1, 3], 8, 2, d, 64).check(5000, 100)
    Case([20001], [1], 8, 2, d, 16).check(300, 4)
    Case([3000 - 41 * i for i in range(70)], [1] * 70, 4, 4, d, 32).check(256, 17)


def test_released_pages_between():
    """Tokens between the sinks and the window need no page: entries -1 there change nothing, nor do stale bytes; a released
    sink is masked."""
    for qlens in ([1, 2], [60, 33]):
        c = Case([500, 260], qlens, 4, 2, 128, 32)
        base = c.run(window=100, sinks=33)
        table = c.table.clone()
        table[0, 2:(500 - qlens[0] - 99) // 32] = -1
        table[1, 2:(260 - qlens[1] - 99) // 32] = c.pages + 5
        assert all(torch.equal(x, y) for x, y in zip(c.run(window=100, sinks=33, pages=table.to(DEV)), base))
        c.table[0, 1] = -1
        c.check(100, 33)


def test_sinks_and_nonfinite_tokens():
    """A poisoned sink makes all later rows of its head NaN, a poisoned token between sinks and window none."""
    for qlens in ([1], [50]):
        c = Case([400], qlens, 4, 2, 64, 16)
        base = c.run(window=60, sinks=5)
        bad = torch.full((1, 2, 64), float("nan"), device=DEV)
        bad[:, 1] = 1
        slot = lambda t: torch.tensor([int(c.table[0, t // 16]) * 16 + t % 16], device=DEV)  # noqa: E731
        for t in (5, 200, 400 - qlens[0] - 60):
            fp4.kv4_write(c.cache, bad, bad, slot(t))
        assert all(torch.equal(x, y) for x, y in zip(c.run(window=60, sinks=5), base))
        fp4.kv4_write(c.cache, bad, bad, slot(4))
        o, lse = c.run(window=60, sinks=5)
        assert bool(o[:, :2].isnan().all()) and bool(lse[:, :2].isnan().all()) and bool(o[:, 2:].isfinite().all())


@pytest.mark.parametrize("qlens", [[1, 1, 1], [40, 17, 3]])
def test_sinks_where_the_table_ends(qlens):
    """A table narrower than the lengths: the window may lie past its end, the sinks are still seen."""
    c = Case([1000, 210, 90], qlens, 4, 2, 64, 16, width=6)
    c.check(50, 20)
    c.check(5, 96)


@pytest.mark.parametrize("qlens", [[1, 2], [40, 3], [300, 200]])
def test_lengths_and_windows_of_any_value(qlens):
    """Lengths far past the table and negative ones, windows and sinks of any size: nothing is read outside, and rows see
    what the table holds of what is theirs."""
    for lens in ([2 ** 31 - 1, 2 ** 31 - 1], [2 ** 30, -2 ** 31], [150, 2 ** 31 - 5]):
        c = Case([96, 96], qlens, 8, 2, 64, 32, width=3)
        c.lens = lens
        for window, sinks in ((1, 1), (50, 40), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 40, 3), (2 ** 30, 2 ** 30), (100, 96)):
            c.check(window, sinks)
        c = Case([96, 96], qlens, 8, 2, 64, 32, width=3, shared=2)
        c.lens = lens
        c.check()


def test_sinks_without_a_window_and_a_window_without_sinks():
    c = Case([300, 77], [40, 1], 4, 2, 128, 32)
    base = c.run()
    assert all(torch.equal(x, y) for x, y in zip(c.run(sinks=9), base))
    c.check(0, 9)
    c.check(31, 0)


# --------------------------------------------------------------------------------------------- shared pages
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (15, 3), (32, 1)])
@pytest.mark.parametrize("shared,page", [(1, 16), (3, 16), (4, 32), (3, 128)])
def test_shared_with_single_tokens(shared, page, hq, hkv, d):
    p = shared * page
    Case([p + 1, p, p + 31, p + 500, p + 64, p + 16, 5, 0, p + 33], [1] * 9, hq, hkv, d, page, shared).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,qlens,hq,hkv,page,shared", [
    ([200, 333, 70], [40, 100, 6], 8, 2, 16, 4), ([129, 300], [65, 172], 4, 4, 64, 2), ([1000, 40, 0, 64], [70, 40, 0, 64], 5, 1, 32, 1),
    ([90, 100], [300, 20], 2, 1, 32, 2), ([2000] * 3, [5, 1, 4], 4, 2, 32, 50)])
def test_shared_with_chunks(lens, qlens, hq, hkv, page, shared, d):
    """Chunks behind the shared pages, inside them, and longer than their sequence."""
    Case(lens, qlens, hq, hkv, d, page, shared).check()


@pytest.mark.parametrize("d", [64, 128])
def test_shared_sizes(d):
    """Prefixes in many splits for few and many rows; own tokens in many splits; no own pages at all."""
    Case([9000, 8200], [1, 1], 4, 2, d, 64, shared=128).check()
    Case([4096 + 3 * i for i in range(70)], [1] * 70, 8, 2, d, 32, shared=128).check()
    Case([12000, 500], [1, 2], 4, 2, d, 32, shared=3).check()
    Case([256 - 3 * i for i in range(20)], [1] * 20, 8, 2, d, 64, shared=4).check()
    Case([300, 256, 280], [60, 60, 60], 8, 2, d, 64, shared=4, width=4).check()


def parts(c):
    nq, hq, d = c.q.shape
    return fp4.lib().fp4_kv4_attention_shared_parts(nq, len(c.lens), c.max_q, hq, c.hkv, d, c.page, c.width, c.shared)


@pytest.mark.parametrize("b,t,hq,hkv,d,page,shared,own", [
    (8, 1, 8, 8, 128, 64, 256, 100), (30, 1, 8, 8, 64, 32, 256, 60), (16, 1, 16, 8, 128, 16, 512, 60), (64, 1, 32, 8, 128, 64, 64, 100),
    (70, 1, 8, 4, 64, 32, 200, 300), (32, 1, 8, 8, 64, 16, 301, 200), (5, 1, 8, 8, 128, 64, 512, 30), (40, 1, 24, 8, 64, 32, 512, 3000),
    (24, 40, 8, 8, 64, 64, 128, 100), (16, 40, 16, 4, 128, 32, 513, 1000), (64, 5, 12, 4, 64, 64, 256, 50), (64, 8, 32, 8, 128, 128, 16, 20)])
def test_shared_in_two_parts(b, t, hq, hkv, d, page, shared, own):
    """Sizes at which the shared bytes are read once: few and many rows of either part, splits joined and taken in;
    sequences that end inside the shared pages or hold nothing, and unlike numbers of queries."""
    p = shared * page
    lens = [p + t + own * (i * 7 % b) // b for i in range(b)]
    c = Case(lens, [t - i * 3 % t for i in range(b)], hq, hkv, d, page, shared, seed=b)
    assert parts(c) == 2
    c.check()
    c.lens[1], c.lens[2], c.lens[3], c.lens[b - 1] = p - page - 3, 0, p, 7
    c.check()
    c.table[:, 1], c.table[0, shared - 1], c.table[b // 2, shared] = -1, c.pages, -5
    c.check(scale=-0.05)


def test_shared_is_row_0s():
    """The other rows' first entries are not those that count; results are the plain call's within the roundings."""
    for qlens in ([1] * 5, [30, 1, 64, 5, 17]):
        c = Case([333, 290, 400, 260, 300], qlens, 8, 2, 128, 32, shared=8)
        plain = c.run(shared=0)
        o, lse = c.run()
        table = c.table.clone()
        table[1:, :8] = torch.tensor([-1, 2 ** 31 - 1, 0, -2 ** 31])[:, None]
        got = c.run(pages=table.to(DEV))
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
        assert float((o.float() - plain[0].float()).abs().max()) <= 2.0 ** -6 * float(plain[0].float().abs().max())
        assert torch.allclose(lse, plain[1], atol=1e-4)


def test_shared_rows_of_no_sequence():
    """A padded batch: rows before, between (past max_q) and behind the sequences get zeros and lse -inf."""
    for qlens, mq, b in (([3, 1, 6], 3, 3), ([70, 30, 50], 40, 3), ([2, 1, 3], 2, 60), ([30, 1, 17], 20, 48)):
        c = Case(([200, 180, 170] if b == 3 else [8200, 8260, 8230]) * (b // 3), qlens * (b // 3), 8, 4, 64, 16,
                 shared=5 if b == 3 else 512, tail=9)
        assert parts(c) == (1 if b == 3 else 2)
        c.check(max_q=mq)
        starts = i32([s + 4 for s in c.starts])
        o, lse = c.run(q_start=starts, max_q=max(qlens), q=torch.cat([c.q[-4:], c.q[:-4]]).to(DEV))
        want = c.run(max_q=max(qlens))
        n = c.starts[-1]
        assert torch.equal(o[4:4 + n], want[0][:n]) and torch.equal(lse[4:4 + n], want[1][:n])
        assert float(o[:4].abs().sum()) == 0 and float(o[4 + n:].abs().sum()) == 0
        assert bool((lse[:4] == -float("inf")).all()) and bool((lse[4 + n:] == -float("inf")).all())


def test_shared_bad_pages_and_nonfinite_tokens():
    for qlens, pre in (([1, 2], 4), ([50, 64], 4), ([1, 2] * 16, 400), ([30, 20] * 24, 300)):
        c = Case([32 * pre + 172, 32 * pre + 94] * (len(qlens) // 2), qlens, 4 if pre == 4 else 16, 2 if pre == 4 else 4, 128, 32,
                 shared=pre)
        assert parts(c) == (1 if pre == 4 else 2)
        c.table[:, 1], c.table[1, pre + 1] = -1, c.pages
        c.check()
        bad = torch.full((1, c.hkv, 128), float("inf"), device=DEV)
        bad[:, :c.hkv // 2] = 1
        fp4.kv4_write(c.cache, bad, bad, torch.tensor([int(c.table[0, 0]) * 32 + 7], device=DEV))
        o, _ = c.run()
        half = o.shape[1] // 2
        assert bool(o[:, half:].isnan().all()) and bool(o[:, :half].isfinite().all())


@pytest.mark.parametrize("qlens", [[1, 1], [40, 70]])
def test_shared_scales_and_strides(qlens):
    c = Case([150, 333], qlens, 6, 2, 64, 16, shared=6)
    c.check(scale=-0.07)
    c.check(scale=0.5)
    big = Case([150, 333], qlens, 6, 2, 64, 16, shared=6, kmul=40.0)
    big.check()
    n = c.starts[-1]
    wide = torch.zeros(n, 10 * 64 + 1, dtype=torch.bfloat16, device=DEV)
    wide[:, 1:1 + 384] = c.q.to(DEV).view(n, -1)
    assert torch.equal(c.run(q=wide[:, 1:1 + 384].view(n, 6, 64))[0], c.run()[0])
    if qlens == [1, 1]:
        got = fp4.kv4_attention(c.q.to(DEV), c.cache, c.table.to(DEV), i32(c.lens), shared=6)
        assert torch.equal(got, c.run()[0])


def test_workspaces_are_enough():
    """The stated bytes suffice (nothing behind them is written), for splits of either part."""
    for lens, qlens, shared, page in (([5000, 4000], [1, 1], 60, 32), ([700] * 30, [3] * 30, 20, 32), ([9000], [2], 1, 64),
                                      ([400, 333], [100, 90], 3, 64), ([8200 + 9 * i for i in range(40)], [1] * 40, 128, 64),
                                      ([5200 + 30 * i for i in range(40)], [5] * 40, 80, 64)):
        c = Case(lens, qlens, 32 if len(lens) == 40 else 8, 8 if len(lens) == 40 else 2, 64, page, shared=shared)
        assert parts(c) == (2 if len(lens) == 40 else 1)
        n = fp4.kv4_attention_workspace(c.q.to(DEV), c.cache, c.table.to(DEV), c.max_q, shared).numel()
        ws = torch.full((n + 4096,), 77, dtype=torch.uint8, device=DEV)
        got = c.run(ws=ws[:n])
        assert bool((ws[n:] == 77).all()) and torch.equal(got[0], c.run()[0])
        if n > 16:
            with pytest.raises(fp4.Fp4Error):
                c.run(ws=ws[:n - 16])


def test_repeated_streamed_and_captured():
    """Replays with other lengths (shorter than the shared pages too), each against the eager call; two graphs on one
    workspace, one after the other."""
    b, sh = 48, 64
    c = Case([4500, 4196, 4100] * 16, [1] * b, 32, 8, 128, 64, shared=sh)
    assert parts(c) == 2
    q, table, lens = c.q.to(DEV), c.table.to(DEV), i32(c.lens)
    ws = max((fp4.kv4_attention_workspace(q, c.cache, table, shared=n) for n in (0, sh)), key=len)
    calls = [lambda: fp4.kv4_attention(q, c.cache, table, lens, return_lse=True, ws=ws, shared=sh),
             lambda: fp4.kv4_attention(q, c.cache, table, lens, return_lse=True, ws=ws, window=100, sinks=20)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        first = [f() for f in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f, a in zip(calls, first):
        assert all(torch.equal(x, y) for x, y in zip(f(), a))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for new in ([4500, 4196, 4100], [3, 0, 4096], [4097, 1, 4500]):
        lens.copy_(i32(new * 16))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for f, got in zip(calls, outs):
            assert all(torch.equal(x, y) for x, y in zip(f(), got))


def test_refusals():
    c = Case([10], [1], 4, 2, 64, 16, shared=1, width=2)
    for kw in (dict(sinks=-1), dict(shared=-1), dict(window=5)):
        with pytest.raises(ValueError):
            c.run(**kw)
    with pytest.raises(fp4.Fp4Error):
        c.run(shared=3)
    with pytest.raises(fp4.Fp4Error):
        c.run(shared=0, window=-1)
    assert fp4.kv4_attention(c.q[:0].to(DEV), c.cache, c.table[:0].to(DEV), i32([]), shared=1).shape == (0, 4, 64)
    o, lse = fp4.kv4_attention(c.q.to(DEV), c.cache, c.table[:0].to(DEV), i32([]), q_start=i32([0]), shared=1, return_lse=True)
    assert float(o.abs().sum()) == 0 and bool((lse == -float("inf")).all())
