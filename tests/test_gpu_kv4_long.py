"""The 4-bit cache's attention where every kernel runs several tiles a workgroup (needs an MI355X).

Sizes are chosen by the plan's rules (rows a head, (sequence, head)s, tokens), so that the second buffers, the
running maxima and the joins all take part.  A score is off by the sum's d additions (2^-23 each, of the magnitudes;
twice that and a margin of 2^-15 are allowed) and the base change; a sum over n tokens by n additions of 2^-23 more;
the output adds P's rounding to bf16 (2^-8), the score's error as a factor on both sums, and its own rounding.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import quantized_linear_layers_fp4_amd as fp4
from test_gpu_kv4 import DEV, Case, f64

pytestmark = pytest.mark.gpu


def put(c, i, t, k, v):
    """Token t of sequence i becomes (k, v) (heads x d), in the cache and in the case's own copy."""
    slot = torch.tensor([int(c.table[i, t // c.page]) * c.page + t % c.page], device=DEV)
    fp4.kv4_write(c.cache, k[None].to(DEV), v[None].to(DEV), slot)
    bad = ~np.isfinite(f64(k)).all(1) | ~np.isfinite(f64(v)).all(1)
    for store, x in ((c.k, k), (c.v, v)):
        val = ref.cache_values(np.where(np.isfinite(f64(x)), f64(x), 0)[None])[0]
        val[bad] = np.nan
        store[i][t] = val


def expected(c, window, scale, hidden=None):
    """o, lse and the magnitudes behind them in 64 bits; hidden[i]: tokens whose page is none of the cache's."""
    nq, hq, d = c.q.shape
    q = f64(c.q)
    o, lse = np.zeros(q.shape), np.full((nq, hq), -np.inf)
    omag, smag = np.zeros(q.shape), np.zeros((nq, hq))
    for i, n in enumerate(c.lens):
        r0, ql = c.starts[i], c.starts[i + 1] - c.starts[i]
        hkv = c.k[i].shape[1]
        g = hq // hkv
        pos, tok = n - ql + np.arange(ql)[:, None], np.arange(n)[None]
        see = (tok <= pos) & ((tok > pos - window) if window else True)
        if hidden and i in hidden:
            see = see & ~np.isin(tok, hidden[i])
        if n == 0 or not ql:
            continue
        for h in range(hkv):
            qq = q[r0:r0 + ql, h * g:(h + 1) * g].reshape(ql * g, d)
            kk, vv = c.k[i][:, h], c.v[i][:, h]
            sr = np.repeat(see, g, 0)
            with np.errstate(invalid="ignore"):
                s = np.where(sr, qq @ kk.T * scale, -np.inf)
                m = s.max(1, keepdims=True)
                p = np.exp(s - np.where(np.isneginf(m), 0, m))
                l = p.sum(1, keepdims=True)
                vz = np.where(np.isfinite(vv), vv, 0)
                out = np.where(l == 0, 0, p @ vz / np.where(l == 0, 1, l))
                mag = np.where(l == 0, 0, p @ np.abs(vz) / np.where(l == 0, 1, l))
                ls = np.where(l == 0, -np.inf, m + np.log(np.where(l == 0, 1, l)))
                sm = np.where(sr, np.abs(qq) @ np.abs(kk).T, 0).max(1)
            rows, heads = slice(r0, r0 + ql), slice(h * g, (h + 1) * g)
            o[rows, heads], omag[rows, heads] = out.reshape(ql, g, d), mag.reshape(ql, g, d)
            lse[rows, heads], smag[rows, heads] = ls.reshape(ql, g), sm.reshape(ql, g) * abs(scale)
    return o, lse, omag, smag


def check(c, window=0, scale=None, hidden=None, **kw):
    scale = c.d ** -0.5 if scale is None else scale
    o, lse = (f64(t) for t in c.run(window, scale=scale, **kw))
    want, wl, omag, smag = expected(c, window, scale, hidden)
    n = max(c.lens)
    nan, none = np.isnan(wl), np.isneginf(wl)
    assert np.array_equal(np.isneginf(lse), none) and (o[none] == 0).all()
    assert np.isnan(lse[nan]).all() and np.isnan(o[nan]).all()
    ok = ~nan & ~none
    assert np.isfinite(o[ok]).all() and np.isfinite(lse[ok]).all()
    ds = smag[ok] * (32 * 2.0 ** -20 + c.d * 2.0 ** -23) + 2.0 ** -21
    err = np.abs(lse[ok] - wl[ok])
    assert (err <= ds + 2.0 ** -21 * (1 + np.abs(wl[ok])) + n * 2.0 ** -23).all(), float(err.max())
    tol = omag[ok] * (2.0 ** -8 + 2 * ds[:, None] + 2.0 ** -16 + n * 2.0 ** -22) + np.abs(want[ok]) * 2.0 ** -8 + 1e-30
    err = np.abs(o[ok] - want[ok])
    assert (err <= tol).all(), float((err / tol).max())


# lens, queries a sequence, query heads, key/value heads, page
PATHS = {
    # one launch of sixteen waves, several tiles a wave
    "wide": ([3001, 2900, 2048, 1537, 33] + [1200] * 11, 1, 16, 8, 64),
    "wide_page16": ([1000, 517, 1024, 0], 1, 10, 10, 16),
    # four waves, split, six tiles a wave at most
    "split": ([3000, 2999, 2500, 1, 129] + [777] * 10, 1, 20, 20, 32),
    "split_page16": ([2100, 1800] + [400] * 13, 2, 20, 20, 16),
    # four waves, one workgroup a (sequence, head)
    "one": ([700, 513, 641, 2, 31] + [300] * 27, 1, 32, 32, 128),
    # two splits of many rows, joined a group of lanes to a row
    "join_rows": ([1500, 1499, 1000, 770] + [769] * 12, 1, 512, 32, 64),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", PATHS)
def test_decode_of_several_tiles(name, d):
    lens, t, hq, hkv, page = PATHS[name]
    c = Case(lens, [t] * len(lens), hq, hkv, d, page)
    for i, n in enumerate(lens[:3]):  # the maximum moves in the last and in a middle tile
        for at in (n - 1, n // 2):
            if 0 <= at < n:
                g = torch.Generator().manual_seed(at)
                put(c, i, at, (torch.randn(hkv, d, generator=g) * 6).bfloat16(), torch.randn(hkv, d, generator=g).bfloat16())
    check(c)
    check(c, window=600)


# rows a head over 32, so the many-rows kernel: lens, queries, query heads, key/value heads, page
ROWS = {
    # one workgroup a row tile, five and fewer tiles of 64 tokens; 40 and 320 rows a head
    "unsplit": ([300, 299, 256, 65, 64, 40, 200, 129], 40, 64, 64, 16),
    "unsplit_wide": ([300, 257, 193, 64, 32, 128, 129, 320], 40, 256, 32, 32),
    # three tiles a split, row tiles of 128 and of 256
    "split": ([1300, 1215, 700, 90], 40, 16, 16, 64),
    "split_wide": ([1400, 1399], 70, 64, 16, 128),
    # four splits of many rows, joined a group of lanes to a row
    "join_rows": ([800, 799, 513, 100], 100, 32, 32, 16),
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", ROWS)
def test_chunks_of_several_tiles(name, d):
    lens, t, hq, hkv, page = ROWS[name]
    c = Case(lens, [min(t, n) for n in lens], hq, hkv, d, page)
    for i, n in enumerate(lens[:3]):
        for at in (n - min(t, n), n // 2):
            g = torch.Generator().manual_seed(at)
            put(c, i, at, (torch.randn(hkv, d, generator=g) * 6).bfloat16(), torch.randn(hkv, d, generator=g).bfloat16())
    check(c)
    check(c, window=150)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,t,hq,hkv,page", [
    ([3000] * 4, 1, 16, 8, 64), ([2500] * 15, 1, 20, 20, 16), ([1290, 1300], 50, 16, 16, 32), ([320] * 8, 40, 64, 64, 16),
    ([1400, 1300], 70, 64, 16, 64)])
def test_poisoned_tokens_and_bad_pages_in_later_tiles(lens, t, hq, hkv, page, d):
    """Hidden pages and a token with a NaN in one head, tiles apart: rows that see it are NaN in that head's
    queries and finite in the others', and hidden tokens count nowhere."""
    c = Case(lens, [t] * len(lens), hq, hkv, d, page)
    table, hidden = c.table.clone(), {}
    for i, n in enumerate(lens):
        pages = [p for p in (1, n // page // 2, n // page - 2) if 0 < p < n // page]
        for j, p in enumerate(pages):
            table[i, p] = (-1, c.pages, 2 ** 31 - 1)[j % 3]
        hidden[i] = np.concatenate([np.arange(p * page, (p + 1) * page) for p in pages])
    bad = torch.ones(hkv, d, dtype=torch.bfloat16)
    bad[1, 3] = float("nan")
    at = [x for x in range(lens[0] - 20, lens[0]) if x not in hidden[0]][0]
    put(c, 0, at, bad, torch.ones(hkv, d, dtype=torch.bfloat16))
    check(c, hidden=hidden, pages=table.to(DEV))
    check(c, window=200, hidden=hidden, pages=table.to(DEV))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("t,window", [(4, 0), (40, 0), (40, 70), (300, 0), (300, 70)])
def test_zero_scale_is_the_mean(t, window, d):
    """All visible tokens weigh the same, in either kernel, with hidden pages and a sequence shorter than its queries."""
    c = Case([400, 33], [t, min(t, 40)], 4, 2, d, 16)
    check(c, window, scale=0.0)
    check(c, window, scale=-0.0)
    table = c.table.clone()
    table[0, 3] = -1
    check(c, window, scale=0.0, hidden={0: np.arange(48, 64)}, pages=table.to(DEV))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("qlens,mq", [([9, 2, 30], 3), ([80, 40, 1], 40), ([300, 5, 0], 70)])
def test_queries_of_no_computed_row(qlens, mq, d):
    """Queries past max_q, before the first offset and after the last are zeros and -inf, whatever the memory held."""
    c = Case([200, 120, 500], qlens, 8, 2, d, 16)
    front, back = 7, 11
    q = torch.cat([c.q[:1].expand(front, -1, -1), c.q, c.q[:1].expand(back, -1, -1)]).contiguous().to(DEV)
    starts = torch.tensor(c.starts, dtype=torch.int32, device=DEV) + front
    want, wl = c.run(max_q=max(qlens))
    computed = torch.zeros(q.shape[0], dtype=torch.bool, device=DEV)
    rows = torch.cat([c.starts[i] + torch.arange(min(n, mq)) for i, n in enumerate(qlens)]).to(DEV)
    computed[rows + front] = True
    for _ in range(2):
        held = [torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device=DEV)]
        del held  # the outputs come from this memory
        o, lse = c.run(q=q, q_start=starts, max_q=mq)
        assert (o[~computed] == 0).all() and torch.isneginf(lse[~computed]).all()
        assert torch.allclose(o[rows + front].float(), want[rows].float(), atol=2.0 ** -5, rtol=2.0 ** -6)
        assert torch.allclose(lse[rows + front], wl[rows], atol=1e-4)
    o = c.run(q=q, q_start=starts, max_q=mq, return_lse=False)
    assert (o[~computed] == 0).all()


def test_max_q_not_given():
    """With offsets and no bound on a sequence's queries all of them are computed; without offsets there is one."""
    c = Case([130, 50, 9], [60, 3, 2], 4, 2, 64, 16)
    check(c, max_q=None)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q = c.q[:3].to(DEV)
    assert torch.equal(fp4.kv4_attention(q, c.cache, c.table.to(DEV), i32(130, 50, 9)),
                       fp4.kv4_attention(q, c.cache, c.table.to(DEV), i32(130, 50, 9), q_start=i32(0, 1, 2, 3), max_q=1))


def test_no_sequences():
    """Queries of no sequence at all: zeros and -inf."""
    c = Case([10], [1], 4, 2, 64, 16)
    held = [torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((5, 4), 7.0, device=DEV)]
    del held
    e = torch.zeros(1, dtype=torch.int32, device=DEV)
    o, lse = fp4.kv4_attention(torch.ones(5, 4, 64, dtype=torch.bfloat16, device=DEV), c.cache, c.table[:0].to(DEV), e[:0],
                               q_start=e, return_lse=True)
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 + 7, 2 ** 30, 1200])
@pytest.mark.parametrize("lens,qlens", [([2, 1500, 0, 7], [7, 2, 5, 8]), ([2, 1500, 40, 5], [40, 50, 90, 60])])
def test_largest_windows(lens, qlens, window, d):
    """A window of any size, with sequences of more queries than tokens: their later queries see tokens."""
    c = Case(lens, qlens, 8, 4, d, 32)
    check(c, window)
    if window > 1500:
        for got, want in zip(c.run(window), c.run(0)):
            assert torch.allclose(got.float(), want.float(), atol=2.0 ** -5, rtol=2.0 ** -6)


@pytest.mark.parametrize("t", [3, 40])
def test_lengths_and_offsets_out_of_range(t):
    """A negative length is an empty sequence, and offsets count as the nearest query: the sequences beside them are as
    they were."""
    c = Case([200, 90, 33], [t, t, t], 8, 2, 64, 16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    want, wl = c.run()
    for n in (-1, -2 ** 31):
        o, lse = c.run(lens=i32([200, n, 33]))
        assert torch.equal(o[:t], want[:t]) and torch.equal(o[2 * t:], want[2 * t:])
        assert (o[t:2 * t] == 0).all() and torch.isneginf(lse[t:2 * t]).all()
    for lo, hi in ((-2 ** 31, 2 ** 31 - 1), (-7, 3 * t + 5)):
        o, lse = c.run(q_start=i32([lo, t, 2 * t, hi]))
        assert torch.equal(o, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [40, 16384])
def test_scales_under_which_every_code_is_finite(n, dt):
    """Groups up to the type's largest value: the exponent stops at 125, so that no scale byte of the cache makes an
    infinity of any code, and the group's other values are as near as that scale allows."""
    h, d, page = 2, 128, 32
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn(n, h, d, generator=g), torch.randn(n, h, d, generator=g)
    tops = torch.tensor([1.0, 2.0 ** 60, 2.0 ** 124, 2.0 ** 125, 2.0 ** 126, 2.0 ** 127 * 1.5, torch.finfo(dt).max])
    for x, s in ((k, 0), (v, 3)):
        x *= (tops[(torch.arange(n) + s) % 7] / 8)[:, None, None]
        x[torch.arange(n), :, (torch.arange(n) * 5) % d] = tops[(torch.arange(n) + s) % 7][:, None]
    k[5, 1, 2] = float("nan")
    k, v = k.to(dt), v.to(dt)
    c = fp4.kv4_cache(-(-n // page), page, h, d)
    slots = torch.arange(n, device=DEV)
    fp4.kv4_write(c, k.to(DEV), v.to(DEV), slots)
    region = c.data.view(-1, page * (d + d // 16)).cpu()
    kc, vc = page * d // 2, page * d // 32  # the bytes of a head's codes and of its scales
    ks, vs = region[:, kc:kc + vc], region[:, 2 * kc + vc:]
    assert int(vs.max()) == 252 and set(ks[ks > 252].tolist()) == {255}
    for got, x in zip(fp4.kv4_read(c, slots, out_dtype=torch.float32), (k, v)):
        y = np.where(np.isfinite(f64(x)), f64(x), 0).reshape(-1, 32)
        e = np.minimum(ref.exponent(np.abs(y).max(1, keepdims=True), 7.0), 125)
        want = (ref.nearest(y * np.exp2(-e.astype(float)), ref.E2M1) * np.exp2(e.astype(float))).reshape(n, h, d)
        want[5, 1] = np.nan
        assert np.array_equal(f64(got), want, equal_nan=True)


def test_page_tables_of_one_column_and_of_one_row():
    """A single column needs no stride along it, and a single row none between rows."""
    c = Case([100, 3, 64], [1, 1, 1], 8, 2, 64, 128)
    want, wl = c.run()
    turned = torch.full((4, 3), -1, dtype=torch.int32, device=DEV)
    turned[0] = c.table[:, 0]
    for table in (turned.t()[:, :1], turned[:1].t(), torch.stack([c.table.to(DEV)[:, 0]] * 5, 1)[:, 2:3]):
        assert table.shape == (3, 1)
        o, lse = c.run(pages=table)
        assert torch.equal(o, want) and torch.equal(lse, wl)
    c = Case([100], [1], 8, 2, 64, 16)
    want, wl = c.run()
    o, lse = c.run(pages=c.table[0].to(DEV).as_strided((1, c.width), (0, 1)))
    assert torch.equal(o, want) and torch.equal(lse, wl)
    for table in (c.table.to(DEV).expand(2, -1), torch.zeros(2, 4, dtype=torch.int32, device=DEV)[:, ::2]):
        with pytest.raises(ValueError):
            c.run(pages=table, lens=torch.ones(2, dtype=torch.int32, device=DEV), q_start=torch.arange(3, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("t,hq", [(1, 8), (6, 8), (40, 8), (70, 32)])
def test_captured_batches_of_changing_sizes(t, hq):
    """One captured call for a batch that fills and empties: offsets, lengths and tables change between the replays, and
    every replay writes every row, those of no sequence too."""
    c = Case([900, 333, 64, 500], [t] * 4, hq, 4, 64, 32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    q, table, lens, starts = c.q.to(DEV), c.table.to(DEV), i32(c.lens), i32(c.starts)
    ws = fp4.kv4_attention_workspace(q, c.cache, table, t)
    call = lambda: fp4.kv4_attention(q, c.cache, table, lens, q_start=starts, max_q=t, window=400, return_lse=True, ws=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        og, lg = call()
    for qlens, ln in (([t] * 4, [900, 333, 64, 500]), ([t, 0, 0, 0], [900, 0, 0, 0]), ([1, t, 1, 0], [77, 333, 1, 0]),
                      ([0] * 4, [0] * 4), ([t] * 4, [500, 333, 10, 499])):
        starts.copy_(i32([0, *np.cumsum(qlens).tolist()]))
        lens.copy_(i32(ln))
        og.fill_(7.0)
        lg.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        want, wl = call()
        n = sum(qlens)
        assert torch.equal(og, want) and torch.equal(lg, wl)
        assert (og[n:] == 0).all() and torch.isneginf(lg[n:]).all() and not (lg[:n] == 7).any()
