"""Page tables kept on the GPU against a list-based model (needs an MI355X).  Everything is whole numbers: equal or wrong."""
import numpy as np
import pytest
import torch

import quantized_linear_layers_fp4_amd as fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731


class Model:
    """The same by lists, one sequence after the other."""

    def __init__(self, b, width, pages, page):
        self.t = np.full((b, width), -1, np.int64)
        self.lens = np.zeros(b, np.int64)
        self.stack = list(range(pages - 1, -1, -1))
        self.b, self.width, self.pages, self.P = b, width, pages, page

    def up(self, n):
        return -(-int(n) // self.P)

    def extend(self, new, n):
        """The largest running sums decide: pages first, then tokens."""
        new = np.maximum(np.asarray(new, np.int64), 0)
        pages = tokens = 0
        height = len(self.stack)
        slots, pos = [-1] * n, [-1] * n
        q_start, got = [0], []
        for i, a in enumerate(new.tolist()):
            fits = self.lens[i] + a <= self.width * self.P
            want = self.up(self.lens[i] + a) - self.up(self.lens[i]) if fits else 0
            pages += want
            fits = fits and (want == 0 or pages <= height)
            tokens += a if fits else 0
            fits = fits and (a == 0 or tokens <= n)
            got.append(a if fits else 0)
            q_start.append(q_start[-1] + got[-1])
        for i, a in enumerate(got):
            for j in range(self.up(self.lens[i]), self.up(self.lens[i] + a)):
                self.t[i, j] = self.stack.pop()
            for j in range(a):
                p = int(self.lens[i]) + j
                e = self.t[i, p // self.P]
                slots[q_start[i] + j] = e * self.P + p % self.P if 0 <= e < self.pages else -1
                pos[q_start[i] + j] = p
            self.lens[i] += a
        return slots, pos, q_start

    def release(self, keep=None, window=0, sinks=0, shared=0):
        back = []
        for i in range(self.b):
            old = int(self.lens[i])
            kept = old if keep is None else min(max(int(keep[i]), 0), old)
            cols = []
            if window:
                last = min(max(kept - window + 1, 0) // self.P, self.up(kept))
                cols += range(max(self.up(sinks), shared), last)
            cols += range(max(self.up(kept), shared), min(self.up(old), self.width))
            for j in cols:
                if 0 <= self.t[i, j] < self.pages:
                    back.append(int(self.t[i, j]))
                self.t[i, j] = -1
            self.lens[i] = kept
        self.stack += back[::-1]

    def check(self, tables):
        n = len(self.stack)
        assert np.array_equal(tables.table.cpu().numpy(), self.t)
        assert np.array_equal(tables.lens.cpu().numpy(), self.lens)
        assert int(tables.count) == n and tables.free[:n].tolist() == self.stack


def both(b, width, pages, page):
    return fp4.kv4_page_tables(b, width, pages, page), Model(b, width, pages, page)


def extend(t, m, new, n):
    slots, pos, q_start = fp4.kv4_extend(t, i32(new), n)
    assert slots.dtype == torch.int64 and pos.dtype == q_start.dtype == torch.int32
    want = m.extend(new, n)
    for got, w in zip((slots, pos, q_start), want):
        assert got.tolist() == w
    m.check(t)


@pytest.mark.parametrize("b,width,page", [(1, 1, 16), (1, 300, 16), (7, 9, 64), (64, 40, 32), (300, 60, 16), (1024, 3, 128),
                                          (2500, 5, 16)])
def test_random_steps(b, width, page):
    """Appending and giving back at random, the stack now and then too small, in one launch and in two."""
    rng = np.random.RandomState(b)
    t, m = both(b, width, max(1, b * width // 2), page)
    for step in range(12):
        most = [3, page, width * page + 9][step % 3]
        new = rng.randint(-1, most + 1, b) * (rng.rand(b) < 0.7)
        total = int(np.maximum(new, 0).sum())
        extend(t, m, new.tolist(), min([total, total + 17, total // 2, 0][step % 4], 200000))
        keep = (m.lens * rng.rand(b)).astype(int) + rng.randint(-2, 3, b)
        args = [dict(), dict(keep=keep), dict(window=page + 5, sinks=3), dict(keep=np.maximum(m.lens - 2, 0), window=1, sinks=page),
                dict(keep=keep, shared=1)][step % 5]
        if "keep" in args and step % 5 == 3:  # the windows of before left pages behind: no deeper than two tokens
            args["window"] = 4
        kw = {k: (i32(np.asarray(v).tolist()) if k == "keep" else v) for k, v in args.items()}
        fp4.kv4_release(t, **kw)
        m.release(**args)
        m.check(t)


@pytest.mark.parametrize("b,n", [(5, 64), (5, 9000), (1500, 64)])
def test_refusals_in_order(b, n):
    """The row's width, the stack and the call's tokens each stop a sequence; those behind that ask for nothing
    more, or fit a page that they have, still get theirs."""
    t, m = both(b, 4, 7, 16)
    extend(t, m, [3, 65, 17, 0, 64] + [0] * (b - 5), n)         # 1 page, too wide, 2 pages, nothing, 4 pages
    extend(t, m, [13, 1, 15, 0, 0] + [1] * (b - 5), n)          # one's own page, no page left, the rest of a page
    fp4.kv4_release(t, keep=i32([0] * b))
    m.release(keep=[0] * b)
    m.check(t)
    extend(t, m, [10, 10, 10, 10, 10] + [0] * (b - 5), 39)      # the fifth's ten tokens pass 39
    extend(t, m, [1, 40, 1, 0, 3] + [2] * (b - 5), 30)          # the second's 40 pass 30, and so do all later ones
    assert int(t.lens[0]) == 11


def test_one_token_a_sequence():
    t, m = both(1300, 2, 1400, 16)
    slots, pos = fp4.kv4_extend(t)
    want = m.extend([1] * 1300, 1300)
    assert slots.tolist() == want[0] and pos.tolist() == want[1]
    new = [i % 3 for i in range(1300)]                           # more than one counts as one
    slots, pos = fp4.kv4_extend(t, i32(new))
    s, p, q = m.extend([min(a, 1) for a in new], 1300)
    assert slots.tolist() == [s[q[i]] if q[i + 1] > q[i] else -1 for i in range(1300)]
    assert pos.tolist() == [p[q[i]] if q[i + 1] > q[i] else -1 for i in range(1300)]
    m.check(t)
    t, m = both(3, 2, 1, 16)                                     # the stack ends: the others get nothing
    slots, pos = fp4.kv4_extend(t)
    assert slots.tolist() == [0, -1, -1] and pos.tolist() == [0, -1, -1] and t.lens.tolist() == [1, 0, 0]


def test_cut_and_append_gives_the_table_again():
    t, m = both(40, 64, 40 * 64, 16)
    extend(t, m, [(i * 37) % 1000 for i in range(40)], 20000)
    before = t.table.clone()
    keep = t.lens // 2
    new = t.lens - keep
    fp4.kv4_release(t, keep=keep)
    fp4.kv4_extend(t, new, 30000)
    assert torch.equal(t.table, before) and torch.equal(t.lens, keep + new)


@pytest.mark.parametrize("b,width", [(3, 8), (600, 64)])
def test_entries_that_are_no_pages(b, width):
    """Garbage in the table or the stack is never given back and never a slot."""
    t, m = both(b, width, 50, 16)
    extend(t, m, [40, 33, 1] + [0] * (b - 3), 200)
    t.table[0, 1], t.table[1, 0] = 50, -7
    m.t[0, 1], m.t[1, 0] = 50, -7
    slots, _, q = fp4.kv4_extend(t, i32([5, 5, 5] + [0] * (b - 3)), 16)
    want = m.extend([5, 5, 5] + [0] * (b - 3), 16)
    assert slots.tolist() == want[0]
    fp4.kv4_release(t, keep=i32([0] * b))
    m.release(keep=[0] * b)
    m.check(t)
    t.free[int(t.count) - 1] = 10 ** 9
    slots, pos, _ = fp4.kv4_extend(t, i32([2, 17, 0] + [0] * (b - 3)), 19)
    assert slots[:2].tolist() == [-1, -1] and pos[:2].tolist() == [0, 1] and int(slots[2:].min()) >= 0
    t.count.fill_(10 ** 6)                                       # a height past the stack is the stack's
    fp4.kv4_extend(t, i32([16, 0, 0] + [0] * (b - 3)), 16)
    assert int(t.count) == 49
    t.count.fill_(-5)
    assert fp4.kv4_extend(t, i32([0, 0, 40] + [0] * (b - 3)), 40)[2].tolist()[3] == 0 and int(t.count) == 0


def test_captured_steps_go_on():
    """A captured append (and give-back) moves on with every replay, on another stream too."""
    t, m = both(6, 20, 100, 16)
    extend(t, m, [5, 0, 31, 16, 100, 7], 200)
    new = i32([1, 1, 1, 1, 1, 1])

    def step():
        a = fp4.kv4_extend(t, new, 8)
        fp4.kv4_release(t, window=40, sinks=16)
        return a
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    m.extend([1] * 6, 8)
    m.release(window=40, sinks=16)
    torch.cuda.synchronize()
    m.check(t)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        slots, pos, q_start = step()
    for i in range(40):
        if i == 20:
            new.copy_(i32([2, 0, 1, 0, 0, 5]))
        g.replay()
        want = m.extend(new.tolist(), 8)
        m.release(window=40, sinks=16)
        torch.cuda.synchronize()
        assert (slots.tolist(), pos.tolist(), q_start.tolist()) == want
        m.check(t)


def test_python_refusals():
    t = fp4.kv4_page_tables(3, 4, 9, 16)
    with pytest.raises(ValueError):
        fp4.kv4_extend(t, None, 3)
    with pytest.raises(ValueError):
        fp4.kv4_extend(t, i32([1, 1]), 3)
    with pytest.raises(ValueError):
        fp4.kv4_extend(t, torch.ones(3, dtype=torch.int64, device=DEV), 3)
    with pytest.raises(ValueError):
        fp4.kv4_extend(t, i32([1, 1, 1]), -1)
    with pytest.raises(ValueError):
        fp4.kv4_extend(t, i32([1, 0, 1, 0, 1, 0])[::2], 3)
    with pytest.raises(ValueError):
        fp4.kv4_release(t, keep=i32([1]))
    for kw in (dict(window=-1), dict(sinks=-1), dict(shared=-1)):
        with pytest.raises(fp4.Fp4Error):
            fp4.kv4_release(t, **kw)
    with pytest.raises(ValueError):
        fp4.KV4Pages(t.table, t.lens[:2], t.free, t.count, 16)
    with pytest.raises(AttributeError):
        t.table = t.table
