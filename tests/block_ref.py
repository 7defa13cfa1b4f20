"""64-bit references of the block-scaled E4M3 operands, the 4-bit cache and its attention (numpy,
from the definitions; nothing here is shared with the package)."""
import numpy as np

E4M3 = np.array([c * 2.0 ** -9 if c < 8 else (1 + (c % 8) / 8) * 2.0 ** (c // 8 - 7) for c in range(127)])
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6.0])


def exponent(amax, limit):
    """Smallest e >= -127 with amax <= limit * 2^e (-127 for 0)."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, -127)
    pos = amax > 0
    g = np.floor(np.log2(np.where(pos, amax, 1.0) / limit)).astype(int)
    for d in (2, 1, 0, -1):
        e = np.where(pos & (amax <= limit * np.exp2(g + d)), g + d, e)
    return np.maximum(e, -127)


def nearest(x, grid):
    """Nearest grid value, ties to the even index, saturating, sign kept."""
    a = np.abs(x)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = np.searchsorted(mid, a, "left"), np.searchsorted(mid, a, "right")
    return np.copysign(grid[np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))], x)


def blocks(x, rows, cols, limit=448.0, grid=E4M3):
    """x (2-D, float64) after quantization with one scale per rows x cols block."""
    R, C = x.shape
    p = np.zeros((-(-R // rows) * rows, -(-C // cols) * cols))
    p[:R, :C] = x
    b = p.reshape(p.shape[0] // rows, rows, p.shape[1] // cols, cols)
    bad = ~np.isfinite(b).all(axis=(1, 3), keepdims=True)
    s = np.exp2(exponent(np.where(bad, 0, np.abs(b).max(axis=(1, 3), keepdims=True)), limit).astype(np.float64))
    with np.errstate(invalid="ignore"):
        q = np.where(bad, np.nan, nearest(np.where(bad, 0, b) / s, grid) * s)
    return q.reshape(p.shape)[:R, :C]


def cache_values(x):
    """x (n, heads, d) as the 4-bit cache holds it."""
    n, h, d = x.shape
    return blocks(x.reshape(-1, 32), 1, 32, 7.0, E2M1).reshape(n, h, d)


def attention(q, k, v, lens, starts, window, scale):
    """o, lse and the sum of |terms| behind each of them; k, v: per sequence (tokens, hkv, d)."""
    nq, hq, d = q.shape
    o, lse = np.zeros(q.shape), np.full((nq, hq), -np.inf)
    omag, smag = np.zeros(q.shape), np.zeros((nq, hq))
    for i, n in enumerate(lens):
        ql = starts[i + 1] - starts[i]
        for j in range(ql):
            pos = n - ql + j
            lo, hi = max(0, pos - window + 1) if window else 0, min(pos + 1, k[i].shape[0])
            if hi <= lo:
                continue
            for h in range(hq):
                g = h // (hq // k[i].shape[1])
                kk, vv, qq = k[i][lo:hi, g], v[i][lo:hi, g], q[starts[i] + j, h]
                s = kk @ qq * scale
                m = s.max()
                p = np.exp(s - m)
                row = starts[i] + j
                lse[row, h] = m + np.log(p.sum())
                o[row, h] = p @ vv / p.sum()
                omag[row, h] = p @ np.abs(vv) / p.sum()
                smag[row, h] = (np.abs(kk) @ np.abs(qq)).max() * abs(scale)
    return o, lse, omag, smag
