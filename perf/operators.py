"""Measured cases of the FP8 block-128 linear layer and of the 4-bit key/value cache.

Four operators, each through the package's public calls:

  linear     Y = X . W with X quantized to E4M3 in blocks of 128 along K and W held in E4M3 with
             one scale per 128 x 128 block (the serving form: W is quantized once).
  step       the training form: W quantized, forward, and the gradients dX and dW, whose operands
             are E4M3 in blocks of 128 along the contraction of each product.
  cache      keys and values quantized to E2M1 in groups of 32 as they are written into the
             paged cache, and the same tokens read back.
  attention  attention of packed queries over the paged 4-bit cache.

Scales are powers of two: a block's exponent is the smallest e with max|x| <= 448 * 2^e (E4M3) or
max|x| <= 7 * 2^e (E2M1), at least -127.  Codes are nearest with ties to even; E2M1 saturates at 6.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token through the gate+up projection of a 7B layer: the serving latency of a
        # projection, all of it the weight's bytes
        dict(name="linear_token", op="linear", M=1, K=4096, N=22016, dtype="bf16"),
        # a few dozen tokens of a decode batch through the 7B down projection
        dict(name="linear_batch", op="linear", M=48, K=11008, N=4096, dtype="bf16"),
        # a prompt of 8192 tokens through the 1.3B qkv projection
        dict(name="linear_prompt", op="linear", M=8192, K=2048, N=6144, dtype="bf16"),
        # one training step of a small layer, fp32, no size a multiple of a block
        dict(name="step_odd", op="step", M=1111, K=777, N=1290, dtype="fp32"),
        # one training step of the 7B qkv projection at 8192 tokens: the largest case
        dict(name="step_layer", op="step", M=8192, K=4096, N=12288, dtype="bf16"),
        # a decode batch writes one token per sequence: the smallest call, launch latency
        dict(name="cache_tokens", op="cache", n=64, hkv=8, d=128, page=16, dtype="bf16"),
        # a prompt of 16384 tokens written in one call, multi-head layout (32 heads)
        dict(name="cache_prompt", op="cache", n=16384, hkv=32, d=128, page=64, dtype="bf16"),
        # one sequence decodes at a short odd context, multi-head: the latency of a single token
        dict(name="attn_one", op="attention", b=1, t=1, hq=32, hkv=32, d=128, page=16, ctx=777, ragged=False,
             window=0),
        # a decode batch with grouped heads at mixed contexts up to 8192: the serving work horse
        dict(name="attn_batch", op="attention", b=64, t=1, hq=32, hkv=8, d=128, page=64, ctx=8192, ragged=True,
             window=0),
        # one sequence decodes at a long context: the split along the tokens
        dict(name="attn_long", op="attention", b=1, t=1, hq=32, hkv=8, d=128, page=128, ctx=131072, ragged=False,
             window=0),
        # a chunk of two prompts over an 8192-token context: many queries, bound by arithmetic
        dict(name="attn_chunk", op="attention", b=2, t=1024, hq=32, hkv=8, d=128, page=64, ctx=8192, ragged=False,
             window=0),
        # a few draft tokens per sequence, small heads, odd group and lengths, sliding window
        dict(name="attn_window", op="attention", b=9, t=5, hq=20, hkv=4, d=64, page=32, ctx=4001, ragged=True,
             window=1000),
    ]


def draw(rng):
    def logint(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["linear", "linear", "step", "cache", "attention", "attention", "attention"])
    if op == "linear":
        M, K, N = logint(1, 8192), logint(128, 11008), logint(128, 22016)
        return dict(op=op, M=min(M, 3 * 8192 * 4096 * 12288 // (K * N)), K=K, N=N,
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "step":
        return dict(op=op, M=logint(64, 8192), K=logint(128, 4096), N=logint(128, 12288),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "cache":
        return dict(op=op, n=logint(1, 16384), hkv=rng.choice([1, 2, 4, 8, 20, 32]), d=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["bf16", "bf16", "fp32"]))
    hkv = rng.choice([1, 2, 4, 8, 32])
    g = 1 if hkv == 32 else rng.choice([1, 3, 4, 5, 8])
    d, page = rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    if rng.random() < 0.6:   # decode: one to a few tokens per sequence
        b, t = logint(1, 64), rng.choice([1, 1, 1, 2, 5])
        ctx = logint(t, max(t, min(131072, 64 * 8192 * 8 // (b * hkv))))
    else:                    # chunks of prompts
        b, t = logint(1, 4), logint(16, 1024)
        ctx = logint(t, 8192)
        if b * t * hkv * g * ctx > 2 * 1024 * 32 * 8192:
            b = 1
    return dict(op=op, b=b, t=t, hq=hkv * g, hkv=hkv, d=d, page=page, ctx=ctx, ragged=rng.random() < 0.5,
                window=rng.choice([0, 0, 0, logint(1, 4096)]))


# ----------------------------------------------------------------------------------- inputs
def _gen(seed, stream):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 16 + stream)
    return g


def _dtype(case):
    return torch.float32 if case.get("dtype") == "fp32" else torch.bfloat16


def _activations(rows, cols, g, dt):
    """Normal values with a few channels thirty times larger, as a transformer's activations."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    ch = torch.randint(0, cols, (max(1, cols // 256),), generator=g, device=DEV)
    x[:, ch] *= 30.0
    return x.to(dt)


def _linear_inputs(case, seed):
    dt = _dtype(case)
    x = _activations(case["M"], case["K"], _gen(seed, 0), dt)
    w = (torch.randn(case["K"], case["N"], generator=_gen(seed, 1), device=DEV) * 0.02).to(dt)
    dy = None
    if case["op"] == "step":
        dy = (torch.randn(case["M"], case["N"], generator=_gen(seed, 2), device=DEV) * 1e-3).to(dt)
    return x, w, dy


def _kv(n, hkv, d, g, dt):
    """Keys with a few large channels per head; values normal."""
    k = torch.randn(n, hkv, d, generator=g, device=DEV)
    ch = torch.randint(0, d, (hkv, 2), generator=g, device=DEV)
    k.scatter_(2, ch.expand(n, hkv, 2), k.gather(2, ch.expand(n, hkv, 2)) * 8.0)
    v = torch.randn(n, hkv, d, generator=g, device=DEV)
    return k.to(dt), v.to(dt)


def _cache_inputs(case, seed):
    n, page = case["n"], case["page"]
    k, v = _kv(n, case["hkv"], case["d"], _gen(seed, 0), _dtype(case))
    pages = 2 * ((n + page - 1) // page) + 1
    # a decode batch lands anywhere; a prompt fills its pages in order, the pages scattered
    if n <= 256:
        slots = torch.randperm(pages * page, generator=_gen(seed, 1), device=DEV)[:n]
    else:
        order = torch.randperm(pages, generator=_gen(seed, 1), device=DEV)
        t = torch.arange(n, device=DEV)
        slots = order[t // page] * page + t % page
    return k, v, slots, pages


def _lengths(case):
    """Cached tokens and query tokens of each sequence; ragged ones spread over (t, ctx] and [1, t]."""
    b, t, ctx = case["b"], case["t"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * b, [t] * b
    return ([ctx - int((ctx - t) * (i * 0.6180339887 % 1.0)) for i in range(b)], [t - i * 3 % t for i in range(b)])


def _attention_inputs(case, seed):
    b, t, page, ctx = case["b"], case["t"], case["page"], case["ctx"]
    g = _gen(seed, 0)
    width = (ctx + page - 1) // page
    lens, qlen = (torch.tensor(x, device=DEV) for x in _lengths(case))
    q_start = torch.zeros(b + 1, dtype=torch.int32, device=DEV)
    q_start[1:] = qlen.cumsum(0)
    table = torch.randperm(b * width, generator=g, device=DEV).view(b, width).int()
    k, v = _kv(b * width * page, case["hkv"], case["d"], _gen(seed, 1), torch.bfloat16)
    nq = int(q_start[-1])
    q = (torch.randn(nq, case["hq"], case["d"], generator=_gen(seed, 2), device=DEV) * 1.5).bfloat16()
    return q, q_start, lens.int(), table, k, v, b * width


# ------------------------------------------------------------------- plain quantization forms
def _times2(x, e):
    """x * 2^e for fp32 x and whole e in [-252, 254], by factors that are exact (pow() need not be)."""
    h = torch.div(e, 2, rounding_mode="floor").int()
    for part in (h, e.int() - h):
        x = x * ((part + 127) << 23).view(torch.float32)
    return x


def _exponent(amax, limit):
    """Smallest e >= -127 with amax <= limit * 2^e."""
    m, x = torch.frexp(amax)
    lm, lx = math.frexp(limit)
    e = (x - lx + (m > lm).int()).clamp(min=-127)
    return torch.where(amax > 0, e, torch.full_like(e, -127))


def _grid(y, mant, emin):
    """Nearest value, ties to even, of a float format with `mant` mantissa bits."""
    _, x = torch.frexp(y)
    step = (x - 1).clamp(min=emin) - mant
    return _times2(torch.round(_times2(y, -step)), step)


def _pad(x, rows, cols):
    r, c = (-x.shape[0]) % rows, (-x.shape[1]) % cols
    return torch.nn.functional.pad(x, (0, c, 0, r)) if r or c else x


def _vector_blocks(x):
    """Values of x (fp32) after E4M3 quantization in blocks of 128 along its last axis."""
    n = x.shape[1]
    y = _pad(x, 1, 128).view(x.shape[0], -1, 128)
    e = _exponent(y.abs().amax(2, keepdim=True), 448.0)
    y = _times2(_grid(_times2(y, -e), 3, -6), e)
    return y.view(x.shape[0], -1)[:, :n]


def _square_blocks(w):
    """Values of w (fp32) over 2^e, and the exponents e of its 128 x 128 blocks."""
    p = _pad(w, 128, 128)
    y = p.view(p.shape[0] // 128, 128, p.shape[1] // 128, 128)
    e = _exponent(y.abs().amax((1, 3), keepdim=True), 448.0)
    y = _grid(_times2(y, -e), 3, -6).view_as(p)[:w.shape[0], :w.shape[1]]
    return y, e


def _square_values(y, e):
    p = _pad(y, 128, 128)
    z = _times2(p.view(p.shape[0] // 128, 128, p.shape[1] // 128, 128), e)
    return z.view_as(p)[:y.shape[0], :y.shape[1]]


def _e4m3_codes(y):
    """Bytes of values on the E4M3 grid."""
    a = y.abs()
    _, x = torch.frexp(a)
    normal = a >= 2.0 ** -6
    ex = torch.where(normal, x - 1, torch.full_like(x, -6))
    frac = _times2(a, 3 - ex).int()            # 8..15 for normals, 0..7 below
    code = torch.where(normal, (ex + 7) * 8 + frac - 8, frac)
    return (code + (torch.signbit(y)).int() * 128).to(torch.uint8)


def _e4m3_table():
    c = torch.arange(256, device=DEV)
    ex, m = (c >> 3) & 15, (c & 7).float()
    v = torch.where(ex == 0, m * 2.0 ** -9, _times2(1 + m / 8, ex - 7))
    return torch.where(c >= 128, -v, v)


def _e2m1_groups(x):
    """Codes (one per byte) and scale bytes of x (.., d) in groups of 32."""
    y = x.float().view(*x.shape[:-1], -1, 32)
    e = _exponent(y.abs().amax(-1, keepdim=True), 7.0)
    y = _times2(y, -e)
    z = _grid(y, 1, 0).abs().clamp(max=6.0)
    code = torch.where(z < 2, z * 2, torch.where(z < 4, z + 2, z / 2 + 4)).int()
    code = code + torch.signbit(y).int() * 8
    return code.view(x.shape).to(torch.uint8), (e + 127).squeeze(-1).to(torch.uint8)


def _e2m1_table():
    v = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(v + [-a for a in v], device=DEV)


def _pack4(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack4(packed, scales, table):
    """fp32 values (.., d) of packed codes (.., d/2) with scale bytes (.., d/32)."""
    c = torch.stack((packed & 15, packed >> 4), -1).view(*packed.shape[:-1], -1).int()
    v = table[c].view(*scales.shape, 32)
    return _times2(v, (scales.int() - 127).unsqueeze(-1)).view(c.shape)


# ---------------------------------------------------------------------------------- prepare
def prepare(case, seed):
    op = case["op"]
    st = dict(case=case)
    if own:
        import quantized_linear_layers_fp4_amd as fp4
        st["fp4"] = fp4
    if op in ("linear", "step"):
        x, w, dy = _linear_inputs(case, seed)
        st["x"] = x
        if op == "step":
            st.update(w=w, dy=dy)
        elif own:
            st["wq"] = fp4.block8_quantize(w, fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)[1]
        else:
            y, e = _square_blocks(w.float())
            st.update(w8=_e4m3_codes(y), we=e, table=_e4m3_table())
    elif op == "cache":
        k, v, slots, pages = _cache_inputs(case, seed)
        st.update(k=k, v=v, slots=slots)
        if own:
            st["cache"] = fp4.kv4_cache(pages, case["page"], case["hkv"], case["d"], device=k.device)
        else:
            rows, d = pages * case["page"], case["d"]
            st["codes"] = torch.zeros(2, rows, case["hkv"], d // 2, dtype=torch.uint8, device=DEV)
            st["scales"] = torch.zeros(2, rows, case["hkv"], d // 32, dtype=torch.uint8, device=DEV)
            st["table"] = _e2m1_table()
    else:
        q, q_start, lens, table, k, v, pages = _attention_inputs(case, seed)
        st.update(q=q, q_start=q_start, lens=lens, pages=table)
        if own:
            st["cache"] = fp4.kv4_cache(pages, case["page"], case["hkv"], case["d"], device=q.device)
            fp4.kv4_write(st["cache"], k, v, torch.arange(k.shape[0], device=DEV))
            st["ws"] = fp4.kv4_attention_workspace(q, st["cache"], table, max_q=case["t"])
        else:
            kc, ks = _e2m1_groups(k)
            vc, vs = _e2m1_groups(v)
            shape = (pages, case["page"], case["hkv"], -1)
            st.update(kc=_pack4(kc).view(shape), ks=ks.view(shape), vc=_pack4(vc).view(shape), vs=vs.view(shape),
                      table=_e2m1_table())
    return st


# -------------------------------------------------------------------------------------- run
def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _own_linear(s):
    return s["fp4"].block8_linear_forward(s["x"], s["wq"])


def _own_step(s):
    fp4 = s["fp4"]
    w_rows, w_cols = fp4.block8_quantize(s["w"], fp4.FP4_BLOCK_SQUARE, rows=True, cols=True)
    y, x_cols = fp4.block8_linear_forward(s["x"], w_cols, for_backward=True)
    dx, dw = fp4.block8_linear_backward(s["dy"], w_rows, x_cols)
    return y, dx, dw


def _own_cache(s):
    fp4 = s["fp4"]
    fp4.kv4_write(s["cache"], s["k"], s["v"], s["slots"])
    return fp4.kv4_read(s["cache"], s["slots"], s["case"]["d"], out_dtype=s["k"].dtype)


def _own_attention(s):
    c = s["case"]
    return s["fp4"].kv4_attention(s["q"], s["cache"], s["pages"], s["lens"], q_start=s["q_start"], max_q=c["t"],
                                  window=c["window"], return_lse=True, ws=s["ws"])


def _plain_linear(s):
    w = _square_values(s["table"][s["w8"].int()], s["we"])
    return (_vector_blocks(s["x"].float()) @ w).to(s["x"].dtype)


def _plain_step(s):
    dt = s["x"].dtype
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    wv = _square_values(*_square_blocks(w))
    y = _vector_blocks(x) @ wv
    dx = _vector_blocks(dy) @ wv.t()
    dw = _vector_blocks(x.t().contiguous()) @ _vector_blocks(dy.t().contiguous()).t()
    return y.to(dt), dx.to(dt), dw.to(dt)


def _plain_cache(s):
    out = []
    for i, x in enumerate((s["k"], s["v"])):
        codes, scales = _e2m1_groups(x)
        s["codes"][i][s["slots"]] = _pack4(codes)
        s["scales"][i][s["slots"]] = scales
        out.append(_unpack4(s["codes"][i][s["slots"]], s["scales"][i][s["slots"]], s["table"]).to(x.dtype))
    return tuple(out)


def _plain_attention(s):
    c = s["case"]
    b, t, hq, hkv, d = c["b"], c["t"], c["hq"], c["hkv"], c["d"]
    g = hq // hkv
    pages = s["pages"].long()

    def gather(codes, scales):                       # (b, hkv, tokens, d)
        x = _unpack4(codes[pages], scales[pages], s["table"])
        return x.flatten(1, 2).transpose(1, 2).contiguous()

    k = gather(s["kc"], s["ks"])
    qs = s["q_start"].long()
    qlen = qs[1:] - qs[:-1]
    j = torch.arange(t, device=DEV)
    row = (qs[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)          # (b, t)
    q = s["q"][row].float().view(b, t, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * t, d)
    sc = (q @ k.transpose(2, 3).contiguous()) * (d ** -0.5)
    pos = (s["lens"].long() - qlen)[:, None] + j                      # (b, t)
    tok = torch.arange(k.shape[2], device=DEV)
    see = tok <= pos[:, :, None]
    if c["window"]:
        see &= tok > pos[:, :, None] - c["window"]
    see = see[:, None, None].expand(b, hkv, g, t, tok.numel()).reshape(sc.shape)
    sc = torch.where(see, sc, torch.full_like(sc, -math.inf))
    m = sc.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(sc - m)
    l = p.sum(3, keepdim=True)
    o = (p @ gather(s["vc"], s["vs"])) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).view(b, hkv, g, t).permute(0, 3, 1, 2).reshape(b, t, hq)
    o = o.view(b, hkv, g, t, d).permute(0, 3, 1, 2, 4).reshape(b, t, hq, d)
    live = j < qlen[:, None]
    return o[live].to(s["q"].dtype), lse[live]


_OWN = dict(linear=_own_linear, step=_own_step, cache=_own_cache, attention=_own_attention)
_PLAIN = dict(linear=_plain_linear, step=_plain_step, cache=_plain_cache, attention=_plain_attention)


# ------------------------------------------------------------------------------------- work
def _pairs(case):
    """Visible (query, token) pairs and the cached tokens that some query sees."""
    win, pairs, tokens = case["window"], 0, 0
    for n, tq in zip(*_lengths(case)):
        see = [min(p + 1, win) if win else p + 1 for p in range(n - tq, n)]
        pairs += sum(see)
        tokens += min(n, win + tq - 1) if win else n
    return pairs, tokens


def work(case):
    op = case["op"]
    if op in ("linear", "step"):
        M, K, N = case["M"], case["K"], case["N"]
        es = 4 if case["dtype"] == "fp32" else 2
        blocks = ((K + 127) // 128) * ((N + 127) // 128)
        if op == "linear":
            return dict(bytes=es * M * K + K * N + blocks + es * M * N, flops=2 * M * N * K)
        return dict(bytes=2 * es * (M * K + K * N + M * N), flops=6 * M * N * K)
    if op == "cache":
        vals = 2 * case["n"] * case["hkv"] * case["d"]
        es = 4 if case["dtype"] == "fp32" else 2
        # values in and out, codes and scales written and read, slots read twice
        return dict(bytes=2 * es * vals + 2 * (vals // 2 + vals // 32) + 16 * case["n"], flops=4 * vals)
    pairs, tokens = _pairs(case)
    nq = sum(_lengths(case)[1])
    per_token = case["hkv"] * (case["d"] + case["d"] // 16)
    return dict(bytes=int(tokens * per_token + nq * case["hq"] * (4 * case["d"] + 4)),
                flops=int(4 * case["d"] * case["hq"] * pairs))


# ------------------------------------------------------------------------------------ exact
def _nearest(y, grid):
    """Nearest grid value by search, ties to the even index, in 64 bits; beyond it, the last."""
    a = y.abs()
    mid = (grid[1:] + grid[:-1]) / 2
    lo = torch.searchsorted(mid, a, right=False)      # number of midpoints below a
    hi = torch.searchsorted(mid, a, right=True)       # number of midpoints at or below a
    idx = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
    return torch.copysign(grid[idx], y)


def _power64(e):
    """2^e in 64 bits, from the bits of its exponent."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale64(amax, limit):
    e = torch.full_like(amax, -127.0)
    pos = amax > 0
    guess = torch.floor(torch.log2(torch.where(pos, amax, torch.ones_like(amax)) / limit))
    for d in (2, 1, 0, -1):                            # the smallest of the four that holds
        ok = amax <= limit * _power64(guess + d)
        e = torch.where(pos & ok, guess + d, e)
    return _power64(e.clamp(min=-127))


def _e4m3_grid():
    c = np.arange(127)
    v = np.where(c < 8, c * 2.0 ** -9, (1 + (c % 8) / 8.0) * 2.0 ** (c // 8 - 7.0))
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _blocks64(x, rows, cols):
    """x (fp64) quantized to E4M3 with one scale per rows x cols block."""
    grid = _e4m3_grid()
    out = torch.empty_like(x)
    for r0 in range(0, x.shape[0], 1024):              # 1024 is whole blocks of 1 and of 128 rows
        xs = x[r0:r0 + 1024]
        r, c = xs.shape
        p = torch.zeros((r + rows - 1) // rows * rows, (c + cols - 1) // cols * cols, dtype=x.dtype, device=DEV)
        p[:r, :c] = xs
        b = p.reshape(p.shape[0] // rows, rows, p.shape[1] // cols, cols)
        s = _scale64(b.abs().amax((1, 3), keepdim=True), 448.0)
        out[r0:r0 + 1024] = (_nearest(b / s, grid) * s).reshape(p.shape)[:r, :c]
    return out


def _groups64(x):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    for i in range(0, x.shape[0], 16384):
        b = x[i:i + 16384].double().reshape(-1, 32)
        s = _scale64(b.abs().amax(1, keepdim=True), 7.0)
        out[i:i + 16384] = (_nearest(b / s, grid) * s).reshape(out[i:i + 16384].shape)
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("linear", "step"):
        x, w, dy = _linear_inputs(case, seed)
        x, wq = x.double(), _blocks64(w.double(), 128, 128)
        y = _blocks64(x, 1, 128) @ wq
        if op == "linear":
            return y
        dy = dy.double()
        dx = _blocks64(dy, 1, 128) @ wq.t()
        return y, dx, _blocks64(x, 128, 1).t() @ _blocks64(dy, 128, 1)
    if op == "cache":
        k, v, _, _ = _cache_inputs(case, seed)
        return _groups64(k), _groups64(v)
    q, q_start, lens, table, k, v, _ = _attention_inputs(case, seed)
    hq, hkv, d, page, win = case["hq"], case["hkv"], case["d"], case["page"], case["window"]
    g = hq // hkv
    k, v = (_groups64(x).view(-1, page, hkv, d) for x in (k, v))
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    starts, ctxs = q_start.tolist(), lens.tolist()
    for i, n in enumerate(ctxs):
        lo, hi = starts[i], starts[i + 1]
        kk = k[table[i].long()].reshape(-1, hkv, d)[:n]
        vv = v[table[i].long()].reshape(-1, hkv, d)[:n]
        pos = n - (hi - lo) + torch.arange(hi - lo, device=DEV)
        tok = torch.arange(n, device=DEV)
        hide = tok[None] > pos[:, None]
        if win:
            hide |= tok[None] <= pos[:, None] - win
        for h in range(hq):
            s = (q[lo:hi, h].double() @ kk[:, h // g].t()) / math.sqrt(d)
            s.masked_fill_(hide, -math.inf)
            z = torch.logsumexp(s, 1)
            lse[lo:hi, h] = z
            p = torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z), z)[:, None])
            out[lo:hi, h] = p @ vv[:, h // g]
    return out, lse
