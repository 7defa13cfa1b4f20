"""A batch that answers over one common instruction: two attention layers on the 4-bit cache, all of a step on the GPU.

    python examples/decode_batch.py [--hidden 2048 --heads 16 --kv-heads 4 --batch 16 --prefix 2048 --steps 64]

The first layer sees everything: its sequences share the instruction's pages, whose keys and values are read once for the
whole batch.  The second sees a window and the first few tokens, and gives back the pages that no later token sees.  A
step takes pages for its tokens, projects in FP8, norms and rotates queries and keys while keys and values go to the
cache, attends and projects back; decode steps are one captured HIP graph, which moves the page tables on with every replay.
Prints the time of each part and how far the layers are from fp32 on the values that the caches hold; last a training step
of the projection through the norm and the rotation.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_linear_layers_fp4_amd as fp4  # noqa: E402

EPS = 1e-6


class Layer:
    """FP8 projections, norm of queries and keys, rotation, and attention over a paged 4-bit cache."""

    def __init__(self, hidden, heads, kv_heads, d, batch, max_tokens, window=0, sinks=0, page=32, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.d, self.window, self.sinks, self.shared = heads, kv_heads, d, window, sinks, 0
        rows = heads + 2 * kv_heads
        self.w_qkv = (torch.randn(hidden, rows * d, generator=g, device=device) * hidden ** -0.5).bfloat16()
        self.w_out = (torch.randn(heads * d, hidden, generator=g, device=device) * (heads * d) ** -0.5).bfloat16()
        self.qkv, self.out = (fp4.block8_quantize(w, fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)[1]
                              for w in (self.w_qkv, self.w_out))
        self.q_norm, self.k_norm = (torch.rand(d, generator=g, device=device).add_(0.5).bfloat16() for _ in range(2))
        width = (max_tokens + page - 1) // page
        self.cache = fp4.kv4_cache(batch * width, page, kv_heads, d, device=device)
        self.tables = fp4.kv4_page_tables(batch, width, batch * width, page, device=device)
        self.angles = fp4.rope_table(max_tokens, d, device=device)

    def share(self, tokens: int):
        """Row 0's first tokens, whole pages, become every sequence's."""
        t = self.tables
        self.shared = tokens // t.page
        t.table[1:, :self.shared] = t.table[0, :self.shared]
        t.lens[1:] = tokens

    def __call__(self, x, new, max_q):
        """x: the packed new tokens (n x hidden), new[i] of sequence i."""
        n = x.shape[0]
        slots, pos, q_start = fp4.kv4_extend(self.tables, new, n)
        y = fp4.block8_linear_forward(x, self.qkv).view(n, -1, self.d)
        q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = fp4.kv4_norm_rope(self.cache, q, k, v, slots, self.angles, pos, self.q_norm, self.k_norm, EPS)
        seen = dict(window=self.window, sinks=self.sinks) if self.window else dict(shared=self.shared)
        o = fp4.kv4_attention(q, self.cache, self.tables.table, self.tables.lens, q_start=q_start, max_q=max_q, **seen)
        if self.window:
            fp4.kv4_release(self.tables, window=self.window, sinks=self.sinks, shared=self.shared)
        return fp4.block8_linear_forward(o.view(n, -1), self.out)

    def reference(self, x, seq: int):
        """The last x.shape[0] tokens of sequence seq in fp32, on the values that the weights and the cache stand for."""
        t, page, n = self.tables, self.tables.page, int(self.tables.lens[seq])
        wq, wo = (fp4.block8_dequantize(w).t().contiguous() for w in (self.qkv, self.out))
        tok = torch.arange(n, device=x.device)
        entry = t.table[seq, tok // page].long()
        k, v = fp4.kv4_read(self.cache, entry * page + tok % page, out_dtype=torch.float32)
        m, g = x.shape[0], self.heads // self.kv_heads
        pos = torch.arange(n - m, n, device=x.device)
        q = (x.float() @ wq)[:, :self.heads * self.d].view(m, self.heads, self.d)
        q = q * torch.rsqrt((q * q).mean(-1, keepdim=True) + EPS) * self.q_norm.float()
        cos, sin = self.angles[pos][:, None].chunk(2, -1)
        a, b = q.chunk(2, -1)
        q = torch.cat((a * cos - b * sin, b * cos + a * sin), -1).view(m, self.kv_heads, g, self.d)
        see = (tok[None] <= pos[:, None]) & (entry >= 0)
        if self.window:
            see &= (tok[None] > pos[:, None] - self.window) | (tok[None] < self.sinks)
        o = torch.empty_like(q)
        for h in range(self.kv_heads):
            s = (q[:, h].reshape(m * g, self.d) @ k[:, h].t().contiguous()).view(m, g, n) * self.d ** -0.5
            p = torch.softmax(s.masked_fill(~see[:, None], float("-inf")), 2)
            o[:, h] = (p.view(m * g, n) @ v[:, h].contiguous()).view(m, g, self.d)
        return o.view(m, -1) @ wo

    def train_step(self, x, pos, dq, dk, dv):
        """(dx, dw, dq_norm, dk_norm) of the projection followed by norm and rotation, from the gradients of q, k and v."""
        n, rows, cols = x.shape[0], *fp4.block8_quantize(self.w_qkv, fp4.FP4_BLOCK_SQUARE, rows=True, cols=True)
        y, xt = fp4.block8_linear_forward(x, cols, for_backward=True)
        q, k, _ = y.view(n, -1, self.d).split([self.heads, self.kv_heads, self.kv_heads], 1)
        how = dict(table=self.angles, positions=pos, q_weight=self.q_norm, k_weight=self.k_norm, eps=EPS)
        fp4.qk_norm_rope(q, k, **how)
        dy = torch.empty_like(y).view(n, -1, self.d)
        gq, gk, gv = dy.split([self.heads, self.kv_heads, self.kv_heads], 1)
        _, _, wq, wk = fp4.qk_norm_rope_backward(dq, dk, q, k, **how, out=(gq, gk))
        gv.copy_(dv)
        return (*fp4.block8_linear_backward(dy.view(n, -1), rows, xt), wq, wk)

    def train_reference(self, x, pos, dq, dk, dv):
        """The same by autograd in fp32 on the unquantized weights."""
        x, w, wq, wk = (t.float().requires_grad_() for t in (x, self.w_qkv, self.q_norm, self.k_norm))
        y = (x @ w).view(x.shape[0], -1, self.d)
        cos, sin = self.angles[pos.long()][:, None].chunk(2, -1)
        outs = []
        for t, n in zip(y.split([self.heads, self.kv_heads, self.kv_heads], 1)[:2], (wq, wk)):
            a, b = (t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS) * n).chunk(2, -1)
            outs.append(torch.cat((a * cos - b * sin, b * cos + a * sin), -1))
        outs.append(y[:, self.heads + self.kv_heads:])
        return torch.autograd.grad(outs, (x, w, wq, wk), [t.float() for t in (dq, dk, dv)])


def off(got, want) -> float:
    return float((got.float() - want).norm() / want.norm())


def run(hidden=2048, heads=16, kv_heads=4, d=128, batch=16, prefix=2048, prompt=50, steps=64, window=256, sinks=8,
        quiet=False) -> dict:
    """The example; returns the relative errors it prints, and the pages that the second layer holds at its end."""
    dev, page = torch.device("cuda"), 32
    prefix = prefix // page * page
    g = torch.Generator(device=dev).manual_seed(1)
    most = prefix + prompt + steps + 1
    layers = [Layer(hidden, heads, kv_heads, d, batch, most, page=page, device=dev, seed=2),
              Layer(hidden, heads, kv_heads, d, batch, most, window, sinks, page=page, device=dev, seed=3)]
    i32 = dict(dtype=torch.int32, device=dev)
    res = {}

    def both(x, new, max_q):
        h = x + layers[0](x, new, max_q)
        return h, h + layers[1](h, new, max_q)

    def say(name, start, end):
        torch.cuda.synchronize()
        if not quiet:
            print(f"{name:44s} {start.elapsed_time(end) * 1e3:9.1f} us")

    def timed(name, fn):
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        a.record()
        r = fn()
        b.record()
        say(name, a, b)
        return r

    def compare(name, x, h, y, seq):
        """x, h, y: the last tokens of sequence seq, before, between and after the layers."""
        e = max(off((h - x), layers[0].reference(x, seq)), off((y - h), layers[1].reference(h, seq)))
        res[name] = max(res.get(name, 0.0), e)

    x = torch.randn(prefix, hidden, generator=g, device=dev).bfloat16()
    new = torch.zeros(batch, **i32)
    new[0] = prefix
    timed(f"instruction of {prefix} tokens, once", lambda: both(x, new, prefix))
    for layer in layers:
        layer.share(prefix)

    counts = [1 + (prompt - 1) * (i % 3) // 2 for i in range(batch)]     # prompts of unlike lengths
    x = torch.randn(sum(counts), hidden, generator=g, device=dev).bfloat16()
    h, y = timed(f"{batch} prompts of up to {prompt} tokens", lambda: both(x, torch.tensor(counts, **i32), prompt))
    compare("prompt", x[-1:], h[-1:], y[-1:], batch - 1)

    tok, one = torch.randn(batch, hidden, generator=g, device=dev).bfloat16(), torch.ones(batch, **i32)
    both(tok, one, 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, y = both(tok, one, 1)
    for i in range(steps):
        tok.copy_(torch.randn(batch, hidden, generator=g, device=dev))
        (lambda f: timed(f"token of {batch} sequences (one graph)", f) if i == steps - 1 else f())(graph.replay)
        if i in (0, steps - 1):
            compare("decode", tok[-1:], h[-1:], y[-1:], batch - 1)
    held = layers[1].tables.table[-1]
    res["held"] = int((held >= 0).sum())
    for layer in layers:       # the batch ends: its own pages go back, the shared ones stay
        fp4.kv4_release(layer.tables, keep=torch.full((batch,), prefix, **i32), shared=layer.shared)
    res["free"] = [int(layer.tables.count) for layer in layers]

    n = 2 * prompt
    x, pos = torch.randn(n, hidden, generator=g, device=dev).bfloat16(), torch.arange(n, **i32) % most
    grads = [torch.randn(n, k, d, generator=g, device=dev).bfloat16() for k in (heads, kv_heads, kv_heads)]
    got = timed("training step of projection, norm, rotation", lambda: layers[0].train_step(x, pos, *grads))
    for name, a, b in zip(("dx", "dw", "dq_norm", "dk_norm"), got, layers[0].train_reference(x, pos, *grads)):
        res[name] = off(a, b)
    if not quiet:
        print("relative errors:", ", ".join(f"{k} {v:.2e}" for k, v in res.items() if isinstance(v, float)))
        print(f"pages that a sequence of {most} tokens holds in the second layer: {res['held']}")
    return res


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("hidden", 2048), ("heads", 16), ("kv-heads", 4), ("d", 128), ("batch", 16), ("prefix", 2048),
                          ("prompt", 50), ("steps", 64), ("window", 256), ("sinks", 8)):
        p.add_argument("--" + name, type=int, default=default)
    run(**vars(p.parse_args()))


if __name__ == "__main__":
    main()
