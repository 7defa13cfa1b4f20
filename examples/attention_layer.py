"""One attention layer on the FP8 projections and the 4-bit key/value cache: a prompt, then single tokens,
then a training step of its projection.

    python examples/attention_layer.py [--hidden 2048 --heads 16 --kv-heads 4 --prompt 1000 --steps 32]

The layer's weights are quantized once (E4M3, one power-of-two scale per 128 x 128 block).  Each call projects
its tokens to q, k and v, writes k and v into the paged cache in 4 bits, attends over it and projects back.
Decode steps run from one captured HIP graph.  Prints the time of each part and how far the outputs are from the
same layer in fp32 on the values that the quantized weights and the cache stand for.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_linear_layers_fp4_amd as fp4  # noqa: E402


class AttentionLayer:
    """q, k, v and output projections in FP8 with block-128 scales, keys and values in a 4-bit paged cache."""

    def __init__(self, hidden: int, heads: int, kv_heads: int, d: int, batch: int, max_tokens: int, page: int = 64,
                 device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.d, self.page = heads, kv_heads, d, page
        self.w_qkv = (torch.randn(hidden, (heads + 2 * kv_heads) * d, generator=g, device=device) * hidden ** -0.5).bfloat16()
        self.w_out = (torch.randn(heads * d, hidden, generator=g, device=device) * (heads * d) ** -0.5).bfloat16()
        self.qkv, self.out = (fp4.block8_quantize(w, fp4.FP4_BLOCK_SQUARE, rows=False, cols=True)[1]
                              for w in (self.w_qkv, self.w_out))
        width = (max_tokens + page - 1) // page
        self.table = torch.randperm(batch * width, generator=g, device=device).view(batch, width).int()
        self.cache = fp4.kv4_cache(batch * width, page, kv_heads, d, device=device)

    def slots(self, seq: torch.Tensor, pos: torch.Tensor) -> torch.Tensor:
        """Cache slots of tokens pos of sequences seq."""
        return self.table[seq, pos // self.page].long() * self.page + pos % self.page

    def __call__(self, x, slots, lens, q_start=None, max_q=1):
        """x: the packed tokens (n x hidden) that go to `slots`; lens: each sequence's tokens, these among them."""
        y = fp4.block8_linear_forward(x, self.qkv).view(x.shape[0], self.heads + 2 * self.kv_heads, self.d)
        q, k, v = y[:, :self.heads], y[:, self.heads:self.heads + self.kv_heads], y[:, self.heads + self.kv_heads:]
        fp4.kv4_write(self.cache, k, v, slots)
        o = fp4.kv4_attention(q, self.cache, self.table, lens, q_start=q_start, max_q=max_q)
        return fp4.block8_linear_forward(o.view(x.shape[0], -1), self.out)

    def reference(self, x, seq: int, n: int):
        """The same in fp32 for the last x.shape[0] of sequence seq's n tokens, from the cache's values."""
        dev = x.device
        wq, wo = (fp4.block8_dequantize(w).t().contiguous() for w in (self.qkv, self.out))
        pos = torch.arange(n, device=dev)
        k, v = fp4.kv4_read(self.cache, self.slots(torch.full_like(pos, seq), pos), out_dtype=torch.float32)
        t, g = x.shape[0], self.heads // self.kv_heads
        q = (x.float() @ wq)[:, :self.heads * self.d].view(t, self.kv_heads, g, self.d)
        o = torch.empty(t, self.kv_heads, g, self.d, device=dev)
        see = pos[None, :] <= torch.arange(n - t, n, device=dev)[:, None]
        for h in range(self.kv_heads):
            s = (q[:, h].reshape(t * g, self.d) @ k[:, h].t().contiguous()).view(t, g, n) * self.d ** -0.5
            s = s.masked_fill(~see[:, None], float("-inf"))
            o[:, h] = (torch.softmax(s, 2).view(t * g, n) @ v[:, h].contiguous()).view(t, g, self.d)
        return o.view(t, -1) @ wo

    def train_step(self, x, dy):
        """Gradients of the qkv projection: (y, dx, dw), every product in FP8."""
        rows, cols = fp4.block8_quantize(self.w_qkv, fp4.FP4_BLOCK_SQUARE, rows=True, cols=True)
        y, xt = fp4.block8_linear_forward(x, cols, for_backward=True)
        return (y, *fp4.block8_linear_backward(dy, rows, xt))


def off(got, want) -> float:
    return float((got.float() - want).norm() / want.norm())


def run(hidden=2048, heads=16, kv_heads=4, d=128, batch=4, prompt=1000, steps=32, quiet=False) -> dict:
    """The example; returns the relative errors it prints."""
    dev = torch.device("cuda")
    layer = AttentionLayer(hidden, heads, kv_heads, d, batch, prompt + steps, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    i32 = dict(dtype=torch.int32, device=dev)
    res = {}

    def timed(name, fn):
        fn()
        torch.cuda.synchronize()
        a, b = torch.cuda.Event(True), torch.cuda.Event(True)
        a.record()
        r = fn()
        b.record()
        torch.cuda.synchronize()
        if not quiet:
            print(f"{name:34s} {a.elapsed_time(b) * 1e3:9.1f} us")
        return r

    x = torch.randn(batch * prompt, hidden, generator=g, device=dev).bfloat16()
    seq, pos = torch.arange(batch, device=dev), torch.arange(prompt, device=dev)
    slots = layer.slots(seq.repeat_interleave(prompt), pos.repeat(batch))
    lens = torch.full((batch,), prompt, **i32)
    starts = torch.arange(batch + 1, **i32) * prompt
    y = timed(f"prompt of {batch} x {prompt} tokens", lambda: layer(x, slots, lens, starts, prompt))
    res["prompt"] = off(y[-prompt:], layer.reference(x[-prompt:], batch - 1, prompt))

    tok = torch.randn(batch, hidden, generator=g, device=dev).bfloat16()
    step_pos = torch.zeros(batch, dtype=torch.int64, device=dev)

    def step():
        return layer(tok, layer.slots(seq, step_pos), (step_pos + 1).int())
    step_pos.fill_(prompt)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(steps):
        tok.copy_(torch.randn(batch, hidden, generator=g, device=dev))
        step_pos.fill_(prompt + i)
        graph.replay()
        if i in (0, steps - 1):
            e = off(out[:1], layer.reference(tok[:1], 0, prompt + i + 1))
            res["decode"] = max(res.get("decode", 0.0), e)
    timed(f"token of {batch} sequences (one graph)", graph.replay)

    dy = torch.randn(x.shape[0], layer.w_qkv.shape[1], generator=g, device=dev).bfloat16()
    y, dx, dw = timed("training step of the projection", lambda: layer.train_step(x, dy))
    w = layer.w_qkv.float()
    res["y"], res["dx"], res["dw"] = off(y, x.float() @ w), off(dx, dy.float() @ w.t().contiguous()), off(dw, x.float().t().contiguous() @ dy.float())
    if not quiet:
        print("relative errors:", ", ".join(f"{k} {v:.2e}" for k, v in res.items()))
    return res


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("hidden", 2048), ("heads", 16), ("kv-heads", 4), ("d", 128), ("batch", 4), ("prompt", 1000),
                          ("steps", 32)):
        p.add_argument("--" + name, type=int, default=default)
    run(**{k: v for k, v in vars(p.parse_args()).items()})


if __name__ == "__main__":
    main()
