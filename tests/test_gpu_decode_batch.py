"""The batch example at small sizes (needs an MI355X): instruction, prompts, captured steps, training step.

Layers against fp32 on the values that weights and caches hold: an E4M3 operand is off by at most 2^-4 a value, rounded
independently, so a projection's result by at most that in norm (2^-4); the queries' error e turns into about e |s| of a
weight, |s| here up to a few: 4 x 2^-4, then the output projection's 2^-4: below 0.5.
Gradients against unquantized fp32: two operands a product, 2^-3; the projection's own error (2^-3, its two operands) goes
through the norm's and rotation's gradients once more, at most twice (both terms of x's): below 3 x 2^-3.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("heads,kv_heads,d,batch,prefix,prompt,steps,window,sinks", [
    (8, 2, 64, 5, 96, 20, 6, 40, 3), (4, 4, 128, 3, 320, 33, 40, 64, 40), (6, 1, 64, 1, 64, 1, 3, 1, 1)])
def test_decode_batch(heads, kv_heads, d, batch, prefix, prompt, steps, window, sinks):
    spec = importlib.util.spec_from_file_location("decode_batch", os.path.join(ROOT, "examples", "decode_batch.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.run(hidden=520, heads=heads, kv_heads=kv_heads, d=d, batch=batch, prefix=prefix, prompt=prompt, steps=steps,
              window=window, sinks=sinks, quiet=True)
    assert all(r[k] <= 0.5 for k in ("prompt", "decode")), r
    assert all(r[k] <= 0.375 for k in ("dx", "dw", "dq_norm", "dk_norm")), r
    width = -(-(prefix + prompt + steps + 1) // 32)
    assert r["free"][0] == batch * width - prefix // 32 <= r["free"][1]  # (the second gave back some of the instruction's)
    # of the second layer's own pages, those of the window and of its ends are held at most
    assert r["held"] <= prefix // 32 + (window + 30) // 32 + 1
