"""The attention-layer example at small sizes (needs an MI355X): prompt, captured decode steps, training step.

Against fp32 on unquantized activations an E4M3 operand is off by at most 2^-4 a value, rounded independently, and
a product's relative error (in norm) by at most that of its two operands together, 2^-3; through the layer two such
products follow each other, and the scores turn the first one's error e into about e |s| of a weight, |s| here up to a few: 4 x 2^-3.
"""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("heads,kv_heads,d,batch,prompt", [(8, 2, 64, 3, 77), (4, 4, 128, 1, 300)])
def test_attention_layer_example(heads, kv_heads, d, batch, prompt):
    spec = importlib.util.spec_from_file_location("attention_layer", os.path.join(ROOT, "examples", "attention_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.run(hidden=520, heads=heads, kv_heads=kv_heads, d=d, batch=batch, prompt=prompt, steps=3, quiet=True)
    assert all(r[k] <= 2.0 ** -3 for k in ("y", "dx", "dw")), r
    assert all(r[k] <= 0.5 for k in ("prompt", "decode")), r
