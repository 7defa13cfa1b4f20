"""Single tokens through a window with sinks: which calls are split along their tokens (needs an MI355X).

A call that is split leaves partial results in its workspace, one that is not leaves it as it was.  Results of either are the same
within the roundings of the sums: p in bf16 (2^-8 of a term, either way) and the output (2^-8).
"""
import pytest
import torch

import quantized_linear_layers_fp4_amd as fp4

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def run(b, hkv, d, window, lens, width, page=64, sinks=64, g=2):
    """(o, lse, whether the workspace was written) of sequences over few pages, which stand for long ones."""
    gen = torch.Generator(device=DEV).manual_seed(b)
    cache = fp4.kv4_cache(200, page, hkv, d)
    k, v = (torch.randn(200 * page, hkv, d, generator=gen, device=DEV) for _ in range(2))
    fp4.kv4_write(cache, k, v, torch.arange(200 * page, device=DEV))
    table = torch.randint(0, 200, (b, width), generator=gen, device=DEV, dtype=torch.int32)
    q = torch.randn(b, hkv * g, d, generator=gen, device=DEV).bfloat16()
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ws = torch.full((fp4.kv4_attention_workspace(q, cache, table).numel(),), 77, dtype=torch.uint8, device=DEV)
    got = fp4.kv4_attention(q, cache, table, n, window=window, sinks=sinks, return_lse=True, ws=ws)
    few = [fp4.kv4_attention(q[i:i + 1], cache, table[i:i + 1], n[i:i + 1], window=window, sinks=sinks, return_lse=True)
           for i in range(0, b, 7)]
    mag = float(v.abs().max())
    for j, (o, lse) in enumerate(few):
        assert float((o - got[0][7 * j:7 * j + 1]).float().abs().max()) <= 4 * 2.0 ** -8 * mag
        assert torch.allclose(lse, got[1][7 * j:7 * j + 1], rtol=0, atol=2.0 ** -18 * 32)
    return bool((ws != 77).any())


@pytest.mark.parametrize("b,hkv,d,window,split", [
    (32, 8, 128, 1900, False), (32, 8, 128, 8000, True), (32, 8, 128, 32000, True), (40, 8, 128, 1800, False), (40, 8, 128, 4000, True),
    (64, 8, 128, 2048 - 64, False), (64, 8, 128, 7000, False), (64, 8, 128, 16000, True), (64, 8, 64, 3000, False), (64, 8, 64, 8000, True)])
def test_long_windows_are_split(b, hkv, d, window, split):
    """A batch of unlike lengths through a long window is not left to one workgroup for each (sequence, head)."""
    width = 1100
    lens = [(1 << (5 + i % 12)) + 31 * i for i in range(b)]
    assert run(b, hkv, d, window, lens, width) == split
