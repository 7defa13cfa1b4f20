"""The attention calls' plans and limits, as far as the host alone decides them."""
import ctypes as C

import quantized_linear_layers_fp4_amd as fp4


def test_own_tokens_of_256_heads_take_the_prefix_in():
    """32 sequences of 8 heads of 64 over 16384 shared tokens: as for 31, whose rows are as many tiles, own tokens leave no partial
    results (they take the prefix's in), so the workspace is the prefix's alone."""
    size, parts = fp4.lib().fp4_kv4_attention_shared_workspace_bytes, fp4.lib().fp4_kv4_attention_shared_parts
    for own in (7, 15, 30):
        a, b = ((n, n, 1, 32, 8, 64, 64, 256 + own, 256) for n in (31, 32))
        assert parts(*a) == parts(*b) == 2
        assert size(*a) == size(*b)


def test_limits_of_the_header():
    """The attention's documented limits are those of its checks: an odd address is what a call of valid sizes is refused for."""
    L, fake, odd = fp4.lib(), C.c_void_p(0x100000), C.c_void_p(0x100001)
    SHAPE, ALIGN = 2, 9

    def plain(nq=1, b=1, mq=1, hq=32, hkv=8, width=4, page=16):
        return L.fp4_kv4_attention(odd, hq * 128, 128, nq, hq, fake, fake, b, mq, fake, width, width, fake, 9, page, hkv, 128, 0, 0.1,
                                   fake, None, fake, 1 << 62, None)

    def shared(nq=1, b=1, mq=1, hq=32, hkv=8, width=4, page=16, pre=2):
        return L.fp4_kv4_attention_shared(odd, hq * 128, 128, nq, hq, fake, fake, b, mq, fake, width, width, fake, 9, page, hkv, 128, pre,
                                          0.1, fake, None, fake, 1 << 62, None)
    for call in (plain, shared):
        for good, bad in ((dict(width=1 << 20, page=1024), dict(width=(1 << 20) + 1, page=1024)), (dict(b=(1 << 19) - 1), dict(b=1 << 19)),
                          (dict(mq=(1 << 24) - 1, hq=1, hkv=1), dict(mq=1 << 24, hq=1, hkv=1)),
                          (dict(mq=(1 << 21) - 4), dict(mq=1 << 21))):            # 8 heads of (2^21 - 4) * 4 / 16 tiles
            assert call(**good) == ALIGN, (call, good)
            assert call(**bad) == SHAPE, (call, bad)
    assert plain(nq=(1 << 31) // 32 - 1) == ALIGN and plain(nq=(1 << 31) // 32) == SHAPE
    assert shared(nq=(1 << 21) - 4) == ALIGN and shared(nq=(1 << 21) - 3) == SHAPE   # all queries' rows are tiles of the prefix
    assert shared(nq=(1 << 24) - 1, hq=1, hkv=1) == ALIGN and shared(nq=1 << 24, hq=1, hkv=1) == SHAPE
