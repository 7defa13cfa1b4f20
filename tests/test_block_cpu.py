"""Refusals of the block-scaled FP8 layer and of the 4-bit cache: every check runs on the host."""
import ctypes as C

import numpy as np
import pytest
import torch

import block_ref
import quantized_linear_layers_fp4_amd as fp4

OK, ENULL, ESHAPE, EDTYPE, EQ, ECAP, EWS, EDEV, EHIP, EALIGN, ESCRATCH = range(11)
FAKE, ODD = C.c_void_p(0x100000), C.c_void_p(0x100001)
SIDE = (1 << 23) - 128


def test_operand_bytes():
    L = fp4.lib()
    assert L.fp4_block8_codes_bytes(5, 130) == 5 * 256
    assert L.fp4_block8_scales_bytes(5, 130, 0) == 5 * 4            # two blocks in one dword a row
    assert L.fp4_block8_scales_bytes(129, 513, 0) == 2 * 129 * 4    # five blocks: two dwords a row
    assert L.fp4_block8_scales_bytes(129, 513, 1) == 2 * 2 * 4      # two scale rows
    for r, c in ((0, 1), (1, 0), (SIDE + 1, 1), (1, SIDE + 1), (1 << 18, 1 << 17)):
        assert L.fp4_block8_codes_bytes(r, c) == 0 and L.fp4_block8_scales_bytes(r, c, 0) == 0
    assert L.fp4_block8_scales_bytes(4, 4, 2) == 0


def test_quantize_rejects():
    f = fp4.lib().fp4_block8_quantize
    call = lambda X=FAKE, dt=1, R=4, Cn=4, ld=4, mode=0, rc=FAKE, rs=FAKE, cc=None, cs=None: f(  # noqa: E731
        X, dt, R, Cn, ld, mode, rc, rs, cc, cs, None)
    assert call(X=None) == ENULL and call(rc=None, rs=None) == ENULL
    assert call(rs=None) == ENULL and call(cc=FAKE) == ENULL
    assert call(dt=2) == EDTYPE and call(mode=2) == EDTYPE and call(mode=-1) == EDTYPE
    assert call(R=0) == ESHAPE and call(Cn=0) == ESHAPE and call(ld=3) == ESHAPE and call(R=SIDE + 1) == ESHAPE
    assert call(X=ODD) == EALIGN and call(X=C.c_void_p(0x100002), dt=0) == EALIGN and call(rc=ODD) == EALIGN


def test_product_rejects():
    L = fp4.lib()
    g = lambda a=FAKE, am=0, bm=1, M=4, N=4, K=4, Y=FAKE, yd=1: L.fp4_block8_gemm(  # noqa: E731
        a, FAKE, am, FAKE, FAKE, bm, M, N, K, Y, yd, None)
    assert g(a=None) == ENULL and g(am=3) == EDTYPE and g(bm=3) == EDTYPE and g(yd=2) == EDTYPE
    assert g(M=0) == ESHAPE and g(N=0) == ESHAPE and g(K=0) == ESHAPE and g(a=ODD) == EALIGN and g(Y=ODD) == EALIGN
    need = L.fp4_block8_linear_workspace_bytes(4, 200, 8)
    assert need == 1024 + 256 and L.fp4_block8_linear_workspace_bytes(0, 200, 8) == 0
    f = lambda X=FAKE, ld=200, K=200, xt=None, ws=FAKE, n=need, wm=1: L.fp4_block8_linear(  # noqa: E731
        X, 1, 4, K, ld, FAKE, FAKE, wm, 8, FAKE, 1, xt, None, ws, n, None)
    assert f(X=None) == ENULL and f(ws=None) == ENULL and f(xt=FAKE) == ENULL
    assert f(ld=199) == ESHAPE and f(K=0) == ESHAPE and f(n=need - 1) == EWS and f(ws=ODD) == EALIGN and f(wm=9) == EDTYPE
    need = L.fp4_block8_backward_workspace_bytes(4, 8)
    b = lambda w=FAKE, xt=FAKE, dX=FAKE, dW=FAKE, n=need, ld=8, wd=1: L.fp4_block8_backward(  # noqa: E731
        FAKE, 1, 4, 200, 8, ld, w, w, 1, xt, xt, dX, 1, dW, wd, FAKE, n, None)
    assert b(dX=None, dW=None) == ENULL and b(w=None) == ENULL and b(xt=None) == ENULL
    assert b(n=need - 1) == EWS and b(ld=7) == ESHAPE and b(wd=5) == EDTYPE


def test_cache_rejects():
    L = fp4.lib()
    assert L.fp4_kv4_cache_bytes(3, 16, 2, 128) == 3 * 2 * 16 * (128 + 8)
    for bad in ((0, 16, 2, 128), (1, 8, 2, 128), (1, 24, 2, 128), (1, 2048, 2, 128), (1, 16, 0, 128), (1, 16, 2, 96)):
        assert L.fp4_kv4_cache_bytes(*bad) == 0
    w = lambda c=FAKE, page=16, d=128, dt=1, n=4, slots=FAKE, sb=8, k=FAKE: L.fp4_kv4_write(  # noqa: E731
        c, 2, page, 2, d, k, FAKE, dt, n, 256, 128, 256, 128, slots, sb, None)
    assert w(c=None) == ENULL and w(slots=None) == ENULL and w(dt=2) == EDTYPE and w(sb=2) == EDTYPE
    assert w(page=20) == ESHAPE and w(d=32) == ESHAPE and w(n=0) == ESHAPE
    assert w(k=ODD) == EALIGN and w(slots=C.c_void_p(0x100004)) == EALIGN and w(slots=C.c_void_p(0x100004), sb=4) != EALIGN
    r = lambda n=4, K=FAKE, dt=0: L.fp4_kv4_read(FAKE, 2, 16, 2, 128, FAKE, 8, n, K, FAKE, dt, None)  # noqa: E731
    assert r(n=0) == ESHAPE and r(K=None) == ENULL and r(K=C.c_void_p(0x100008)) == EALIGN and r(dt=3) == EDTYPE


def test_attention_rejects():
    L = fp4.lib()
    need = L.fp4_kv4_attention_workspace_bytes(1, 1, 8, 2, 128, 16, 64)
    assert need > 0 and L.fp4_kv4_attention_workspace_bytes(1, 1, 7, 2, 128, 16, 64) == 0

    def a(q=FAKE, nq=1, hq=8, qs=None, lens=FAKE, b=1, mq=1, ts=64, width=64, page=16, hkv=2, d=128, win=0, o=FAKE,
          ws=FAKE, n=need):
        return L.fp4_kv4_attention(q, 1024, 128, nq, hq, qs, lens, b, mq, FAKE, ts, width, FAKE, 64, page, hkv, d, win,
                                   0.1, o, None, ws, n, None)
    assert a(q=None) == ENULL and a(lens=None) == ENULL and a(o=None) == ENULL and a(ws=None) == ENULL
    assert a(n=need - 1) == EWS
    assert a(hq=7) == ESHAPE and a(page=12) == ESHAPE and a(d=80) == ESHAPE and a(win=-1) == ESHAPE
    assert a(ts=63) == ESHAPE and a(nq=2) == ESHAPE and a(mq=2) == ESHAPE and a(mq=0, qs=FAKE) == ESHAPE
    assert a(width=0) == ESHAPE and a(nq=0, qs=FAKE) == ESHAPE
    assert a(q=ODD) == EALIGN and a(o=C.c_void_p(0x100008)) == EALIGN


def test_attention_workspace_of_many_sequences():
    """A call of many sequences is not split into more workgroups than a launch can have: 2^21 (sequence, head)s
    over a million tokens are split in two, not in 64."""
    L = fp4.lib()
    row = (128 + 4) * 4
    assert L.fp4_kv4_attention_workspace_bytes(1 << 16, 1, 32, 32, 128, 128, 8192) == (1 << 21) * 2 * row
    assert L.fp4_kv4_attention_workspace_bytes(1 << 10, 1, 32, 32, 128, 128, 8192) == (1 << 15) * 64 * row
    assert L.fp4_kv4_attention_workspace_bytes(64, 1, 32, 8, 128, 64, 128) == 512 * 8 * 4 * row


def test_python_checks():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        fp4.block8_quantize(x)                       # not on a device
    with pytest.raises(fp4.Fp4Error):
        fp4.kv4_cache(1, 20, 2, 128, device="cpu")
    c = fp4.kv4_cache(2, 16, 2, 64, device="cpu")
    assert c.data.numel() == 2 * 2 * 16 * 68 and int(c.data.max()) == 0
    with pytest.raises(TypeError):
        fp4.kv4_attention(torch.zeros(1, 2, 64), c, torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fp4.kv4_read(c, torch.zeros(1, dtype=torch.int64), d=128)


def test_reference_grids():
    """The references' own numbers: exponents at the limits, ties to even, saturation."""
    assert list(block_ref.exponent(np.array([0, 448, 448.5, 896, 1e-45]), 448.0)) == [-127, 0, 1, 1, -127]
    assert list(block_ref.exponent(np.array([7, 7.01, 6, 3.5]), 7.0)) == [0, 1, 0, -1]
    assert list(block_ref.nearest(np.array([0.25, 0.75, 2.5, 5.0, 6.9, -1.25]), block_ref.E2M1)) == [0, 1, 2, 4, 6, -1]
    assert list(block_ref.nearest(np.array([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]), block_ref.E4M3)) == [16, 20, 0, 2.0 ** -8]
