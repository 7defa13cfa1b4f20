"""Refusals of the page tables, the norm with rotation and the attention with sinks or shared pages: every check runs on
the host before any HIP call."""
import ctypes as C

import pytest
import torch

import quantized_linear_layers_fp4_amd as fp4

OK, ENULL, ESHAPE, EDTYPE, EQ, ECAP, EWS, EDEV, EHIP, EALIGN, ESCRATCH = range(11)
FAKE, ODD, HALF = C.c_void_p(0x100000), C.c_void_p(0x100001), C.c_void_p(0x100004)


def test_extend_rejects():
    L = fp4.lib()
    assert L.fp4_kv4_extend_workspace_bytes(5, 8192) == 0 and L.fp4_kv4_extend_workspace_bytes(5, 8193) == 4 * 12
    assert L.fp4_kv4_extend_workspace_bytes(1025, 1) == 4 * 2052
    for b, n in ((0, 1), ((1 << 20) + 1, 1), (1, -1), (1, 0x7FFFFFFF)):
        assert L.fp4_kv4_extend_workspace_bytes(b, n) == 0

    def e(table=FAKE, stride=8, b=4, width=8, lens=FAKE, free=FAKE, count=FAKE, pages=99, page=16, new=FAKE, n=10, slots=FAKE,
          pos=FAKE, qs=FAKE, ws=None, wsb=0):
        return L.fp4_kv4_extend(table, stride, b, width, lens, free, count, pages, page, new, n, slots, pos, qs, ws, wsb, None)
    for kw in (dict(table=None), dict(lens=None), dict(free=None), dict(count=None), dict(slots=None), dict(pos=None),
               dict(n=9000, wsb=40)):
        assert e(**kw) == ENULL
    for kw in (dict(stride=7), dict(b=0), dict(width=0), dict(page=8), dict(page=48), dict(page=2048), dict(pages=0), dict(n=-1),
               dict(n=0x7FFFFFFF), dict(qs=None), dict(b=(1 << 20) + 1), dict(width=1 << 27, stride=1 << 27),
               dict(b=1 << 16, width=1 << 15, stride=1 << 15)):
        assert e(**kw) == ESHAPE, kw
    assert e(n=9000, ws=FAKE, wsb=39) == EWS
    for kw in (dict(table=ODD), dict(lens=ODD), dict(new=ODD), dict(slots=HALF), dict(pos=ODD), dict(qs=ODD), dict(count=ODD)):
        assert e(**kw) == EALIGN, kw


def test_release_rejects():
    L = fp4.lib()
    assert L.fp4_kv4_release_workspace_bytes(4, 4096) == 0 and L.fp4_kv4_release_workspace_bytes(4, 4097) == 4100
    assert L.fp4_kv4_release_workspace_bytes(0, 4) == 0

    def r(table=FAKE, stride=8, width=8, keep=None, window=0, sinks=0, shared=0, ws=None, wsb=0):
        return L.fp4_kv4_release(table, stride, 4, width, FAKE, FAKE, FAKE, 99, 16, keep, window, sinks, shared, ws, wsb, None)
    assert r(table=None) == ENULL and r(width=5000, stride=5000, wsb=4100) == ENULL
    for kw in (dict(stride=7), dict(window=-1), dict(sinks=-1), dict(shared=-1)):
        assert r(**kw) == ESHAPE
    assert r(width=5000, stride=5000, ws=FAKE, wsb=4099) == EWS and r(keep=ODD) == EALIGN


def rope(q=FAKE, hq=4, k=FAKE, hkv=2, n=3, d=64, dt=1, qw=FAKE, kw=FAKE, wdt=1, eps=1e-6, pos=FAKE, tab=FAKE, mp=10, rot=64,
         qo=FAKE, ko=FAKE):
    return fp4.lib().fp4_qk_norm_rope(q, 512, 64, hq, k, 512, 64, hkv, n, d, dt, qw, kw, wdt, eps, pos, tab, mp, rot, 0, qo, ko, None)


SHARED_ARGUMENTS = [
    (dict(pos=None), ENULL), (dict(tab=None), ENULL), (dict(dt=2), EDTYPE), (dict(wdt=7), EDTYPE), (dict(n=0), ESHAPE),
    (dict(n=(1 << 24) + 1), ESHAPE), (dict(n=1 << 24, hq=31), ESHAPE), (dict(d=60), ESHAPE), (dict(d=24, rot=16), ESHAPE),
    (dict(d=264), ESHAPE), (dict(rot=24), ESHAPE), (dict(rot=80), ESHAPE), (dict(rot=-16), ESHAPE), (dict(mp=0), ESHAPE),
    (dict(eps=-2.0), ESHAPE), (dict(eps=float("nan")), ESHAPE), (dict(eps=-1.0), ESHAPE), (dict(hq=0), ESHAPE), (dict(q=ODD), EALIGN),
    (dict(pos=ODD), EALIGN), (dict(tab=HALF), EALIGN), (dict(qw=ODD), EALIGN)]


@pytest.mark.parametrize("kw,status", SHARED_ARGUMENTS)
def test_norm_rejects(kw, status):
    assert rope(**kw) == status


def test_norm_rejects_more():
    assert rope(q=None) == ENULL and rope(qo=None) == ENULL and rope(k=None) == ENULL and rope(ko=None) == ENULL
    assert rope(hkv=-1) == ESHAPE and rope(ko=ODD) == EALIGN and rope(q=C.c_void_p(0x100002), dt=0) == EALIGN
    t = fp4.lib().fp4_rope_table
    assert t(None, 4, 16, 1e4, 1.0, None) == ENULL and t(HALF, 4, 16, 1e4, 1.0, None) == EALIGN
    for a in ((0, 16, 1e4, 1.0), (4, 8, 1e4, 1.0), (4, 24, 1e4, 1.0), (4, 272, 1e4, 1.0), (1 << 29, 16, 1e4, 1.0), (4, 16, 0.0, 1.0),
              (4, 16, 1e4, 0.0), (4, 16, float("nan"), 1.0)):
        assert t(FAKE, *a, None) == ESHAPE


@pytest.mark.parametrize("kw,status", SHARED_ARGUMENTS)
def test_gradients_reject(kw, status):
    assert backward(**kw) == status


def backward(q=FAKE, hq=4, k=FAKE, hkv=2, n=3, d=64, dt=1, qw=FAKE, kw=FAKE, wdt=1, eps=1e-6, pos=FAKE, tab=FAKE, mp=10, rot=64,
             dq=FAKE, dk=FAKE, gq=FAKE, gk=FAKE, wq=FAKE, wk=FAKE, ws=FAKE, wsb=1 << 22):
    return fp4.lib().fp4_qk_norm_rope_backward(dq, 512, 64, dk, 512, 64, q, 512, 64, hq, k, 512, 64, hkv, n, d, dt, qw, kw, wdt, eps,
                                               pos, tab, mp, rot, 0, gq, 512, 64, gk, 512, 64, wq, wk, ws, wsb, None)


def test_gradients_reject_more():
    L = fp4.lib()
    need = L.fp4_qk_norm_rope_backward_workspace_bytes(64)
    assert need > 0 and L.fp4_qk_norm_rope_backward_workspace_bytes(60) == 0 and L.fp4_qk_norm_rope_backward_workspace_bytes(264) == 0
    for name in ("q", "k", "dq", "dk", "gq", "gk", "ws"):
        assert backward(**{name: None}) == ENULL, name
    assert backward(wsb=need - 1) == EWS and backward(ws=ODD) == EALIGN and backward(wq=ODD) == EALIGN and backward(gk=ODD) == EALIGN
    assert backward(qw=None, kw=None, eps=-1.0) == ESHAPE                     # a weight's gradient without a norm
    assert backward(hkv=0, k=None, dk=None, gk=None, kw=None) == ESHAPE       # ... without keys


def test_fused_write_rejects():
    def w(cache=FAKE, pages=2, page=16, q=FAKE, k=FAKE, v=FAKE, hq=4, hkv=2, n=3, d=64, dt=1, slots=FAKE, sb=8, rot=64, qo=FAKE,
          eps=1e-6):
        return fp4.lib().fp4_kv4_norm_rope(cache, pages, page, q, 512, 64, hq, k, 512, 64, v, 512, 64, hkv, n, d, dt, slots, sb, FAKE,
                                           FAKE, 1, eps, FAKE, FAKE, 10, rot, 0, qo, None)
    for name in ("cache", "q", "k", "v", "slots", "qo"):
        assert w(**{name: None}) == ENULL, name
    assert w(sb=2) == EDTYPE and w(dt=5) == EDTYPE
    for kw in (dict(pages=0), dict(page=20), dict(d=32, rot=32), dict(d=256), dict(hkv=0), dict(n=0), dict(rot=8), dict(eps=-3.0)):
        assert w(**kw) == ESHAPE, kw
    for kw in (dict(cache=ODD), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(slots=HALF), dict(qo=ODD)):
        assert w(**kw) == EALIGN, kw
    assert w(slots=HALF, sb=4) != EALIGN


def test_sinks_and_shared_reject():
    L = fp4.lib()
    need = L.fp4_kv4_attention_workspace_bytes(1, 1, 8, 2, 128, 16, 64)

    def s(win=5, sinks=3, n=need, q=FAKE, ws=FAKE):
        return L.fp4_kv4_attention_sinks(q, 1024, 128, 1, 8, None, FAKE, 1, 1, FAKE, 64, 64, FAKE, 64, 16, 2, 128, win, sinks, 0.1, FAKE,
                                         None, ws, n, None)
    assert s(sinks=-1) == ESHAPE and s(win=-1) == ESHAPE and s(n=need - 1) == EWS and s(q=None) == ENULL and s(ws=ODD) == EALIGN
    big = dict(nq=64, b=64, mq=1, hq=32, hkv=8, d=128, page=64, width=80, sh=64)
    size, parts = ((lambda fn: lambda **kw: fn(*({**big, **kw}.values())))(fn) for fn in (
        L.fp4_kv4_attention_shared_workspace_bytes, L.fp4_kv4_attention_shared_parts))
    need = size()
    assert need > 0 and parts() == 2
    assert parts(nq=1, b=1) == 1 and parts(nq=4, b=4, width=6, sh=4) == 1     # nothing to save
    for kw in (dict(nq=0), dict(b=0), dict(mq=0), dict(hq=12), dict(d=96), dict(page=24), dict(sh=0), dict(sh=81), dict(nq=1 << 24),
               dict(nq=(1 << 22) + 1)):
        assert size(**kw) == 0 and parts(**kw) == 0, kw

    def f(q=FAKE, nq=64, hq=32, qs=None, b=64, mq=1, ts=80, width=80, sh=64, o=FAKE, ws=FAKE, n=need):
        return L.fp4_kv4_attention_shared(q, 4096, 128, nq, hq, qs, FAKE, b, mq, FAKE, ts, width, FAKE, 9000, 64, 8, 128, sh, 0.1, o,
                                          None, ws, n, None)
    assert f(q=None) == ENULL and f(o=None) == ENULL and f(ws=None) == ENULL and f(n=need - 1) == EWS
    for kw in (dict(sh=0), dict(sh=81), dict(hq=12), dict(ts=79), dict(nq=2), dict(nq=0, qs=FAKE), dict(mq=2)):
        assert f(**kw) == ESHAPE, kw
    assert f(q=ODD) == EALIGN and f(o=HALF) == EALIGN and f(ws=HALF) == EALIGN


def test_python_checks():
    with pytest.raises(fp4.Fp4Error):
        fp4.kv4_page_tables(2, 3, 10, 24, device="cpu")
    with pytest.raises(ValueError):
        fp4.kv4_page_tables(2, 3, 10, 16, device="cpu")      # tables live on a device
    with pytest.raises(ValueError):
        fp4.rope_table(4, 16, device="cpu")
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        fp4.qk_norm_rope(x, x)
    with pytest.raises(ValueError):
        fp4.kv4_norm_rope(fp4.kv4_cache(2, 16, 2, 64, device="cpu"), x, x, x, torch.zeros(4, dtype=torch.int64))
