"""Refusals of the mixture-of-experts calls, the rotating append and the norms around a block: checked before any device
is touched; and the plain forms they are tested against, on cases worked by hand."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

import moe_ref as ref
import weight_only_quantized_matmul_amd as wq

P = 1 << 20  # a 16-byte aligned address that no refused call may touch


def route(**kw):
    a = dict(device=0, scores=P, dt=0, T=2, E=64, stride=64, bias=None, gating=0, groups=1, top=1, k=4, norm=1, scale=1.0, ids=P, w=P)
    a.update(kw)
    return wq.lib.wq_moe_route_dev(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(scores=None), dict(ids=None), dict(w=None), dict(dt=3), dict(dt=-1), dict(T=-1), dict(E=0), dict(E=-4), dict(stride=-1), dict(k=0),
    dict(k=65), dict(gating=2), dict(gating=-1), dict(groups=0), dict(groups=5), dict(groups=8, top=9), dict(groups=8, top=0),
    dict(groups=32, top=1, k=3), dict(scale=math.nan), dict(scale=math.inf), dict(scores=P + 2), dict(ids=P + 2), dict(w=P + 1),
    dict(bias=P + 2), dict(dt=1, scores=P + 1)])
def test_route_refuses(bad):
    assert route(**bad) == wq.WQ_E_INVAL


def test_route_limits():
    assert route(E=wq.WQ_MOE_MAX_EXPERTS + 1) == wq.WQ_E_UNSUPPORTED
    assert route(k=wq.WQ_MOE_MAX_K + 1) == wq.WQ_E_UNSUPPORTED
    assert route(E=650, groups=65, top=2) == wq.WQ_E_UNSUPPORTED
    assert route(T=0) == wq.WQ_OK
    assert route(device=15) == wq.WQ_E_NOTINIT
    assert route(device=-1) == wq.WQ_E_NOTINIT


def test_moe_create_refuses():
    h = ctypes.c_void_p(None)
    one = (ctypes.c_void_p * 1)(None)
    junk = (ctypes.c_char * 256)()
    fake = (ctypes.c_void_p * 1)(ctypes.addressof(junk))
    assert wq.lib.wq_moe_create(None, one, one, 1, ctypes.byref(h)) == wq.WQ_E_INVAL
    assert wq.lib.wq_moe_create(one, None, one, 1, ctypes.byref(h)) == wq.WQ_E_INVAL
    assert wq.lib.wq_moe_create(one, one, None, 1, ctypes.byref(h)) == wq.WQ_E_INVAL
    assert wq.lib.wq_moe_create(one, one, one, 1, None) == wq.WQ_E_INVAL
    assert wq.lib.wq_moe_create(one, one, one, 0, ctypes.byref(h)) == wq.WQ_E_INVAL
    assert wq.lib.wq_moe_create(one, one, one, 1, ctypes.byref(h)) == wq.WQ_E_INVAL  # a null tensor
    assert wq.lib.wq_moe_create(fake, fake, fake, 1, ctypes.byref(h)) == wq.WQ_E_INVAL  # not a tensor
    assert wq.lib.wq_moe_create(one, one, one, wq.WQ_MOE_MAX_EXPERTS + 1, ctypes.byref(h)) == wq.WQ_E_UNSUPPORTED
    assert wq.lib.wq_moe_free(None) == wq.WQ_OK
    assert wq.lib.wq_moe_free(ctypes.addressof(junk)) == wq.WQ_E_INVAL
    assert wq.lib.wq_moe_ffn_dev(None, P, 0, 1, 64, P, P, 1, None, 0, P, 64, None) == wq.WQ_E_INVAL
    assert wq.lib.wq_moe_ffn_dev(ctypes.addressof(junk), P, 0, 1, 64, P, P, 1, None, 0, P, 64, None) == wq.WQ_E_INVAL
    with pytest.raises(wq.WqError):
        wq.wq_moe_create([], [], [])
    with pytest.raises(ValueError):
        wq.wq_moe_create([], [None], [])


def norm(**kw):
    a = dict(device=0, x=P, xd=0, xs=64, wpost=P, gate=P, gs=64, alpha=0.5, res=P, rs=64, wpre=P, eps=1e-6, rows=2, n=64, y=P, yd=0, ys=64,
             sum=P, ss=64)
    a.update(kw)
    return wq.lib.wq_rmsnorm_block_dev(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(res=None), dict(y=None), dict(wpre=None), dict(y=None, wpre=None, sum=None), dict(rows=-1), dict(n=0), dict(xd=3),
    dict(yd=3), dict(yd=-1), dict(eps=-1.0), dict(eps=math.nan), dict(alpha=math.nan), dict(alpha=math.inf), dict(xs=-1), dict(rs=-1),
    dict(gs=-1), dict(ys=-1), dict(ss=-1), dict(x=P + 2), dict(res=P + 2), dict(gate=P + 1), dict(sum=P + 2), dict(y=P + 2),
    dict(wpost=P + 2), dict(wpre=P + 1)])
def test_block_norm_refuses(bad):
    assert norm(**bad) == wq.WQ_E_INVAL


def test_block_norm_limits():
    assert norm(n=wq.WQ_NORM_MAX_N + 1) == wq.WQ_E_UNSUPPORTED
    assert norm(rows=0) == wq.WQ_OK
    assert norm(device=15) == wq.WQ_E_NOTINIT


def append(cache=None, batch=None, **kw):
    rc, h = 0, ctypes.c_void_p(None)
    sec = kw.pop("sections", [32])
    assert wq.lib.wq_rope_create(2 * sum(sec), 0, 1e4, (ctypes.c_int * len(sec))(*sec), len(sec), ctypes.byref(h)) == 0
    c = wq._KvCacheC(kw.pop("device", 0), 1, 4, 2, 16, 64, P, P, P, P, (ctypes.c_long * 3)(2048, 1024, 64), (ctypes.c_long * 3)(32, 16, 1))
    b = wq._KvBatchC(1, kw.pop("T", 3), 4, 3, 20, 4, P, P, P)
    a = dict(rope=h, q=P, H=4, qt=256, qh=64, o=P, ot=256, oh=64, k=P, v=P, dt=0, tok=128, head=64, pos=P, ps=3)
    a.update(kw)
    rc = wq.lib.wq_kv_append_rope_dev(ctypes.byref(c) if cache is None else cache, ctypes.byref(b) if batch is None else batch, *a.values(), None)
    wq.lib.wq_rope_free(h)
    return rc


@pytest.mark.parametrize("bad", [
    dict(rope=None), dict(q=None), dict(o=None), dict(H=0), dict(H=-1), dict(qt=-1), dict(qh=-1), dict(ot=-1), dict(oh=-1), dict(k=None),
    dict(v=None), dict(dt=3), dict(tok=-1), dict(head=-1), dict(ps=-1), dict(q=P + 2), dict(o=P + 2), dict(k=P + 2), dict(v=P + 2),
    dict(pos=P + 2), dict(sections=[16, 16], pos=None), dict(sections=[64])])
def test_append_rope_refuses(bad):
    assert append(**bad) == wq.WQ_E_INVAL


def test_append_rope_limits():
    assert append(H=wq.WQ_KV_MAX_HEADS + 1) == wq.WQ_E_UNSUPPORTED
    assert append(T=0) == wq.WQ_OK
    assert append(device=15) == wq.WQ_E_NOTINIT


def test_plain_route_by_hand():
    ln = math.log
    ids, w = ref.route(np.array([[ln(1), ln(2), ln(4), ln(1)]]), 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[2 / 3, 1 / 3]], rtol=1e-15)
    ids, w = ref.route(np.array([[0.0, 0.0, 0.0, 0.0]]), 3, normalise=False, scale=2.0)
    assert ids.tolist() == [[0, 1, 2]] and np.allclose(w, 0.5, rtol=1e-15)  # ties: the lower first
    # groups {0, 1} and {2, 3}: the largest expert is in the first, the larger sum in the second
    ids, w = ref.route(np.array([[ln(9), ln(0.25), ln(4), ln(4)]]), 1, gating="sigmoid", groups=2, top_groups=1, normalise=False)
    assert ids.tolist() == [[2]] and np.allclose(w, 0.8, rtol=1e-15)  # 0.9 + 0.2 < 0.8 + 0.8
    ids, w = ref.route(np.array([[0.0, 0.0]]), 1, bias=np.array([0.0, 0.1], dtype=np.float32), gating="sigmoid", normalise=False)
    assert ids.tolist() == [[1]] and w.tolist() == [[0.5]]  # the bias chooses and does not weigh
    ids, w = ref.route(np.array([[np.nan, -np.inf, -np.inf]]), 2)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


def test_plain_moe_by_hand():
    # one input, one hidden element, one output: y = w * d * silu(g x) * (u x)
    g, u, d = (np.array([[v]]) for v in (2.0, 3.0, 5.0))
    x, w = math.log(3) / 2, 0.5
    y, _ = ref.moe(np.array([[x]]), np.array([[0, -1]]), np.array([[w, 9.0]]), [(g, u, d)], add=np.array([[1.0]]))
    assert np.isclose(y[0, 0], 1 + w * 5 * (2 * x * 0.75) * (3 * x), rtol=1e-15)  # silu(ln 3) = ln 3 * 3/4
    codes = np.array([[0x21]], dtype=np.uint8)
    assert ref.open_matrix(codes, np.array([2.0]), 2, ref.I4, 0).tolist() == [[-14.0, -12.0]]
    assert ref.open_matrix(codes, np.array([1.0]), 3, ref.I2, 0).tolist() == [[-1.0, -2.0, 0.0]]
    assert ref.open_matrix(np.array([[0xFE]], dtype=np.uint8), np.array([1.0]), 1, ref.I8, 0).tolist() == [[-2.0]]


def test_plain_block_norm_by_hand():
    x = np.array([[3.0, 4.0]])
    r, _, y, _ = ref.block_norm(x, np.array([[1.0, 1.0]]), np.array([1.0, 0.5]), np.array([[1.0, 2.0]]), 2.0, np.array([1.0, 1.0]), 0.0)
    z = x / math.sqrt(12.5)
    want = np.array([[1 + 2 * z[0, 0], 1 + 2 * 2 * 0.5 * z[0, 1]]])
    assert np.allclose(r, want, rtol=1e-15)
    assert np.allclose(y, want / math.sqrt((want ** 2).mean()), rtol=1e-15)
