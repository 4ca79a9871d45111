"""Refusals of the calls between a decoder layer's products: checked before any device is touched."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

import decoder_ref as ref
import weight_only_quantized_matmul_amd as wq

P = 1 << 20  # a 16-byte aligned address that no refused call may touch


def norm(**kw):
    a = dict(device=0, x=P, xd=0, xs=64, res=None, rs=0, w=P, eps=1e-6, rows=2, n=64, y=P, yd=0, ys=64, sc=None, sum=None, ss=0)
    a.update(kw)
    return wq.lib.wq_rmsnorm_dev(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(w=None), dict(y=None), dict(rows=-1), dict(n=0), dict(n=-3), dict(xd=3), dict(xd=7), dict(yd=4),
    dict(yd=3), dict(sc=P), dict(eps=-1.0), dict(eps=math.nan), dict(xs=-1), dict(ys=-1), dict(res=P, rs=-1),
    dict(sum=P, ss=-1), dict(x=P + 2), dict(w=P + 1), dict(y=P + 2), dict(res=P + 2), dict(sum=P + 1)])
def test_norm_refuses(bad):
    assert norm(**bad) == wq.WQ_E_INVAL


def test_norm_limits():
    assert norm(n=wq.WQ_NORM_MAX_N + 1) == wq.WQ_E_UNSUPPORTED
    assert norm(rows=0) == wq.WQ_OK
    assert norm(device=15) == wq.WQ_E_NOTINIT
    assert norm(device=-1) == wq.WQ_E_NOTINIT


def rope_create(rot, pairing, theta, sections):
    h = ctypes.c_void_p(None)
    arr = (ctypes.c_int * max(1, len(sections)))(*sections)
    return wq.lib.wq_rope_create(rot, pairing, theta, arr, len(sections), ctypes.byref(h)), h


@pytest.mark.parametrize("args", [(0, 0, 1e4, [0]), (7, 0, 1e4, [3]), (8, 2, 1e4, [4]), (8, 0, 0.0, [4]), (8, 0, math.inf, [4]),
                                  (8, 0, math.nan, [4]), (8, 0, 1e4, [3]), (8, 0, 1e4, [5, -1]), (8, 0, 1e4, []), (-2, 0, 1e4, [-1])])
def test_rope_create_refuses(args):
    assert rope_create(*args)[0] == wq.WQ_E_INVAL


def test_rope_limits():
    assert rope_create(258, 0, 1e4, [129])[0] == wq.WQ_E_UNSUPPORTED
    assert rope_create(18, 0, 1e4, [1] * 9)[0] == wq.WQ_E_UNSUPPORTED
    rc, h = rope_create(256, 1, 1e6, [60, 0, 68])
    assert rc == wq.WQ_OK

    def run(**kw):
        a = dict(h=h, device=15, x=P, dt=0, T=1, H=1, D=256, xt=256, xh=256, pos=P, ps=1, y=P, yt=256, yh=256)
        a.update(kw)
        return wq.lib.wq_rope_dev(*a.values(), None)

    for bad in (dict(h=None), dict(x=None), dict(y=None), dict(pos=None), dict(dt=3), dict(T=-1), dict(H=-1), dict(D=255),
                dict(xt=-1), dict(yh=-1), dict(ps=-1), dict(x=P + 2), dict(pos=P + 2)):
        assert run(**bad) == wq.WQ_E_INVAL
    assert run(H=wq.WQ_KV_MAX_HEADS + 1) == wq.WQ_E_UNSUPPORTED
    assert run(T=0) == wq.WQ_OK
    assert run() == wq.WQ_E_NOTINIT
    assert wq.lib.wq_rope_free(h) == wq.WQ_OK
    assert wq.lib.wq_rope_free(None) == wq.WQ_OK
    r = wq.wq_rope_create(64, 0, 1e4, [32])
    wq.wq_rope_free(r)
    with pytest.raises(wq.WqError):
        wq.wq_rope_create(64, 0, 1e4, [31])


def cache(**kw):
    a = dict(device=15, kind=1, pages=4, heads=2, page=16, dim=64, k=P, v=P, k_scale=P, v_scale=P,
             row_stride=(2048, 1024, 64), scale_stride=(32, 16, 1))
    a.update(kw)
    a["row_stride"], a["scale_stride"] = (ctypes.c_long * 3)(*a["row_stride"]), (ctypes.c_long * 3)(*a["scale_stride"])
    return wq._KvCacheC(*a.values())


def batch(**kw):
    a = dict(B=1, T=1, width=4, max_q=0, max_kv=0, table_stride=4, q_start=P, kv_len=P, table=P)
    a.update(kw)
    return wq._KvBatchC(*a.values())


def calls(c, b, dt=0, p=P, tok=128, head=64):
    c, b = (None if x is None else ctypes.byref(x) for x in (c, b))
    return (wq.lib.wq_kv_append_dev(c, b, p, P, dt, tok, head, None), wq.lib.wq_kv_read_dev(c, b, P, p, dt, tok, head, None),
            wq.lib.wq_attn_paged_dev(c, b, p, dt, 4, tok, head, 0.125, 1, 0, P, tok, head, None, None))


@pytest.mark.parametrize("bad", [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(kind=3), dict(kind=-1),
                                 dict(pages=0), dict(heads=0), dict(page=0), dict(dim=0), dict(k=P + 8), dict(k_scale=P + 2),
                                 dict(row_stride=(2048, 1024, 8)), dict(row_stride=(-16, 16, 16)), dict(scale_stride=(1, -1, 1))])
def test_cache_refuses(bad):
    assert set(calls(cache(**bad), batch())) == {wq.WQ_E_INVAL}


@pytest.mark.parametrize("bad", [dict(B=-1), dict(T=-1), dict(width=-1), dict(max_q=-1), dict(max_kv=-1), dict(table_stride=-1),
                                 dict(B=0), dict(q_start=None), dict(kv_len=None), dict(table=None), dict(q_start=P + 2)])
def test_batch_refuses(bad):
    assert set(calls(cache(), batch(**bad))) == {wq.WQ_E_INVAL}


def test_cache_calls_limits():
    assert set(calls(None, batch())) == {wq.WQ_E_INVAL}
    assert set(calls(cache(), None)) == {wq.WQ_E_INVAL}
    for dim in (32, 80, 96, 512):
        assert set(calls(cache(dim=dim), batch())) == {wq.WQ_E_UNSUPPORTED}
    assert set(calls(cache(heads=1025), batch())) == {wq.WQ_E_UNSUPPORTED}
    assert set(calls(cache(), batch(B=0, T=0))) == {wq.WQ_OK}
    assert set(calls(cache(), batch(), dt=3)) == {wq.WQ_E_INVAL}
    assert set(calls(cache(), batch(), p=None)) == {wq.WQ_E_INVAL}
    assert set(calls(cache(), batch(), p=P + 2)) == {wq.WQ_E_INVAL}
    assert set(calls(cache(), batch(), tok=-1)) == {wq.WQ_E_INVAL}
    assert set(calls(cache(), batch())) == {wq.WQ_E_NOTINIT}


@pytest.mark.parametrize("H,scale,window", [(0, 0.1, 0), (3, 0.1, 0), (4, math.nan, 0), (4, math.inf, 0), (4, 0.1, -1)])
def test_attention_refuses(H, scale, window):
    c, b = cache(), batch()
    assert wq.lib.wq_attn_paged_dev(ctypes.byref(c), ctypes.byref(b), P, 0, H, 64, 64, scale, 1, window, P, 64, 64, None,
                                    None) == wq.WQ_E_INVAL


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        wq.wq_rmsnorm_dev(x, torch.ones(64), 1e-6, x)
    with pytest.raises(TypeError):
        wq.wq_rmsnorm_dev(x.numpy(), torch.ones(64), 1e-6, x)
    r = wq.wq_rope_create(64, 0, 1e4, [32])
    with pytest.raises(ValueError):
        wq.wq_rope_dev(r, x[:, None], torch.zeros(1, 2, dtype=torch.int32), x[:, None])
    pool, sc = torch.zeros(1, 1, 16, 64, dtype=torch.uint8), torch.zeros(1, 1, 16)
    with pytest.raises(ValueError):
        wq.KvCache(wq.WQ_KV_I8, pool, pool, sc, sc)
    with pytest.raises(ValueError):
        wq.KvCache(5, pool, pool, sc, sc)
    with pytest.raises(ValueError):
        wq.KvBatch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32), 0)


# ---------------------------------------------------------------------------------------
# the 64-bit references themselves, and where a position lies


def test_pages_that_are_not_there():
    table = np.array([[3, -1, 9, 2]], dtype=np.int32)
    got = [ref.place_at(table, 4, 16, 0, t) for t in (0, 15, 16, 31, 32, 48, 63, 64, -1)]
    assert got == [(3, 0), (3, 15), None, None, None, (2, 0), (2, 15), None, None]


def test_reference_formats():
    x = np.array([[1.0, -2.0, 0.5, 7.0], [0, 0, 0, 0], [1, np.nan, 0, 0], [2.0 ** -101, 0, 0, 0]], dtype=np.float32)
    for kind, want in ((ref.I8, [18, -36, 9, 127]), (ref.I4, [1, -2, 0, 7])):
        rows, scale = ref.quantise(x, kind)
        codes = ref.open_rows(rows, kind)
        assert codes[0].tolist() == want and (codes[1:] == 0).all()
        assert scale[0] == np.float32(7 / (127 if kind == ref.I8 else 7)) and scale[1] == 0 and np.isnan(scale[2]) and scale[3] == 0
    rows, scale = ref.quantise(x, ref.F16)
    assert (ref.open_rows(rows, ref.F16)[0] * scale[0] == x[0]).all() and scale[0] == 2.0 ** -12


def test_reference_attention_against_a_second_form():
    rng = np.random.default_rng(5)
    q = rng.normal(size=(3, 2, 64))
    k, v = (rng.integers(0, 256, (3, 1, 4, 64), dtype=np.uint8) for _ in "kv")
    ks, vs = (rng.uniform(0.01, 0.02, (3, 1, 4)).astype(np.float32) for _ in "kv")
    table = np.array([[2, 0]], dtype=np.int32)
    o, lse, _, _ = ref.attention(q, ref.I8, k, v, ks, vs, [0, 3], [7], table, 0.1, True, 3)
    K, V = (np.concatenate([x[2, 0], x[0, 0]])[:7].view(np.int8).astype(float) * np.concatenate([s[2, 0], s[0, 0]])[:7, None].astype(float)
            for x, s in ((k, ks), (v, vs)))
    for i in range(3):
        for h in range(2):
            z = [0.1 * float(K[t] @ q[i, h]) for t in range(4 + i - 2, 4 + i + 1)]
            den = sum(math.exp(a) for a in z)
            want = sum(math.exp(a) / den * V[t] for a, t in zip(z, range(2 + i, 5 + i)))
            assert np.abs(o[i, h] - want).max() < 1e-12 and abs(lse[i, h] - math.log(den)) < 1e-12
