"""The binding of the calls between a decoder layer's products and the plans of attention, without a GPU."""
from __future__ import annotations

import ctypes

import pytest

import weight_only_quantized_matmul_amd as wq


@pytest.mark.parametrize("rot,pairing,sections", [((1 << 32) + 8, 0, [4]), (8, 1 << 32, [4]), (8, 0, [(1 << 32) + 4]),
                                                  (8, 0, [5, -1 - (1 << 32)])])
def test_rope_create_takes_no_number_modulo_2_to_the_32(rot, pairing, sections):
    with pytest.raises(wq.WqError):
        wq.wq_rope_create(rot, pairing, 1e4, sections)


def test_c_ints():
    assert [wq._int(v) for v in (-1, 0, 7, (1 << 31) - 1, 1 << 31, 1 << 70, -2, -(1 << 40))] == [
        -1, 0, 7, (1 << 31) - 1, (1 << 31) - 1, (1 << 31) - 1, -1, -1]


P = 1 << 20


def describe(dtype, kind, D, heads, G, B, T, max_q, max_kv, page=64, causal=1, window=0, buf=256):
    rb = (2 * D, D, D // 2)[kind]
    c = wq._KvCacheC(15, kind, 4, heads, page, D, P, P, P, P, (ctypes.c_long * 3)(page * heads * rb, page * rb, rb),
                     (ctypes.c_long * 3)(page * heads, page, 1))
    width = -(-max_kv // page)
    b = wq._KvBatchC(B, T, width, max_q, max_kv, width, P, P, P)
    out = ctypes.create_string_buffer(256)
    return wq.lib.wq_describe_attn(ctypes.byref(c), ctypes.byref(b), dtype, heads * G, causal, window, out, buf), out.value.decode()


@pytest.mark.parametrize("args,want", [
    ((0, 1, 128, 8, 6, 1, 1, 1, 1500), "few rows=16 step=32 "),  # one token
    ((0, 1, 128, 8, 6, 4, 20, 5, 1500), "few rows=32 step=32 "),  # a few tokens
    ((1, 2, 64, 2, 8, 64, 64, 1, 3000), "join=1x4"),  # many rows, few splits
    ((0, 2, 64, 1, 4, 1, 1, 1, 30000), "join=4x8"),  # many splits
    ((1, 0, 128, 8, 4, 1, 4096, 4096, 4096), "tiled waves=8 rows=256 step=64 splits=1 "),  # a long prompt, 16-bit
    ((0, 1, 128, 8, 4, 1, 4096, 4096, 4096), "tiled waves=8 rows=128 step=64 splits=1 "),  # ... and f32
    ((2, 0, 256, 8, 4, 1, 4096, 4096, 4096), "tiled waves=8 rows=128 step=32 splits=1 "),
    ((1, 0, 64, 8, 4, 1, 4096, 4096, 4096), "tiled waves=4 rows=128 step=64 splits=1 "),  # rows of 64: four waves
    ((1, 0, 128, 8, 4, 1, 1024, 1024, 1024), "tiled waves=4 rows=128 "),  # a short prompt
])
def test_plans_of_attention(args, want):
    """On 256 CUs, which the plan takes where the device is not open (15 never is)."""
    rc, plan = describe(*args)
    assert rc == wq.WQ_OK and want in plan, plan


def test_plan_refusals():
    assert describe(0, 1, 128, 8, 6, 0, 0, 0, 1500) == (wq.WQ_OK, "none")
    assert describe(3, 1, 128, 8, 6, 1, 1, 1, 1500)[0] == wq.WQ_E_INVAL
    assert describe(0, 1, 128, 8, 0, 1, 1, 1, 1500)[0] == wq.WQ_E_INVAL
    assert describe(0, 1, 128, 8, 6, 1, 1, 1, 1500, window=-1)[0] == wq.WQ_E_INVAL
    assert describe(0, 1, 128, 8, 6, 1, 1, 1, 1500, buf=0)[0] == wq.WQ_E_INVAL
    assert describe(0, 1, 96, 8, 6, 1, 1, 1, 1500)[0] == wq.WQ_E_UNSUPPORTED
