"""Calls with more work than one dimension of a launch holds (2^32 threads): they do all of it, or are refused.

Inputs are windows of one buffer (a row starts a few elements after the last), so that the rows all differ and the
memory stays small. Bounds are those of test_gpu_decoder.py: a norm's scale is within 38 u, codes and scales of the cache
are exact."""
from __future__ import annotations

import numpy as np
import pytest

import decoder_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

import gpu_util as gu  # noqa: E402
import weight_only_quantized_matmul_amd as wq  # noqa: E402

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def device():
    gu.reinit_with_env(WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None)
    yield
    torch.cuda.empty_cache()


def test_rope_of_many_tokens():
    T = (1 << 28) + 4099  # 16 tokens a block of 256 threads
    gu.banner("rope T=%d" % T)
    x = torch.ones((T, 1, 2), dtype=torch.float16, device="cuda")
    x[:, 0, 1] = 0
    pos = torch.arange(T, dtype=torch.int32, device="cuda")[None] % 3
    y = torch.full_like(x, 9.0)
    wq.wq_rope_dev(wq.wq_rope_create(2, 0, 1e4, [1]), x, pos, y)
    want = torch.tensor([[np.cos(p), np.sin(p)] for p in range(3)]).half().cuda()
    wrong = 0
    for first in range(0, T, 1 << 26):
        got = y[first:first + (1 << 26), 0]
        wrong += int(((got - want[pos[0, first:first + (1 << 26)].long()]).abs() > 2.0 ** -10).sum())
    assert wrong == 0


def test_norm_of_many_rows():
    rows, n = 6_200_000, 16392  # 704 threads a row
    gu.banner("norm %d x %d" % (rows, n))
    g = torch.Generator("cuda").manual_seed(1)
    buf = torch.randn(8 * rows + n, device="cuda", generator=g).bfloat16()
    x = buf.as_strided((rows, n), (8, 1))
    w = torch.ones(n, device="cuda")
    y = torch.empty((1, n), dtype=torch.int8, device="cuda").expand(rows, n)  # the scales are what is looked at
    sc = torch.full((rows,), float("nan"), device="cuda")
    wq.wq_rmsnorm_dev(x, w, 1e-6, y, y_scale=sc)
    torch.cuda.synchronize()
    assert not sc.isnan().any()
    for r in [0, 1, (1 << 32) // 704 - 1, (1 << 32) // 704, (1 << 32) // 704 + 1, rows - 1]:
        t = x[r].double()
        want = float(t.abs().max() / (t.square().mean() + 1e-6).sqrt() / 127)
        assert abs(float(sc[r]) - want) <= 38 * U * want, r


def test_append_of_many_tokens():
    """Keys that are not aligned for wide loads: 32 threads a row. All pages but the last are not there."""
    heads, D, page = 4, 256, 1 << 20
    T = (1 << 24) + 3
    gu.banner("append T=%d" % T)
    g = torch.Generator("cuda").manual_seed(2)
    buf = torch.randn(8 * T + heads * D + 8, device="cuda", generator=g).half()
    k, v = (buf.as_strided((T, heads, D), (8, D, 1), off) for off in (1, 3))
    pools = [torch.zeros((1, heads, page, D // 2), dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.zeros((1, heads, page), device="cuda") for _ in "kv"]
    cache = wq.KvCache(ref.I4, *pools, *scales)
    table = torch.full((1, 17), -1, dtype=torch.int32, device="cuda")
    table[0, 16] = 0
    start, lens = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, T], [T]))
    wq.wq_kv_append_dev(cache, wq.KvBatch(start, lens, table, T), k, v)
    torch.cuda.synchronize()
    for x, pool, sc in zip((k, v), pools, scales):
        rows, scale = ref.quantise(x[1 << 24:].float().cpu().numpy(), ref.I4)
        np.testing.assert_array_equal(pool[0, :, :3].cpu().numpy(), rows.transpose(1, 0, 2))
        np.testing.assert_array_equal(sc[0, :, :3].cpu().numpy(), scale.T)
        assert not pool[0, :, 3:].any() and not sc[0, :, 3:].any()


def test_attention_of_too_many_tiles_is_refused():
    B = 1 << 24  # a tile a sequence at least, 256 threads a tile
    start = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    start[-1] = 1
    lens, table = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    pools = [torch.zeros((1, 1, 16, 64), dtype=torch.uint8, device="cuda") for _ in "kv"]
    cache = wq.KvCache(ref.I8, *pools, *(torch.zeros((1, 1, 16), device="cuda") for _ in "kv"))
    q = torch.zeros((1, 1, 64), device="cuda")
    with pytest.raises(wq.WqError) as e:
        wq.wq_attn_paged_dev(cache, wq.KvBatch(start, lens, table, 1, max_q=1, max_kv=1), q, torch.empty_like(q), scale=1.0)
    assert e.value.code == wq.WQ_E_UNSUPPORTED


def far_context(new):
    """A context of 2^31 - 1 positions: one page of 2^20 slots, 2048 times."""
    page, D = 1 << 20, 64
    g = torch.Generator("cuda").manual_seed(7)
    pools = [torch.randint(0, 256, (1, 1, page, D // 2), dtype=torch.uint8, device="cuda", generator=g) for _ in "kv"]
    scales = [0.05 + 0.05 * torch.rand((1, 1, page), device="cuda", generator=g) for _ in "kv"]
    cache = wq.KvCache(ref.I4, *pools, *scales)
    start, lens = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, new], [(1 << 31) - 1]))
    batch = wq.KvBatch(start, lens, torch.zeros((1, 2048), dtype=torch.int32, device="cuda"), new, max_q=new, max_kv=(1 << 31) - 1)
    opened = [ref.open_rows(p.cpu().numpy()[0, 0], ref.I4) * s.cpu().numpy()[0, 0].astype(np.float64)[:, None] for p, s in zip(pools, scales)]
    q = torch.randn((new, 2, D), device="cuda", generator=g)
    return cache, batch, q, opened


@pytest.mark.parametrize("new,window", [(1, 100), (1, 5000), (9, 70), (90, 300), (300, 6000)])
def test_last_positions_before_2_to_the_31(new, window):
    gu.banner("window %d at position 2^31, %d new" % (window, new))
    cache, batch, q, (K, V) = far_context(new)
    o, l = torch.empty_like(q), torch.empty((new, 2), device="cuda")
    wq.wq_attn_paged_dev(cache, batch, q, o, scale=0.125, window=window, lse=l)
    o, l = o.double().cpu().numpy(), l.double().cpu().numpy()
    for i in range(new):
        p = (1 << 31) - 1 - new + i
        at = np.arange(p - window + 1, p + 1) % (1 << 20)
        for h in range(2):
            s = 0.125 * (K[at] @ q[i, h].double().cpu().numpy())
            w = np.exp(s - s.max())
            A = (w / w.sum()) @ np.abs(V[at])
            e = 72 * U * 0.125 * (np.abs(K[at]) @ np.abs(q[i, h].double().cpu().numpy())).max()
            assert (np.abs(o[i, h] - (w / w.sum()) @ V[at]) <= A * (2 * e + (window + 72) * U + 2.0 ** -21) + U * A).all(), i
            assert abs(l[i, h] - s.max() - np.log(w.sum())) <= e + (window + 72) * U + 30 * U, i


def test_all_positions_before_2_to_the_31():
    """Weights in fp32 sums: a split's chain is 2^31 / 512 positions, 32 or 64 a step and four waves, then the join."""
    gu.banner("attention over 2^31 - 1 positions")
    cache, batch, q, (K, V) = far_context(1)
    o, l = torch.empty_like(q), torch.empty((1, 2), device="cuda")
    wq.wq_attn_paged_dev(cache, batch, q, o, scale=0.125, lse=l)
    o, l = o.double().cpu().numpy(), l.double().cpu().numpy()
    n = np.full(1 << 20, 2048.0)
    n[-1] = 2047
    for h in range(2):
        s = 0.125 * (K @ q[0, h].double().cpu().numpy())
        w = n * np.exp(s - s.max())
        A = (w / w.sum()) @ np.abs(V)
        e = 72 * U * 0.125 * (np.abs(K) @ np.abs(q[0, h].double().cpu().numpy())).max()
        chain = (1 << 31) // 512 // 128 + 512
        assert (np.abs(o[0, h] - (w / w.sum()) @ V) <= A * (2 * e + 2 * chain * U + 2.0 ** -21)).all()
        assert abs(l[0, h] - s.max() - np.log(w.sum())) <= e + chain * U + 40 * U


def test_append_at_the_last_position():
    cache, batch, _, _ = far_context(1)
    k, v = (torch.randn((1, 1, 64), device="cuda", generator=torch.Generator("cuda").manual_seed(i)) for i in (1, 2))
    was = [t.clone() for t in cache.tensors]
    wq.wq_kv_append_dev(cache, batch, k, v)
    back = [torch.empty_like(k) for _ in "kv"]
    wq.wq_kv_read_dev(cache, batch, *back)
    for x, b, pool, sc, p0, s0 in zip((k, v), back, cache.tensors[:2], cache.tensors[2:], was[:2], was[2:]):
        rows, scale = ref.quantise(x.cpu().numpy(), ref.I4)
        p0[0, 0, (1 << 20) - 2], s0[0, 0, (1 << 20) - 2] = torch.from_numpy(rows[0, 0]).cuda(), float(scale[0, 0])
        assert torch.equal(pool, p0) and torch.equal(sc, s0)
        np.testing.assert_array_equal(b.cpu().numpy()[0, 0], (ref.open_rows(rows, ref.I4) * scale[..., None]).astype(np.float32)[0, 0])


@pytest.mark.parametrize("kv", [-1, -5, -(1 << 31)])
def test_negative_lengths_are_empty(kv):
    """No position is there: nothing is written, zeros are read, attention sees nothing."""
    cache, _, _, _ = far_context(1)
    start, lens = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, 2], [kv]))
    batch = wq.KvBatch(start, lens, torch.zeros((1, 2048), dtype=torch.int32, device="cuda"), 2)
    x, back, q = torch.ones((2, 1, 64), device="cuda"), torch.ones((2, 1, 64), device="cuda"), torch.ones((2, 2, 64), device="cuda")
    was = [t.clone() for t in cache.tensors]
    wq.wq_kv_append_dev(cache, batch, x, x)
    wq.wq_kv_read_dev(cache, batch, back, back)
    o, l = torch.ones_like(q), torch.ones((2, 2), device="cuda")
    wq.wq_attn_paged_dev(cache, batch, q, o, scale=0.1, lse=l)
    assert all(torch.equal(a, b) for a, b in zip(was, cache.tensors))
    assert not back.any() and not o.any() and (l == -float("inf")).all()


def test_numbers_past_a_c_int():
    """A window longer than any position is no window; negative and too large counts are refused, not taken modulo 2^32."""
    cache, batch, q, _ = far_context(1)
    lens = torch.tensor([3000], dtype=torch.int32, device="cuda")
    batch = wq.KvBatch(batch.tensors[0], lens, batch.tensors[2], 1, max_q=1 << 32, max_kv=(1 << 32) + 5)
    want = torch.empty_like(q)
    wq.wq_attn_paged_dev(cache, batch, q, want, scale=0.125)
    for window in ((1 << 31) - 1, 1 << 31, (1 << 32) + 1, 1 << 63):
        o = torch.empty_like(q)
        wq.wq_attn_paged_dev(cache, batch, q, o, scale=0.125, window=window)
        assert torch.equal(o, want), window
    for window in (-1, -(1 << 32)):
        with pytest.raises(wq.WqError) as e:
            wq.wq_attn_paged_dev(cache, batch, q, want, scale=0.125, window=window)
        assert e.value.code == wq.WQ_E_INVAL
    with pytest.raises(ValueError):
        wq.KvBatch(batch.tensors[0], lens, batch.tensors[2], (1 << 32) + 1)
    x = torch.ones((1, 4), device="cuda").expand((1 << 32) + 1, 4)
    with pytest.raises(ValueError):
        wq.wq_rmsnorm_dev(x, torch.ones(4, device="cuda"), 1e-6, x)
