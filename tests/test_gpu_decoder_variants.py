"""The kernel variants that large sizes take, against 64 bits on the same GPU with elementary operations: eight-wave tiles,
the join with one wave a row and beyond 64 splits, cache rows four a lane group, the norm's row-walking form.

Bounds as in test_gpu_decoder.py. Each test first asks for the plan (wq_describe_attn), or derives the size from the
device's CU count, so that it keeps reaching the variant it is named after."""
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
from test_gpu_decoder import DT, HALF, SMALL, U, f64, guarded, check_guard  # noqa: E402

CODE = {"f32": wq.WQ_DT_F32, "bf16": wq.WQ_DT_BF16, "f16": wq.WQ_DT_F16}
CUS = torch.cuda.get_device_properties(0).multi_processor_count


@pytest.fixture(scope="module", autouse=True)
def device():
    gu.reinit_with_env(WQ_FORCE_PATH=None, WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None)
    yield
    torch.cuda.empty_cache()


class Context:
    """A written cache of B sequences and a batch of their last tokens; pages in no order, one table entry missing."""

    def __init__(self, seed, kind, D, heads, q_len, kv_len, page=64, missing=None):
        self.kind, self.D, self.heads, self.page, self.q_len, self.kv_len = kind, D, heads, page, q_len, kv_len
        g = torch.Generator("cuda").manual_seed(seed)
        need = [-(-n // page) for n in kv_len]
        pages, width = sum(need) + 2, max(need)
        order = torch.randperm(pages, device="cuda", generator=g)[: sum(need)].to(torch.int32)
        self.table = torch.full((len(kv_len), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        if missing is not None:
            self.table[missing] = -1
        shape = (pages, heads, page)
        if kind == ref.F16:
            self.codes = [torch.randn(shape + (D,), device="cuda", generator=g).mul_(8000).clamp_(-32000, 32000).half() for _ in "kv"]
            pools = [c.view(torch.uint8) for c in self.codes]
        elif kind == ref.I8:
            self.codes = [torch.randint(-127, 128, shape + (D,), device="cuda", generator=g, dtype=torch.int8) for _ in "kv"]
            pools = [c.view(torch.uint8) for c in self.codes]
        else:
            self.codes = [torch.randint(-7, 8, shape + (D,), device="cuda", generator=g, dtype=torch.int8) for _ in "kv"]
            n = [(c + 8).to(torch.uint8) for c in self.codes]
            pools = [x[..., 0::2] | (x[..., 1::2] << 4) for x in n]
        unit = (1 / 8000, 1 / 60, 1 / 4)[kind]
        self.scales = [(0.5 + torch.rand(shape, device="cuda", generator=g)) * unit for _ in "kv"]
        self.cache = wq.KvCache(kind, *pools, *self.scales)
        self.T = sum(q_len)
        start = torch.tensor([0] + list(np.cumsum(q_len)), dtype=torch.int32, device="cuda")
        self.batch = wq.KvBatch(start, torch.tensor(kv_len, dtype=torch.int32, device="cuda"), self.table, self.T,
                                max_q=max(q_len), max_kv=max(kv_len))
        self.g = g

    def queries(self, H, dtype):
        return torch.randn((self.T, H, self.D), device="cuda", generator=self.g).to(DT[dtype])

    def check(self, q, dtype, causal=True, window=0):
        H, G, scale = q.shape[1], q.shape[1] // self.heads, self.D ** -0.5
        obuf, o = guarded(q.shape, DT[dtype])
        lbuf, l = guarded(q.shape[:2], torch.float32)
        wq.wq_attn_paged_dev(self.cache, self.batch, q, o, scale=scale, causal=causal, window=window, lse=l)
        torch.cuda.synchronize()
        check_guard(obuf), check_guard(lbuf)
        o2, l2 = torch.empty_like(o), torch.empty_like(l)
        wq.wq_attn_paged_dev(self.cache, self.batch, q, o2, scale=scale, causal=causal, window=window, lse=l2)
        assert torch.equal(o, o2) and torch.equal(l, l2), "two runs differ"
        r = 2.0 ** -21 if dtype == "f32" else 2 * 2.0 ** -11
        first = 0
        for b, (n, kv) in enumerate(zip(self.q_len, self.kv_len)):
            t = torch.arange(kv, device="cuda")
            page, slot = self.table[b].long()[t // self.page], t % self.page
            p = kv - n + torch.arange(n, device="cuda")[:, None]
            seen = (page >= 0)[None, :].expand(n, kv)
            if causal:
                seen = seen & (t[None, :] <= p)
            if window:
                seen = seen & (t[None, :] > p - window)
            page = page.clamp(min=0)
            for h in range(H):
                K, V = (c[page, h // G, slot].double() * s[page, h // G, slot].double()[:, None] for c, s in zip(self.codes, self.scales))
                x = q[first:first + n, h].double()
                z = (x @ K.t().contiguous()) * scale
                S = (x.abs() @ K.t().contiguous().abs() * scale).where(seen, torch.zeros((), dtype=torch.float64, device="cuda")).amax(1)
                z = z.where(seen, torch.full((), -float("inf"), dtype=torch.float64, device="cuda"))
                lse = torch.logsumexp(z, 1)
                w = (z - lse[:, None]).exp().where(seen, torch.zeros((), dtype=torch.float64, device="cuda"))
                want, A = w @ V, w @ V.abs()
                e = (self.D + 8) * U * S
                tol = A * (2 * e + (kv + 72) * U + r)[:, None] + 1.01 * HALF[dtype] * want.abs() + SMALL[dtype]
                err = (o[first:first + n, h].double() - want).abs()
                assert (err <= tol).all(), "sequence %d head %d: worst %.3g of the bound" % (b, h, float((err / tol).max()))
                none = ~seen.any(1)
                got = l[first:first + n, h].double()
                assert (got[none] == -float("inf")).all()
                assert ((got - lse).abs() <= e + (kv + 72) * U + U * lse.abs() + U)[~none].all()
            first += n


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", [ref.F16, ref.I8, ref.I4])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 333), (False, 0)])
def test_eight_wave_tiles(dtype, kind, D, causal, window):
    if not causal and (kind != ref.I8 or D == 256):
        causal = True
    c = Context(D + kind, kind, D, 8, [1030, 3, 1003], [1500, 3, 1003], missing=(0, 5))
    plan = wq.wq_describe_attn(c.cache, c.batch, CODE[dtype], 32, causal, window)
    gu.banner("%s kind=%d D=%d causal=%d window=%d: %s" % (dtype, kind, D, causal, window, plan))
    assert plan.startswith("tiled waves=8 "), plan
    c.check(c.queries(32, dtype), dtype, causal, window)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind,D,heads,G,B,kv", [(ref.I8, 64, 2, 8, 64, 3000), (ref.F16, 128, 2, 8, 65, 1500), (ref.I4, 256, 1, 16, 70, 2000)])
def test_join_with_one_wave_a_row(dtype, kind, D, heads, G, B, kv):
    lens = [max(1, kv - 37 * i) for i in range(B)]
    c = Context(B, kind, D, heads, [1] * B, lens)
    plan = wq.wq_describe_attn(c.cache, c.batch, CODE[dtype], heads * G)
    gu.banner("%s kind=%d D=%d: %s" % (dtype, kind, D, plan))
    assert "join=1x4" in plan, plan
    c.check(c.queries(heads * G, dtype), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("q_len,kv", [([1], 30000), ([1, 1], 60000), ([70], 30000)])
def test_join_beyond_64_splits(dtype, q_len, kv):
    c = Context(kv, ref.I4, 64, 1, q_len, [kv - 1000 * i for i in range(len(q_len))])
    plan = wq.wq_describe_attn(c.cache, c.batch, CODE[dtype], 4)
    gu.banner("%s q=%s kv=%d: %s" % (dtype, q_len, kv, plan))
    assert int(plan.split("splits=")[1].split()[0]) > 64 and "join=4x8" in plan, plan
    c.check(c.queries(4, dtype), dtype)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", [ref.F16, ref.I8, ref.I4])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cache_rows_four_a_lane_group(dtype, kind, D):
    """10 rows a token: the last lane group of a token holds two."""
    heads, page = 5, 64
    T = (1 << 20) // (2 * heads * (D // 8)) + 33
    q_len = [T // 3, 0, T - T // 3]
    kv_len = [q_len[0] + 100, 7, q_len[2]]
    gu.banner("cache %s kind=%d D=%d T=%d" % (dtype, kind, D, T))
    c = Context(T, kind, D, heads, q_len, kv_len, page)
    was = [t.clone() for t in c.cache.tensors]
    new = [torch.randn((T, heads, D), device="cuda", generator=c.g).to(DT[dtype]) for _ in "kv"]
    new[0][5, 3] = 0
    new[1][T - 1, 4, 7] = float("nan")
    wq.wq_kv_append_dev(c.cache, c.batch, *new)
    b = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(q_len, device="cuda"))
    start = torch.tensor([0, q_len[0], q_len[0]], device="cuda")
    p = torch.tensor(kv_len, device="cuda")[b] - torch.tensor(q_len, device="cuda")[b] + torch.arange(T, device="cuda") - start[b]
    pg, slot = c.table.long()[b, p // page], p % page
    out = [torch.empty((T, heads, D), dtype=DT[dtype], device="cuda") for _ in "kv"]
    wq.wq_kv_read_dev(c.cache, c.batch, *out)
    for side in range(2):
        rows, scales = ref.quantise(new[side].float().cpu().numpy(), kind)
        was[side][pg, :, slot], was[2 + side][pg, :, slot] = torch.from_numpy(rows).cuda(), torch.from_numpy(scales).cuda()
        assert torch.equal(c.cache.tensors[side], was[side])
        assert torch.equal(c.cache.tensors[2 + side].nan_to_num(nan=-1.0), was[2 + side].nan_to_num(nan=-1.0))
        want = torch.from_numpy(ref.open_rows(rows, kind).astype(np.float32) * scales[..., None]).to(DT[dtype])
        np.testing.assert_array_equal(out[side].float().cpu().numpy(), want.float().numpy())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("out", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("n", [256, 1000, 1001, 2048, 2055, 4096, 6144, 8192])
def test_norm_walking_rows(dtype, out, n):
    """At least three rows a block: 16 waves a CU, blocks of at least 64 threads with at most four loads each."""
    vec = 4 if dtype == "f32" else 8
    chunks = -(-n // vec)
    threads = min(-(-(-(-chunks // k)) // 64) * 64 for k in (1, 2, 3, 4) if -(-chunks // k) <= 512)
    rows = 3 * CUS * (1024 // threads) + 7
    if n <= 1001:
        rows = 3 * CUS * 16 + 7
    gu.banner("norm %s -> %s %d x %d" % (dtype, out, rows, n))
    g = torch.Generator("cuda").manual_seed(n)
    x, r = (torch.randn((rows, n), device="cuda", generator=g).to(DT[dtype]) for _ in range(2))
    x[7], r[7] = 0, 0
    w = 1 + 0.2 * torch.randn(n, device="cuda", generator=g)
    ybuf, y = guarded((rows, n), torch.int8 if out == "i8" else DT[out])
    sbuf, s = guarded((rows, n), DT[dtype])
    sc = torch.full((rows,), 5.0, device="cuda") if out == "i8" else None
    wq.wq_rmsnorm_dev(x, w, 1e-6, y, residual=r, sum_out=s, y_scale=sc)
    torch.cuda.synchronize()
    check_guard(ybuf), check_guard(sbuf)
    t = x.float() + r.float()
    assert torch.equal(s, t.to(DT[dtype]))
    for first in range(0, rows, 4096):
        z = t[first:first + 4096].double()
        want = z / (z.square().mean(1, keepdim=True) + float(np.float32(1e-6))).sqrt() * w.double()
        if out == "i8":
            tw = z * w.double()
            top = tw.abs().amax(1, keepdim=True)
            assert torch.equal(y[first:first + 4096].double(), (tw * 127 / top.where(top > 0, torch.ones_like(top))).round())
            scale = want.abs().amax(1) / 127
            assert ((sc[first:first + 4096].double() - scale).abs() <= 38 * U * scale).all()
        else:
            assert ((y[first:first + 4096].double() - want).abs() <= (36 * U + 1.01 * HALF[out]) * want.abs() + SMALL[out]).all()
    if out == dtype:  # results over their inputs, while a block's next row is on its way
        wq.wq_rmsnorm_dev(x, w, 1e-6, x, residual=r, sum_out=r)
        assert torch.equal(x, y) and torch.equal(r, s)
