"""The norm, rotary positions, the quantised cache and attention over it on the GPU, against 64-bit references.

Tolerances are bounds of the arithmetic, derived before the first run; u = 2^-24 is half a step of fp32 and h(t) half a
step of the output type (bf16 2^-8, fp16 2^-11), relative to the value.

norm: the fp32 sum of n <= 32768 squares has a chain of at most 32 + 6 + 16 additions a path, so 1/sqrt(mean) is within
  28 u + 4 u; r * rstd * w adds 2 u: 36 u in all, then h(t).
rope: fp32 sine and cosine of an argument rounded once (2 u) and evaluated to 2 ulp (4 u), a product and a sum (2 u each):
  within 8 u (|a| + |b|), then h(t).
cache: codes, scales and values are exact by definition.
attention: S = max_t sum_d |scale q_d k_td|. A score has D fp32 additions in any order, the split of q (2 u), the scales
  and the exponent's argument (6 u): e = (D + 8) u S; a weight is within 2 e + 8 u of its own size; sums over kv positions,
  rescales and the joining of splits add (kv + 64) u. With A = sum_t w_t |v_t|: |o - o_ref| <= A (2 e + (kv + 72) u + r)
  + h(t) |o|, r = 2 * 2^-11 for 16-bit types (probabilities rounded to fp16) and 2^-21 for f32 (two fp16 parts).
"""
from __future__ import annotations

import ctypes

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
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": U, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALL = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -25}  # half a step next to zero
KINDS = [ref.F16, ref.I8, ref.I4]


@pytest.fixture(scope="module", autouse=True)
def device():
    gu.reinit_with_env(WQ_FORCE_PATH=None, WQ_GEMV_MAX_S=None, WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None,
                       WQ_TILED_MODE=None, WQ_TILED_SHAPE=None, WQ_WAVES_PER_CU=None)
    yield


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def guarded(shape, dtype):
    """(buffer, view): the view stands among 64 elements of a pattern that check_guard() wants back."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), 77, dtype=dtype, device="cuda")
    return buf, buf[64:64 + n].view(shape)


def check_guard(buf):
    assert (buf[:64] == 77).all() and (buf[-64:] == 77).all(), "write outside the output"


# ---------------------------------------------------------------------------------------
# norm


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("out", ["f32", "bf16", "f16", "i8"])
@pytest.mark.parametrize("rows,n,res", [(1, 1, True), (3, 64, False), (2, 777, True), (5, 6144, True), (700, 1000, True),
                                        (600, 2048, False), (1, 32768, True), (2, 20001, True), (520, 12288, True)])
def test_norm(dtype, out, rows, n, res):
    gu.banner("norm %s -> %s rows=%d n=%d res=%d" % (dtype, out, rows, n, res))
    rng = np.random.default_rng(rows * 7 + n)
    x = cuda(rng.normal(size=(rows, n)).astype(np.float32), DT[dtype])
    r = cuda(2 * rng.normal(size=(rows, n)).astype(np.float32), DT[dtype]) if res else None
    w = cuda((1 + 0.2 * rng.normal(size=n)).astype(np.float32))
    if rows > 2:
        x[1] = 0
        if res:
            r[1] = 0
    ybuf, y = guarded((rows, n), torch.int8 if out == "i8" else DT[out])
    sbuf, s = guarded((rows, n), DT[dtype])
    sc = torch.full((rows,), 5.0, device="cuda") if out == "i8" else None
    wq.wq_rmsnorm_dev(x, w, 1e-6, y, residual=r, sum_out=s, y_scale=sc)
    torch.cuda.synchronize()
    check_guard(ybuf), check_guard(sbuf)
    t = (x.float() + (0 if r is None else r.float())).cpu()  # a 32-bit value by definition
    assert torch.equal(s.cpu(), t.to(DT[dtype]))
    t, w64 = t.double().numpy(), f64(w)
    want = t / np.sqrt((t * t).mean(1, keepdims=True) + 1e-6) * w64
    if out == "i8":
        tw = t * w64
        top = np.abs(tw).max(1, keepdims=True)
        codes = np.rint(tw * 127 / np.where(top == 0, 1, top))
        assert np.array_equal(y.cpu().numpy(), codes)
        scale = np.abs(want).max(1) / 127
        assert (np.abs(f64(sc) - scale) <= 38 * U * scale).all()
    else:
        assert (np.abs(f64(y) - want) <= (36 * U + 1.01 * HALF[out]) * np.abs(want) + SMALL[out]).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_norm_strides_and_places(dtype):
    """Rows of a wider buffer, misaligned rows, and sums and results over their inputs give the same bits."""
    rng = np.random.default_rng(11)
    rows, n = 9, 512
    x = cuda(rng.normal(size=(rows, n)).astype(np.float32), DT[dtype])
    r = cuda(rng.normal(size=(rows, n)).astype(np.float32), DT[dtype])
    w = cuda(rng.normal(size=n).astype(np.float32))
    y, s = torch.empty_like(x), torch.empty_like(x)
    wq.wq_rmsnorm_dev(x, w, 1e-5, y, residual=r, sum_out=s)
    for shift, width in ((8, 1024), (3, 531)):
        gu.banner("norm strides %s shift=%d" % (dtype, shift))
        big = torch.full((4, rows, width), 7.0, dtype=DT[dtype], device="cuda")
        a, b, c, d = (big[i, :, shift:shift + n] for i in range(4))
        a.copy_(x), b.copy_(r)
        wq.wq_rmsnorm_dev(a, w, 1e-5, c, residual=b, sum_out=d)
        tol = 0 if shift == 8 else 2.02 * (36 * U + HALF[dtype])  # the other path adds in another order
        assert torch.equal(d, s) and (np.abs(f64(c) - f64(y)) <= tol * np.abs(f64(y))).all()
        big[2:, :, shift:shift + n] = 7.0
        assert (big[:, :, :shift] == 7).all() and (big[2:] == 7).all() and (big[:, :, shift + n:] == 7).all()
    r2, x2 = r.clone(), x.clone()
    wq.wq_rmsnorm_dev(x2, w, 1e-5, x2, residual=r2, sum_out=r2)
    torch.cuda.synchronize()
    assert torch.equal(x2, y) and torch.equal(r2, s)


def test_norm_not_finite_rows():
    x = torch.ones(4, 100, device="cuda")
    x[1, 5], x[2, 7] = float("inf"), float("nan")
    y, sc = torch.full((4, 100), 9, dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    wq.wq_rmsnorm_dev(x, torch.ones(100, device="cuda"), 0.0, y, y_scale=sc)
    assert sc[[1, 2]].isnan().all() and (y[[1, 2]] == 0).all() and (y[[0, 3]] == 127).all() and sc[[0, 3]].isfinite().all()


def test_norm_tiny_and_large_rows_keep_their_codes():
    rng = np.random.default_rng(3)
    base = rng.normal(size=(1, 300)).astype(np.float32)
    for e in (-60, -126, 60, 100):
        x = cuda(np.ldexp(base, e).astype(np.float32))
        w = cuda(np.full(300, np.ldexp(1.0, -20 if e < 0 else 20), dtype=np.float32))
        y, sc = torch.empty((1, 300), dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
        wq.wq_rmsnorm_dev(x, w, 0.0, y, y_scale=sc)
        t = f64(x) * f64(w)
        if np.abs(t).max() > 2.0 ** -126:
            assert np.array_equal(y.cpu().numpy(), np.rint(t * 127 / np.abs(t).max())), e


# ---------------------------------------------------------------------------------------
# rotary positions


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("T,H,D,rot,sections", [(1, 1, 64, 64, [32]), (5, 3, 128, 128, [40, 24]), (3, 7, 128, 64, [8, 12, 12]),
                                                (70, 2, 256, 256, [32, 32, 32, 32]), (2, 3, 10, 6, [1, 0, 2]), (9, 64, 64, 64, [32]),
                                                (3000, 1, 64, 32, [16])])
def test_rope(dtype, pairing, T, H, D, rot, sections):
    gu.banner("rope %s pairing=%d T=%d H=%d D=%d rot=%d %s" % (dtype, pairing, T, H, D, rot, sections))
    rng = np.random.default_rng(T + H + D + rot)
    x = cuda(rng.normal(size=(T, H, D)).astype(np.float32), DT[dtype])
    pos = rng.integers(0, 2_000_000, (len(sections), T)).astype(np.int32)
    pos[:, :1] = 0 if T > 1 else 1_999_999
    if T > 2:
        pos[0, 2] = -5
    h = wq.wq_rope_create(rot, pairing, 1e6, sections)
    buf, y = guarded((T, H, D), DT[dtype])
    wq.wq_rope_dev(h, x, cuda(pos), y)
    torch.cuda.synchronize()
    check_guard(buf)
    x64 = f64(x)
    want = ref.rope(x64, pos, rot, pairing, 1e6, sections)
    mag = np.zeros_like(x64)
    i = np.arange(rot // 2)
    a, b = (i, i + rot // 2) if pairing == 0 else (2 * i, 2 * i + 1)
    mag[..., a] = mag[..., b] = np.abs(x64[..., a]) + np.abs(x64[..., b])
    assert (np.abs(f64(y) - want) <= 8 * U * mag + 1.01 * HALF[dtype] * np.abs(want) + SMALL[dtype]).all()
    assert np.array_equal(f64(y)[..., rot:], x64[..., rot:])
    wide = torch.full((T, H * D + 24), 3.0, dtype=DT[dtype], device="cuda")  # queries inside a fused projection, turned in place
    for off in (8, 5):
        wide.fill_(3.0)
        v = wide[:, off:off + H * D].unflatten(1, (H, D))
        v.copy_(x)
        wq.wq_rope_dev(h, v, cuda(pos), v)
        assert torch.equal(v, y)
        assert (wide[:, :off] == 3).all() and (wide[:, off + H * D:] == 3).all()


# ---------------------------------------------------------------------------------------
# the cache


class Case:
    """Pools, a page table and a batch. Slots that no sequence owns hold NaN scales and 0xff bytes (NaN as halves)."""

    def __init__(self, seed, kind, D, heads, page, q_len, kv_len, fill=True, slots_first=False, extra=0, spare=2, width=None):
        rng = np.random.default_rng(seed)
        self.rng, self.kind, self.D, self.heads, self.page = rng, kind, D, heads, page
        self.kv_len = np.array(kv_len, dtype=np.int32)
        self.q_start = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        self.T = int(self.q_start[-1])
        self.pages, self.table = ref.paging(rng, kv_len, page, spare, width)
        rb = ref.row_bytes(kind, D)
        self.pools, self.scales = [], []
        for _ in "kv":
            rows = np.full((self.pages, heads, page, rb), 255, dtype=np.uint8)
            sc = np.full((self.pages, heads, page), np.nan, dtype=np.float32)
            if fill:
                for b, n in enumerate(kv_len):
                    for t in range(n):
                        at = ref.place_at(self.table, self.pages, page, b, t)
                        if at is not None:
                            rows[at[0], :, at[1]], sc[at[0], :, at[1]] = ref.quantise(rng.normal(size=(heads, D)) * rng.uniform(0.5, 2), kind)
            self.pools.append(rows), self.scales.append(sc)
        # strides: pages further apart than they need, or slots outside heads
        self.dev = []
        for a in self.pools + self.scales:
            if slots_first:
                t = cuda(np.moveaxis(a, 1, 2)).transpose(1, 2)
            else:
                t = torch.zeros((self.pages, 1 + extra) + a.shape[1:], dtype=torch.from_numpy(a).dtype, device="cuda")[:, 0]
                t.copy_(torch.from_numpy(a))
            self.dev.append(t)
        self.cache = wq.KvCache(kind, *self.dev)
        self.batch = wq.KvBatch(cuda(self.q_start), cuda(self.kv_len), cuda(self.table), self.T)

    def host(self):
        """The pools as they are on the GPU now."""
        return [t.cpu().numpy() for t in self.dev]


LENS = [([1], [1]), ([1, 1, 1], [17, 33, 5]), ([5, 0, 3, 16], [5, 0, 40, 16]), ([0, 2, 1], [9, 1, 64]), ([33], [70])]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads,page,lens", [(1, 16, LENS[0]), (5, 16, LENS[1]), (2, 7, LENS[2]), (3, 64, LENS[3]), (1, 1, LENS[4])])
def test_append_and_read(dtype, kind, D, heads, page, lens):
    gu.banner("append %s kind=%d D=%d heads=%d page=%d %s" % (dtype, kind, D, heads, page, lens))
    c = Case(D + kind, kind, D, heads, page, lens[0], lens[1], fill=False, slots_first=heads == 2, extra=heads % 2)
    x = [c.rng.normal(size=(c.T, heads, D)).astype(np.float32) * np.where(c.rng.random((heads, D)) < 0.04, 8, 1) for _ in "kv"]
    x[0][0, 0, :] = 0
    if heads > 2:
        x[1][0, 1, 3], x[1][1, 2, 7], x[0][1, 2] = np.inf, np.nan, 2.0 ** -101
    new = [cuda(a.astype(np.float32), DT[dtype]) for a in x]
    want_rows, want_scales = [p.copy() for p in c.pools], [s.copy() for s in c.scales]
    back = [np.zeros((c.T, heads, D), dtype=np.float32) for _ in "kv"]
    for side in range(2):
        rows, scales = ref.quantise(new[side].float().cpu().numpy(), kind)
        values = ref.open_rows(rows, kind).astype(np.float32) * scales[..., None]
        for b in range(len(lens[0])):
            for tok in range(c.q_start[b], c.q_start[b + 1]):
                at = ref.place(c.kv_len, c.q_start, c.table, c.pages, page, b, tok)
                if at is not None:
                    want_rows[side][at[0], :, at[1]], want_scales[side][at[0], :, at[1]] = rows[tok], scales[tok]
                    back[side][tok] = values[tok]
    wq.wq_kv_append_dev(c.cache, c.batch, *new)
    k, v, ks, vs = c.host()
    for got, want in ((k, want_rows[0]), (v, want_rows[1]), (ks, want_scales[0]), (vs, want_scales[1])):
        np.testing.assert_array_equal(got, want)
    for off in (0, 3):  # plain outputs, and misaligned ones inside a wider row
        out = [torch.full((c.T, heads * D + 8), 7.0, dtype=DT[dtype], device="cuda") for _ in "kv"]
        view = [o[:, off:off + heads * D].unflatten(1, (heads, D)) for o in out]
        wq.wq_kv_read_dev(c.cache, c.batch, *view)
        for side in range(2):
            want = torch.from_numpy(back[side]).to(DT[dtype])
            np.testing.assert_array_equal(view[side].float().cpu().numpy(), want.float().numpy())
            assert (out[side][:, :off] == 7).all() and (out[side][:, off + heads * D:] == 7).all()
    wide = torch.zeros((c.T, 2 * heads * D + 3), dtype=DT[dtype], device="cuda")  # keys and values inside a fused projection
    views = [wide[:, 3 + i * heads * D:3 + (i + 1) * heads * D].unflatten(1, (heads, D)) for i in range(2)]
    views[0].copy_(new[0]), views[1].copy_(new[1])
    wq.wq_kv_append_dev(c.cache, c.batch, *views)
    for got, want in zip(c.host(), (want_rows[0], want_rows[1], want_scales[0], want_scales[1])):
        np.testing.assert_array_equal(got, want)


def test_append_codes_next_to_a_border():
    """Values that are whole codes and a half: ties go to even, as the fp64 quotient has them."""
    for kind, n in ((ref.I8, 127), (ref.I4, 7)):
        c = Case(1, kind, 64, 1, 16, [4], [4], fill=False)
        x = np.zeros((4, 1, 64), dtype=np.float32)
        for t, s in enumerate((1.0, 0.375, 3.0e-5, 7.0e9)):
            x[t, 0] = (c.rng.integers(-n, n, 64) + 0.5).astype(np.float32) * np.float32(s)
            x[t, 0, 0] = np.float32(n) * np.float32(s)
        new = cuda(x)
        wq.wq_kv_append_dev(c.cache, c.batch, new, new)
        rows, scales = ref.quantise(x, kind)
        k, _, ks, _ = c.host()
        for t in range(4):
            at = ref.place(c.kv_len, c.q_start, c.table, c.pages, 16, 0, t)
            np.testing.assert_array_equal(k[at[0], 0, at[1]], rows[t, 0])
            assert ks[at[0], 0, at[1]] == scales[t, 0]


def test_pages_that_are_not_there_are_left_alone():
    """Refused on the CPU's reference first: entries outside the pool, and a table that is too short."""
    c = Case(2, ref.I8, 64, 2, 16, [40, 20], [40, 60], fill=False)
    c.table[0, 1], c.table[1, 2] = -7, c.pages
    table = cuda(c.table[:, :3])
    batch = wq.KvBatch(cuda(c.q_start), cuda(c.kv_len), table, c.T)
    x = [cuda(c.rng.normal(size=(c.T, 2, 64)).astype(np.float32)) for _ in "kv"]
    wq.wq_kv_append_dev(c.cache, batch, *x)
    out = [torch.full_like(a, 7.0) for a in x]
    wq.wq_kv_read_dev(c.cache, batch, *out)
    k, _, ks, _ = c.host()
    written = np.zeros((c.pages, 16), dtype=bool)
    rows, _ = ref.quantise(x[0].cpu().numpy(), ref.I8)
    for b in range(2):
        for tok in range(c.q_start[b], c.q_start[b + 1]):
            at = ref.place(c.kv_len, c.q_start, c.table[:, :3], c.pages, 16, b, tok)
            if at is None:
                assert (out[0][tok] == 0).all() and (out[1][tok] == 0).all()
            else:
                written[at] = True
                np.testing.assert_array_equal(k[at[0], :, at[1]], rows[tok])
    assert (k.transpose(0, 2, 1, 3)[~written] == 255).all() and np.isnan(ks.transpose(0, 2, 1)[~written]).all()


# ---------------------------------------------------------------------------------------
# attention


def attend(c, q, dtype, scale=None, causal=True, window=0, batch=None, lse=True):
    T, H, D = q.shape
    obuf, o = guarded((T, H, D), DT[dtype])
    lbuf, l = guarded((T, H), torch.float32)
    wq.wq_attn_paged_dev(c.cache, batch or c.batch, q, o, scale=D ** -0.5 if scale is None else scale, causal=causal,
                         window=window, lse=l if lse else None)
    torch.cuda.synchronize()
    check_guard(obuf), check_guard(lbuf)
    return o, l


def check_attention(c, q, o, l, dtype, scale=None, causal=True, window=0, table=None, what=""):
    k, v, ks, vs = c.host()
    D = c.D
    want, lse, A, S = ref.attention(f64(q), c.kind, k, v, ks, vs, c.q_start, c.kv_len, c.table if table is None else table,
                                    D ** -0.5 if scale is None else scale, causal, window)
    kv = int(c.kv_len.max())
    e = (D + 8) * U * S
    r = 2.0 ** -21 if dtype == "f32" else 2 * 2.0 ** -11
    tol = A * (2 * e + (kv + 72) * U + r)[..., None] + 1.01 * HALF[dtype] * np.abs(want) + SMALL[dtype]
    err = np.abs(f64(o) - want)
    bad = ~(err <= tol)
    assert not bad.any(), "%s: %d of %d outputs are off, worst %.3g of the bound at %s" % (
        what, bad.sum(), bad.size, np.nanmax(err / tol), np.argwhere(bad)[:3].tolist())
    seen = np.isfinite(lse)
    l = f64(l)
    assert np.array_equal(l[~seen], lse[~seen])
    assert (np.abs(l - lse)[seen] <= (e + (kv + 72) * U + U * np.abs(lse) + U)[seen]).all(), what


def queries(c, H, dtype, loud=2.5):
    return cuda((c.rng.normal(size=(c.T, H, c.D)) * loud).astype(np.float32), DT[dtype])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_len,kv_len,heads,G,page,causal,window", [
    ([1], [1], 1, 1, 16, True, 0),
    ([1, 1, 1], [17, 130, 64], 2, 6, 16, True, 0),
    ([1, 0, 1, 1], [0, 5, 300, 65], 1, 12, 7, True, 0),
    ([2, 5, 1], [40, 5, 200], 2, 3, 32, True, 0),
    ([5, 1], [700, 31], 1, 8, 256, True, 100),
    ([70, 3, 1], [90, 3, 129], 2, 2, 16, True, 33),
    ([40, 20], [30, 20], 1, 4, 1, True, 0),      # more new tokens than positions: the first see nothing
    ([33, 129], [50, 129], 1, 1, 128, False, 0),
    ([150], [333], 1, 5, 64, True, 1),
])
def test_attention(dtype, kind, D, q_len, kv_len, heads, G, page, causal, window):
    what = "attention %s kind=%d D=%d q=%s kv=%s heads=%d G=%d page=%d causal=%d window=%d" % (
        dtype, kind, D, q_len, kv_len, heads, G, page, causal, window)
    gu.banner(what)
    c = Case(D + kind + sum(kv_len), kind, D, heads, page, q_len, kv_len, slots_first=heads == 2, extra=G % 2)
    q = queries(c, heads * G, dtype)
    o, l = attend(c, q, dtype, causal=causal, window=window)
    check_attention(c, q, o, l, dtype, causal=causal, window=window, what=what)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_len,kv_len,G", [([1], [5000], 4), ([1, 1], [3000, 64], 1), ([4], [2500], 16), ([200], [1500], 2)])
def test_attention_long(kind, q_len, kv_len, G):
    """Long enough for the positions to be split among blocks and joined; with the lengths given and not."""
    gu.banner("attention long kind=%d %s %s G=%d" % (kind, q_len, kv_len, G))
    c = Case(sum(kv_len), kind, 64, 1, 64, q_len, kv_len)
    q = queries(c, G, "f32")
    told = wq.KvBatch(*c.batch.tensors, c.T, max_q=max(q_len), max_kv=max(kv_len))
    wrong = wq.KvBatch(*c.batch.tensors, c.T, max_q=1, max_kv=3)  # results are right whatever they say
    for batch in (c.batch, told, wrong):
        o, l = attend(c, q, "f32", batch=batch)
        check_attention(c, q, o, l, "f32", what="long")
        again, l2 = attend(c, q, "f32", batch=batch)
        assert torch.equal(o, again) and torch.equal(l, l2)
        o3, _ = attend(c, q, "f32", batch=batch, lse=False)
        assert torch.equal(o, o3)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_len", [[1, 1, 1], [30, 2, 64]])
def test_attention_masked_places_hold_anything(kind, q_len):
    """NaN and infinities in the scales of positions that a row does not see, and bytes that are no finite half."""
    c = Case(77, kind, 128, 2, 16, q_len, [100, 2, 77])
    q = queries(c, 6, "f32", 1.0)
    o, l = attend(c, q, "f32", window=20)
    first = [int(kv) - n for n, kv in zip(q_len, c.kv_len)]
    for b, at in enumerate(first):
        for t in range(int(c.kv_len[b])):
            pg, slot = ref.place_at(c.table, c.pages, 16, b, t)
            if t + 20 <= at:  # before the first new token's window
                for dst, bad in zip(c.dev, (255, 255, float("nan"), float("inf"))):
                    dst[pg, :, slot] = bad
    o2, l2 = attend(c, q, "f32", window=20)
    assert torch.equal(o, o2) and torch.equal(l, l2)
    # positions after a token's own: only that sequence's later tokens see them
    b = 0
    n = q_len[b]
    if n > 1:
        pg, slot = ref.place_at(c.table, c.pages, 16, b, int(c.kv_len[b]) - 1)
        for dst, bad in zip(c.dev, (255, 255, float("nan"), float("nan"))):
            dst[pg, :, slot] = bad
        o3, l3 = attend(c, q, "f32", window=20)
        keep = torch.ones(c.T, dtype=torch.bool)
        keep[n - 1] = False
        assert torch.equal(o3[keep.cuda()], o[keep.cuda()]) and torch.equal(l3[keep.cuda()], l[keep.cuda()])
        assert o3[n - 1].isnan().all() and l3[n - 1].isnan().all()


def test_attention_pages_that_are_not_there():
    c = Case(5, ref.I8, 64, 2, 16, [1, 30], [100, 90])
    c.table[0, 2], c.table[1, 0], c.table[1, 4] = -1, c.pages + 3, -2147483648
    short = np.ascontiguousarray(c.table[:, :5])  # and positions past the table
    batch = wq.KvBatch(cuda(c.q_start), cuda(c.kv_len), cuda(short), c.T)
    for dtype in DT:
        q = queries(c, 6, dtype)
        o, l = attend(c, q, dtype, batch=batch)
        check_attention(c, q, o, l, dtype, table=short)
    none = torch.full_like(batch.tensors[2], -1)
    o, l = attend(c, q, dtype, batch=wq.KvBatch(cuda(c.q_start), cuda(c.kv_len), none, c.T))
    assert (o == 0).all() and (l == -float("inf")).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0, 1e-3])
def test_attention_scale(scale):
    c = Case(6, ref.I8, 64, 1, 16, [1, 50], [70, 60])
    q = queries(c, 3, "f32")
    o, l = attend(c, q, "f32", scale=scale)
    check_attention(c, q, o, l, "f32", scale=scale)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("q_len", [[1, 1], [20, 50]])
def test_attention_rows_and_scales_of_any_size(dtype, q_len):
    """Queries and values far from one: no intermediate leaves its type's range."""
    for qs, vs in ((1e-8, 1.0), (2e4, 1e-3), (1.0, 1e25), (1.0, 1e-25)):
        if dtype != "f32" and not 1e-3 <= vs <= 1:
            continue
        if dtype == "f16" and not 1e-6 < qs < 1e4:  # such queries are no finite halves
            continue
        gu.banner("attention sizes %s q=%g v=%g" % (dtype, qs, vs))
        c = Case(8, ref.F16, 64, 1, 16, q_len, [40, 90])
        c.dev[3].mul_(vs)
        q = queries(c, 4, dtype, qs)
        o, l = attend(c, q, dtype, scale=0.125 / max(qs, 1.0))
        check_attention(c, q, o, l, dtype, scale=0.125 / max(qs, 1.0), what="q=%g v=%g" % (qs, vs))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("q_len", [[1, 1], [20, 50]])
def test_attention_strides(dtype, q_len):
    c = Case(9, ref.I4, 128, 2, 32, q_len, [40, 90])
    q = queries(c, 4, dtype)
    o, l = attend(c, q, dtype)
    for off in (8, 5):
        wide = torch.full((c.T, 4 * 128 + 30), 3.0, dtype=DT[dtype], device="cuda")
        qv = wide[:, off:off + 512].unflatten(1, (4, 128))
        qv.copy_(q)
        out = torch.full((4, c.T, 128 + off), 3.0, dtype=DT[dtype], device="cuda")
        ov = out.transpose(0, 1)[..., off:]
        wq.wq_attn_paged_dev(c.cache, c.batch, qv, ov, scale=128 ** -0.5)
        assert torch.equal(ov, o) and (out[..., :off] == 3).all()


def test_offsets_past_32_bits():
    """A page stride that puts the last page beyond 2^32 bytes from the first."""
    pages, stride = 5, (1 << 30) + 4096
    big = torch.empty(4 * stride + 2 * 16 * 64, dtype=torch.uint8, device="cuda")
    pools = [big.as_strided((pages, 1, 16, 64), (stride, 1024, 64, 1), off) for off in (0, 1024)]
    sbig = torch.empty(4 * stride + 32, dtype=torch.float32, device="cuda")
    scales = [sbig.as_strided((pages, 1, 16), (stride, 16, 1), off) for off in (0, 16)]
    c = Case(10, ref.I8, 64, 1, 16, [1, 20], [33, 40], spare=0)
    assert c.pages >= pages
    keep = np.array([[4, 0, 3], [4, 1, 2]], dtype=np.int32)
    c.pages, c.table = pages, keep
    for dst, src in zip(pools + scales, c.dev):
        dst.copy_(torch.nan_to_num(src[:pages].float(), nan=0.5).to(dst.dtype))
    c.dev = pools + scales
    c.cache, c.batch = wq.KvCache(ref.I8, *c.dev), wq.KvBatch(cuda(c.q_start), cuda(c.kv_len), cuda(keep), c.T)
    x = cuda(c.rng.normal(size=(c.T, 1, 64)).astype(np.float32))
    wq.wq_kv_append_dev(c.cache, c.batch, x, x)
    back = [torch.empty_like(x) for _ in "kv"]
    wq.wq_kv_read_dev(c.cache, c.batch, *back)
    assert torch.equal(back[0], back[1]) and (back[0] - x).abs().max() <= x.abs().max() / 250
    q = queries(c, 2, "f32")
    o, l = attend(c, q, "f32")
    check_attention(c, q, o, l, "f32")


def test_streams_graphs_and_faults():
    """One decode step on another stream, in a replayed graph, and refused by an injected fault."""
    c = Case(12, ref.I8, 128, 2, 16, [1, 1, 1, 1], [900, 20, 64, 333])
    c.batch = wq.KvBatch(*c.batch.tensors, c.T, max_q=1, max_kv=900)
    x = cuda(c.rng.normal(size=(4, 1280)).astype(np.float32))
    w = cuda(c.rng.normal(size=1280).astype(np.float32))
    pos = cuda((c.kv_len - 1)[None])
    h = wq.wq_rope_create(128, 0, 1e4, [64])
    y, o, l = torch.empty_like(x), torch.empty((4, 6, 128), device="cuda"), torch.empty((4, 6), device="cuda")
    q, k = torch.empty((4, 6, 128), device="cuda"), torch.empty((4, 2, 128), device="cuda")

    def step(stream=None):
        wq.wq_rmsnorm_dev(x, w, 1e-6, y, stream=stream)
        t = y.unflatten(1, (10, 128))
        wq.wq_rope_dev(h, t[:, :6], pos, q, stream=stream)
        wq.wq_rope_dev(h, t[:, 6:8], pos, k, stream=stream)
        v = t[:, 8:]
        wq.wq_kv_append_dev(c.cache, c.batch, k, v.contiguous() if stream is None else vbuf, stream=stream)
        wq.wq_attn_paged_dev(c.cache, c.batch, q, o, scale=0.1, lse=l, stream=stream)

    vbuf = torch.empty((4, 2, 128), device="cuda")
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, q, k, o, l)] + [t.clone() for t in c.dev]
    vbuf.copy_(y.unflatten(1, (10, 128))[:, 8:])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for t in (y, q, k, o, l):
        t.fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    step(stream=side)
    side.synchronize()
    for got, w0 in zip((y, q, k, o, l, *c.dev), want):
        assert torch.equal(got.nan_to_num(), w0.nan_to_num())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(stream=side)
    for _ in range(3):
        for t in (y, q, k, o, l):
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        for got, w0 in zip((y, q, k, o, l, *c.dev), want):
            assert torch.equal(got.nan_to_num(), w0.nan_to_num())
        step()  # eager work between replays
        torch.cuda.synchronize()
    gu.reinit_with_env(WQ_FAULT="launch")
    try:
        with pytest.raises(wq.WqError) as e:
            step()
        assert e.value.code == wq.WQ_E_FAULT
    finally:
        gu.reinit_with_env(WQ_FAULT=None)
