"""Rotary positions with append, and the norms around a block, against their plain forms in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest

import decoder_ref as dref
import moe_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

import gpu_util as gu  # noqa: E402
import weight_only_quantized_matmul_amd as wq  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
THETA = 1e5


@pytest.fixture(autouse=True)
def _init():
    gu.reinit_with_env(WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None)
    yield
    torch.cuda.synchronize()


class Case:
    def __init__(self, rng, kind, dtype, D, heads, q_len, kv_len, page, table=None, pages=None):
        self.kind, self.D, self.heads, self.page = kind, D, heads, page
        self.start = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        self.kv_len = np.array(kv_len, dtype=np.int32)
        self.T = int(self.start[-1])
        if table is None:
            pages, table = dref.paging(rng, kv_len, page)
        self.pages, self.table = pages, table
        rb = dref.row_bytes(kind, D)
        self.k, self.v = (torch.full((pages, heads, page, rb), 0x5A, dtype=torch.uint8, device="cuda") for _ in "kv")
        self.ks, self.vs = (torch.full((pages, heads, page), -3.0, device="cuda") for _ in "kv")
        self.cache = wq.KvCache(kind, self.k, self.v, self.ks, self.vs)
        self.batch = wq.KvBatch(*(torch.from_numpy(a).cuda() for a in (self.start, self.kv_len, self.table)), self.T)
        self.new = [torch.from_numpy(rng.normal(0, 2, (self.T, heads, D)).astype(np.float32)).cuda().to(DT[dtype]) for _ in "kv"]

    def positions(self):
        p = np.zeros(self.T, dtype=np.int64)
        for b in range(len(self.kv_len)):
            n = self.start[b + 1] - self.start[b]
            p[self.start[b]:self.start[b + 1]] = max(int(self.kv_len[b]), 0) - n + np.arange(n)
        return p

    def check_cache(self, k_turned):
        """Every row of the pools: the batch's tokens hold k_turned (float64) and v within half a code, the others are as they were."""
        want = {}
        for b in range(len(self.kv_len)):
            for tok in range(self.start[b], self.start[b + 1]):
                at = dref.place(self.kv_len, self.start, self.table, self.pages, self.page, b, tok)
                if at is not None:
                    want[at] = tok
        for rows, scales, x in ((self.k, self.ks, k_turned), (self.v, self.vs, self.new[1].double().cpu().numpy())):
            rows, scales = rows.cpu().numpy(), scales.cpu().numpy()
            codes = dref.open_rows(rows, self.kind)
            for pg in range(self.pages):
                for sl in range(self.page):
                    if (pg, sl) not in want:
                        assert (rows[pg, :, sl] == 0x5A).all() and (scales[pg, :, sl] == -3.0).all(), "a row of no token was written"
                        continue
                    got, v = codes[pg, :, sl] * scales[pg, :, sl].astype(np.float64)[:, None], x[want[pg, sl]]
                    if self.kind == dref.F16:  # a value is rounded to fp32 and to a half of 11 bits, or of steps of 2^-24 in units of the scale
                        bound = np.abs(v) * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25 * scales[pg, :, sl][:, None]
                    else:  # half a code, and the roundings to fp32 of the value and the scale, times at most 127 codes
                        bound = scales[pg, :, sl][:, None] * (0.5 + 127 * 2.0 ** -23)
                    assert (np.abs(got - v) <= bound).all()
                    top = np.abs(v).max(-1)
                    unit = 127 if self.kind == dref.I8 else 7
                    if self.kind == dref.F16:
                        assert ((top >= scales[pg, :, sl] * 2.0 ** 14 * (1 - 2.0 ** -20)) & (top <= scales[pg, :, sl] * 2.0 ** 15 * (1 + 2.0 ** -20))).all()
                    else:
                        assert (np.abs(scales[pg, :, sl] - top / unit) <= 2.0 ** -22 * top / unit).all()


def check_append(c, rng, dtype, rot, pairing, sections, pos=None, H=None, inplace=False, shift=0):
    """pos: int array [axes, T] or None; H: query heads or None; shift: elements by which rows start past an aligned address."""
    gu.banner("append kind=%d %s D=%d rot=%d pairing=%d sections=%s T=%d H=%s" % (c.kind, dtype, c.D, rot, pairing, sections, c.T, H))
    rope = wq.wq_rope_create(rot, pairing, THETA, sections)
    q = out = None
    if H:
        room = torch.from_numpy(rng.normal(0, 1, (c.T + 2, H * c.D + 2 * shift)).astype(np.float32)).cuda().to(DT[dtype])
        q = room[1:c.T + 1, shift:shift + H * c.D].view(c.T, H, c.D) if shift == 0 else room[1:c.T + 1, shift:shift + H * c.D].unflatten(1, (H, c.D))
        before = room.clone()
        out = q if inplace else torch.empty_like(before)[1:c.T + 1, shift:shift + H * c.D].unflatten(1, (H, c.D))
    was = None if q is None else q.double().cpu().numpy()
    dpos = None if pos is None else torch.from_numpy(pos.astype(np.int32)).cuda()
    wq.wq_kv_append_rope_dev(c.cache, c.batch, rope, *c.new, q=q, q_out=out, pos=dpos)
    torch.cuda.synchronize()
    p = c.positions()[None] if pos is None else pos
    turned = dref.rope(c.new[0].double().cpu().numpy(), p, rot, pairing, THETA, sections)
    c.check_cache(turned)
    if H:
        want = dref.rope(was, p, rot, pairing, THETA, sections)
        # once to fp32, once to the type; the angle's fp64 error grows with the position, which stays below 2^20: 2^-53 * 2^20 * |x|
        # queries of 16 bits turn in fp32: the cosine and the sine, two products and their sum are each within 2^-24 of |x|
        turn = 2.0 ** -30 if dtype == "f32" else 6 * 2.0 ** -24
        bound = np.abs(want) * (ref.HALF[dtype] + 2.0 ** -23) + turn * np.abs(was).max() + ref.TINY[dtype]
        assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()
        if inplace:
            edge = room.clone()
            edge[1:c.T + 1, shift:shift + H * c.D] = before[1:c.T + 1, shift:shift + H * c.D]
            assert torch.equal(edge, before), "written outside of q"


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", [dref.F16, dref.I8, dref.I4])
@pytest.mark.parametrize("D,rot,pairing", [(64, 64, 0), (64, 2, 0), (128, 128, 1), (128, 80, 0), (128, 30, 1), (128, 20, 0), (256, 256, 0), (256, 128, 1)])
def test_append_rope(kind, dtype, D, rot, pairing):
    rng = np.random.default_rng(D + rot)
    c = Case(rng, kind, dtype, D, 3, [5, 1, 0, 2, 4], [9, 1, 5, 40, 3], 5)
    check_append(c, rng, dtype, rot, pairing, [rot // 2], H=6)


@pytest.mark.parametrize("pairing", [0, 1])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_rope_axes_and_far_positions(dtype, pairing):
    rng = np.random.default_rng(2)
    c = Case(rng, dref.I8, dtype, 128, 2, [7, 30], [100, 30], 16)
    pos = rng.integers(-1000, 1 << 20, (3, c.T))
    check_append(c, rng, dtype, 128, pairing, [30, 10, 24], pos=pos, H=4, inplace=True)
    check_append(c, rng, dtype, 96, pairing, [48], pos=pos[:1], H=1)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("inplace", [False, True])
def test_append_rope_unaligned_rows(dtype, inplace):
    rng = np.random.default_rng(3)
    c = Case(rng, dref.I8, dtype, 128, 2, [3, 2], [3, 9], 4)
    for pairing in (0, 1):
        check_append(c, rng, dtype, 128, pairing, [64], H=5, inplace=inplace, shift=3)


def test_append_rope_without_queries_and_one_token():
    rng = np.random.default_rng(4)
    check_append(Case(rng, dref.I4, "f32", 64, 1, [1], [1], 1), rng, "f32", 64, 0, [32])
    check_append(Case(rng, dref.I8, "bf16", 128, 8, [1], [77], 64), rng, "bf16", 128, 0, [64], H=48)


def test_append_rope_tokens_without_a_place():
    """Pages outside the pool, positions before the start and past the table: not written, turned all the same."""
    rng = np.random.default_rng(5)
    table = np.array([[0, -1, 9, 1], [2, 3, 4, 1 << 30]], dtype=np.int32)
    c = Case(rng, dref.I8, "f32", 64, 2, [16, 6], [13, 18], 4, table=table, pages=5)
    check_append(c, rng, "f32", 64, 0, [32], H=3)


def test_append_rope_rows_behind_the_last_sequence():
    rng = np.random.default_rng(6)
    c = Case(rng, dref.I8, "f32", 64, 2, [3, 2], [5, 2], 4)
    more = 4  # tokens that belong to no sequence
    T = c.T + more
    batch = wq.KvBatch(*(torch.from_numpy(a).cuda() for a in (c.start, c.kv_len, c.table)), T)
    k, v, q = (torch.randn((T, 2, 64), device="cuda") for _ in range(3))
    out = torch.full_like(q, 7.0)
    rope = wq.wq_rope_create(64, 0, THETA, [32])
    for pos in (None, torch.zeros((1, T), dtype=torch.int32, device="cuda")):
        wq.wq_kv_append_rope_dev(c.cache, batch, rope, k, v, q=q, q_out=out, pos=pos)
        torch.cuda.synchronize()
        assert (out[c.T:] == 7.0).all() and (out[:c.T] != 7.0).any()


@pytest.mark.parametrize("kind", [dref.F16, dref.I8, dref.I4])
def test_append_rope_rows_that_are_not_finite_or_tiny(kind):
    rng = np.random.default_rng(7)
    c = Case(rng, kind, "f32", 64, 1, [6], [6], 8)
    k, v = c.new
    k[0, 0, 3], k[1, 0, 40], k[2], k[3] = float("nan"), float("inf"), 0.0, 1e-33
    v[4, 0, 0], v[5] = float("-inf"), 0.0
    rope = wq.wq_rope_create(64, 1, THETA, [32])
    wq.wq_kv_append_rope_dev(c.cache, c.batch, rope, k, v)
    torch.cuda.synchronize()
    pg = c.table[0, 0]
    codes, ks, vs = dref.open_rows(c.k.cpu().numpy(), kind)[pg, 0], c.ks.cpu().numpy()[pg, 0], c.vs.cpu().numpy()[pg, 0]
    assert np.isnan(ks[:2]).all() and (codes[:4] == 0).all() and (ks[2:4] == 0).all() and (ks[4:6] > 0).all()
    assert np.isnan(vs[4]) and vs[5] == 0 and (vs[:4] > 0).all()


def test_append_rope_equals_its_parts_and_runs_in_a_graph():
    """Queries as wq_rope_dev turns them; keys as wq_kv_append_dev stores the turned ones, but for roundings; replays follow the lengths."""
    rng = np.random.default_rng(8)
    page, B, D, heads, H = 16, 40, 128, 4, 16
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    kv = torch.from_numpy(rng.integers(1, 60, B).astype(np.int32)).cuda()
    pools = lambda: wq.KvCache(dref.I8, *(torch.zeros((B * 4, heads, page, D), dtype=torch.uint8, device="cuda") for _ in "kv"),  # noqa: E731
                               *(torch.zeros((B * 4, heads, page), device="cuda") for _ in "kv"))
    a, b = pools(), pools()
    batch = wq.KvBatch(start, kv, table, B, max_q=1, max_kv=60)
    k, v, q = torch.empty((B, heads, D), device="cuda"), torch.empty((B, heads, D), device="cuda"), torch.empty((B, H, D), device="cuda")
    q1, q2, k2 = torch.empty_like(q), torch.empty_like(q), torch.empty_like(k)
    rope = wq.wq_rope_create(D, 0, THETA, [D // 2])
    out = [torch.empty((B, heads, D), device="cuda") for _ in range(4)]
    side = torch.cuda.Stream()
    step = lambda: wq.wq_kv_append_rope_dev(a, batch, rope, k, v, q=q, q_out=q1, stream=side)  # noqa: E731
    for t in (k, v, q):
        t.normal_()
    torch.cuda.synchronize()
    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for _ in range(4):
        for t in (k, v, q):
            t.normal_()
        kv.copy_(torch.from_numpy(rng.integers(1, 60, B).astype(np.int32)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        pos = (kv - 1)[None].contiguous()
        wq.wq_rope_dev(rope, q, pos, q2)
        wq.wq_rope_dev(rope, k, pos, k2)
        wq.wq_kv_append_dev(b, batch, k2, v)
        wq.wq_kv_read_dev(a, batch, out[0], out[1])
        wq.wq_kv_read_dev(b, batch, out[2], out[3])
        torch.cuda.synchronize()
        assert torch.equal(out[1], out[3])
        assert (q1 - q2).abs().max() <= 4e-7 * q.abs().max()
        step_ = k2.abs().amax(-1, keepdim=True) / 127
        assert ((out[0] - out[2]).abs() <= 1.001 * step_).all()  # a code at a border may fall to either side


def test_append_rope_more_tokens_than_a_launch_has_threads():
    """A prompt of 2^24 + 9 tokens (a block of 256 threads each): its last tokens as a batch of their own leaves them."""
    T, last, page, D = (1 << 24) + 9, 40, 128, 64
    gu.banner("append_rope T=%d" % T)
    pages = -(-T // page)
    g = torch.Generator("cuda").manual_seed(4)
    k, v = (torch.zeros((T, 1, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    for t in (k, v):
        t[:last].normal_(generator=g)
        t[-last:].normal_(generator=g)
    rope = wq.wq_rope_create(D, 0, 1e6, [D // 2])
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    caches = []
    for n in range(2):
        pools = [torch.zeros((pages, 1, page, D // 2), dtype=torch.uint8, device="cuda") for _ in "kv"]
        caches.append((wq.KvCache(wq.WQ_KV_I4, *pools, *[torch.zeros((pages, 1, page), device="cuda") for _ in "kv"]), pools))
    for (cache, _), lo in zip(caches, (0, T - last)):
        batch = wq.KvBatch(torch.tensor([0, T - lo], dtype=torch.int32, device="cuda"), torch.tensor([T], dtype=torch.int32, device="cuda"), table, T - lo)
        wq.wq_kv_append_rope_dev(cache, batch, rope, k[lo:], v[lo:])
    torch.cuda.synchronize()
    for whole, part in zip(caches[0][1], caches[1][1]):
        whole, part = (p.view(-1, D // 2)[:T] for p in (whole, part))
        assert torch.equal(whole[-last:], part[-last:]) and not torch.equal(whole[:last], part[:last])
    wq.wq_rope_free(rope)


def test_append_rope_refusals_of_the_binding():
    rng = np.random.default_rng(9)
    c = Case(rng, dref.I8, "f32", 64, 2, [3], [3], 4)
    rope, two = wq.wq_rope_create(64, 0, THETA, [32]), wq.wq_rope_create(64, 0, THETA, [16, 16])
    q = torch.zeros((3, 4, 64), device="cuda")
    for kw in (dict(q=q), dict(q_out=q), dict(q=q[:2], q_out=q[:2]), dict(q=q[..., :32], q_out=q[..., :32]), dict(q=q.half(), q_out=q.half()),
               dict(q=q, q_out=q.half()), dict(pos=torch.zeros((1, 3), device="cuda")), dict(pos=torch.zeros((1, 2), dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            wq.wq_kv_append_rope_dev(c.cache, c.batch, rope, *c.new, **kw)
    with pytest.raises(wq.WqError):
        wq.wq_kv_append_rope_dev(c.cache, c.batch, two, *c.new)
    gu.reinit_with_env(WQ_FAULT="launch")
    with pytest.raises(wq.WqError) as e:
        wq.wq_kv_append_rope_dev(c.cache, c.batch, rope, *c.new)
    assert e.value.code == wq.WQ_E_FAULT


# ---------------------------------------------------------------------------------------


def check_norm(rng, rows, n, dtype, out, post=True, gate="all", eps=1e-6, alpha=0.7, scale=1.0, shift=0, keep=True, pre=True):
    gu.banner("block norm %d x %d %s -> %s post=%s gate=%s" % (rows, n, dtype, out, post, gate))

    def make(r, s=1.0, dt=None):
        room = torch.from_numpy((rng.normal(0, s, (r, n + 2 * shift))).astype(np.float32)).cuda().to(DT[dt or dtype])
        return room[:, shift:shift + n]

    x, res = make(rows, scale), make(rows, 2 * scale)
    g = None if gate == "none" else make(1 if gate == "row" else rows)
    wpost = torch.from_numpy(rng.normal(1, 0.2, n).astype(np.float32)).cuda() if post else None
    wpre = torch.from_numpy(rng.normal(1, 0.2, n).astype(np.float32)).cuda() if pre else None
    room_s = torch.full((rows + 2, n + 2 * shift + 1), 7.0, dtype=DT[dtype], device="cuda")
    room_y = torch.full((rows + 2, n + 2 * shift + 1), 7.0, dtype=DT[out], device="cuda")
    s, y = room_s[1:rows + 1, shift:shift + n], room_y[1:rows + 1, shift:shift + n]
    wq.wq_rmsnorm_block_dev(x, res, eps, w_post=wpost, gate=g, alpha=alpha, w_pre=wpre, y=y if pre else None, sum_out=s if keep else None)
    torch.cuda.synchronize()
    np64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    a32 = float(np.float32(alpha))
    r, Er, want, Ey = ref.block_norm(np64(x), np64(res), np64(wpost), np64(g), a32, np64(wpre), float(np.float32(eps)))
    for got, v, E, dt, wanted in ((s, r, Er, dtype, keep), (y, want, Ey, out, pre)):
        if not wanted:
            assert (got == 7.0).all()
            continue
        bound = E + ref.HALF[dt] * (np.abs(v) + E) + ref.TINY[dt]
        err = np.abs(np64(got) - v)
        assert (err <= bound).all(), "worst err/bound %.3g" % (err / bound).max()
    for room in (room_s, room_y):
        edge = room.clone()
        edge[1:rows + 1, shift:shift + n] = 7.0
        assert (edge == 7.0).all(), "written outside of the rows"


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("rows,n", [(1, 1), (1, 6144), (3, 7), (2, 64), (5, 1000), (700, 333), (2, 5001), (3, 16384), (1, 32768), (1200, 768)])
def test_block_norm(rows, n, dtype, out):
    rng = np.random.default_rng(n)
    check_norm(rng, rows, n, dtype, out)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["none", "row", "all"])
@pytest.mark.parametrize("shift", [0, 1])
def test_block_norm_forms(post, gate, shift):
    rng = np.random.default_rng(1)
    check_norm(rng, 4, 520, "f32", "f32", post=post, gate=gate, shift=shift)
    check_norm(rng, 600, 130, "bf16", "bf16", post=post, gate=gate, shift=shift, alpha=1.0)
    check_norm(rng, 4, 520, "f16", "bf16", post=post, gate=gate, shift=shift, keep=False)
    check_norm(rng, 4, 520, "f32", "f32", post=post, gate=gate, shift=shift, pre=False, alpha=-0.3)


@pytest.mark.parametrize("scale", [1e-30, 1e-18, 1e18, 1e30])
def test_block_norm_far_rows(scale):
    rng = np.random.default_rng(2)
    for post in (True, False):
        check_norm(rng, 3, 700, "f32", "f32", post=post, gate="row", scale=scale, eps=0.0 if scale < 1 else 1e-6)


def test_block_norm_overlaps():
    rng = np.random.default_rng(3)
    for dtype in ("f32", "bf16"):
        x, res = (torch.from_numpy(rng.normal(0, 1, (9, 300)).astype(np.float32)).cuda().to(DT[dtype]) for _ in "xr")
        w = torch.ones(300, device="cuda")
        s, y = torch.empty_like(x), torch.empty_like(x)
        wq.wq_rmsnorm_block_dev(x, res, 1e-6, w_post=w, gate=x, w_pre=w, y=y, sum_out=s)
        x2, r2 = x.clone(), res.clone()
        wq.wq_rmsnorm_block_dev(x2, r2, 1e-6, w_post=w, gate=x2, w_pre=w, y=x2, sum_out=r2)
        torch.cuda.synchronize()
        assert torch.equal(s, r2) and torch.equal(y, x2)


def test_block_norm_bad_rows_stay_their_own():
    x, res = (torch.randn((4, 256), device="cuda") for _ in "xr")
    w = torch.ones(256, device="cuda")
    x[1, 3], res[2, 5] = float("nan"), float("inf")
    s, y = torch.empty_like(x), torch.empty_like(x)
    wq.wq_rmsnorm_block_dev(x, res, 1e-6, w_post=w, w_pre=w, y=y, sum_out=s)
    torch.cuda.synchronize()
    assert torch.isfinite(y[[0, 3]]).all() and torch.isfinite(s[[0, 3]]).all()
    assert y[1].isnan().all() and not torch.isfinite(y[2]).all()


def test_block_norm_refusals_of_the_binding():
    x, w = torch.zeros((2, 8), device="cuda"), torch.ones(8, device="cuda")
    for kw in (dict(y=x), dict(w_pre=w), dict(w_post=w[:4], sum_out=x), dict(gate=x[:, :4], sum_out=x), dict(gate=x.half(), sum_out=x),
               dict(sum_out=x.half()), dict(gate=torch.zeros((3, 8), device="cuda"), sum_out=x)):
        with pytest.raises(ValueError):
            wq.wq_rmsnorm_block_dev(x, x, 1e-6, **kw)
    with pytest.raises(wq.WqError):
        wq.wq_rmsnorm_block_dev(x, x, 1e-6)
