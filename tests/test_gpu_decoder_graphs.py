"""A captured decode step whose positions are split keeps its workspace: larger eager calls on the same stream grow that
stream's own, and every replay still equals the eager step."""
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


def pools(rng, pages, heads, page, D):
    k, v = (torch.from_numpy(rng.integers(0, 256, (pages, heads, page, D), dtype=np.uint8)).cuda() for _ in "kv")
    ks, vs = (torch.from_numpy(rng.uniform(0.01, 0.02, (pages, heads, page)).astype(np.float32)).cuda() for _ in "kv")
    return wq.KvCache(ref.I8, k, v, ks, vs)


def batch(pages, page, new, kv):
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    start, lens = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, new], [kv]))
    return wq.KvBatch(start, lens, table, new, max_q=new, max_kv=kv)


def test_replays_after_larger_eager_calls():
    gu.reinit_with_env(WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None)
    rng = np.random.default_rng(4)
    heads, H, D, page, pages = 8, 48, 128, 64, 64
    cache = pools(rng, pages, heads, page, D)
    one, many, more = batch(pages, page, 1, 1500), batch(pages, page, 128, 4096), batch(pages, page, 300, 4096)
    q1, qm, qn = (torch.randn((b.T, H, D), device="cuda", generator=torch.Generator("cuda").manual_seed(b.T)) for b in (one, many, more))
    o1, om, on = (torch.empty_like(q) for q in (q1, qm, qn))
    lse = torch.empty((1, H), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gu.banner("decode step, eager, then captured")
    step = lambda: wq.wq_attn_paged_dev(cache, one, q1, o1, scale=D ** -0.5, lse=lse, stream=side)  # noqa: E731
    step()
    side.synchronize()
    want, want_lse = o1.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    first = None
    for b, q, o in ((many, qm, om), (more, qn, on), (many, qm, om)):
        gu.banner("larger eager call: %d new tokens" % b.T)
        wq.wq_attn_paged_dev(cache, b, q, o, scale=D ** -0.5, stream=side)
        side.synchronize()
        if b is many:
            first = om.clone() if first is None else first
            assert torch.equal(om, first)
        room = torch.full((4 << 20,), float("nan"), device="cuda")  # memory that the library may have given back
        for _ in range(3):
            o1.fill_(float("nan")), lse.fill_(float("nan"))
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o1, want) and torch.equal(lse, want_lse)
            step()
            torch.cuda.synchronize()
            assert torch.equal(o1, want)
        assert room.isnan().all()
        del room
