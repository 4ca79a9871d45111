"""An expert layer that is captured on a stream without a workspace, with another stream's."""
from __future__ import annotations

import numpy as np
import pytest

import moe_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

import gpu_util as gu  # noqa: E402
import weight_only_quantized_matmul_amd as wq  # noqa: E402
from test_gpu_moe_ranges import Layer, choose, matrix  # noqa: E402


@pytest.mark.parametrize("T,k", [(90, 4), (20, 2)])  # a plan in the workspace, with parts made ahead; none
def test_replays_between_the_owners_calls(T, k):
    """Replays and the owner's eager calls, one after another, each give what they give alone, also after the owner has grown."""
    gu.init()
    rng = np.random.default_rng(41)
    D, F, E = 256, 100, 24
    mats = [[matrix(rng, ref.I4, r, c, 0, 0.2 / np.sqrt(c)) for r, c in ((F, D), (F, D), (D, F))] for _ in range(3)]
    layer, other = Layer(mats, E), Layer(mats[::-1], E + 5)
    x = rng.normal(0, 1, (T, D)).astype(np.float32)
    (ids, w), (ids2, w2) = choose(rng, T, E, k), choose(rng, T, E + 5, k)
    want, want2 = layer.check(x, ids, w, "layer"), other.check(x, ids2, w2, "other")  # warms the current stream
    dx, di, dw, di2, dw2 = (torch.from_numpy(a).cuda() for a in (x, ids, w, ids2, w2))
    y, y2 = torch.empty_like(want), torch.empty_like(want2)
    cold = torch.cuda.Stream()
    torch.cuda.synchronize()
    gu.banner("capture on a cold stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cold):
        wq.wq_moe_ffn_dev(layer.moe, dx, di, dw, y, stream=cold)
    for i in range(6):
        y.fill_(float("nan")), y2.fill_(float("nan"))
        g.replay()  # on the current stream, between the owner's calls
        wq.wq_moe_ffn_dev(other.moe, dx, di2, dw2, y2)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(y2, want2)
        if i == 2:  # the owner needs more and leaves the block to the graph
            big = torch.zeros((1200, D), device="cuda")
            wq.wq_moe_ffn_dev(layer.moe, big, torch.zeros((1200, 8), dtype=torch.int32, device="cuda"), torch.zeros((1200, 8), device="cuda"), torch.empty_like(big))
            torch.cuda.synchronize()
    layer.free(), other.free()
