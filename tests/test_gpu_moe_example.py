"""The example layer with a mixture of experts on a stream that is not torch's current one."""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import gpu_util as gu  # noqa: E402
import moe_layer  # noqa: E402


def test_all_of_a_call_runs_on_its_stream():
    """A step with stream= while torch's current stream is busy for longer than the step takes: the same bits as with it current."""
    layer = moe_layer.MoeLayer()
    pages = moe_layer.Pages(64, layer.page, 2, 16)
    batch, _ = pages.extend([5, 9])
    rng = np.random.default_rng(3)
    x = torch.from_numpy(rng.normal(size=(14, layer.hidden)).astype(np.float32)).cuda()
    one, other, side = layer.buffers(14), layer.buffers(14), torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device="cuda")
    gu.banner("example layer, current stream")
    layer(x, batch, one)
    layer(x, batch, other, stream=side)  # (workspaces grow, which waits for the device)
    torch.cuda.synchronize()
    # what the first call of `other` left there is not what this one has to leave
    other["ids"][:, :layer.k].fill_(-1), other["stream"].zero_()
    torch.cuda.synchronize()
    gu.banner("example layer, side stream")
    for _ in range(200):
        torch.mm(busy, busy)
    layer(x, batch, other, stream=side)
    side.synchronize()
    got = other["stream"].clone()
    torch.cuda.synchronize()
    assert torch.equal(got, one["stream"])
    layer.close()
