"""The choice of experts where the bias holds infinities: experts that are forced and forbidden."""
from __future__ import annotations

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

import gpu_util as gu  # noqa: E402
import weight_only_quantized_matmul_amd as wq  # noqa: E402

INF = float("inf")


@pytest.mark.parametrize("bias,groups,top,k,ids", [
    ([0, 0, 0, 0, 0, 0, 0, 0], 1, 1, 3, [7, 6, 5]),
    ([INF, 0, 0, 0, 0, 0, 0, -INF], 1, 1, 3, [0, 6, 5]),  # one forced, one forbidden
    ([0, 0, INF, 0, 0, 0, 0, 0], 4, 1, 2, [2, 3]),  # a forced one's group is the largest
    ([0, -INF, 0, 0, 0, 0, -INF, -INF], 4, 2, 4, [5, 4, 3, 2]),  # groups with a forbidden one are the last
    ([INF, -INF, 0, 0, 0, 0, 0, 0], 4, 1, 2, [7, 6]),  # +inf and -inf are no sum: the group counts as -inf
    ([-INF] * 8, 4, 2, 3, [0, 1, 2]),  # all alike: the lowest
    ([float("nan"), 0, 0, 0, 0, 0, 0, 0], 1, 1, 8, [7, 6, 5, 4, 3, 2, 1, 0])])
@pytest.mark.parametrize("gating", ["softmax", "sigmoid"])
def test_infinite_bias(gating, bias, groups, top, k, ids):
    gu.init()
    scores = torch.arange(8, dtype=torch.float32, device="cuda")[None] / 4
    got, w = torch.empty((1, k), dtype=torch.int32, device="cuda"), torch.empty((1, k), device="cuda")
    wq.wq_moe_route_dev(scores, got, w, bias=torch.tensor(bias, dtype=torch.float32, device="cuda"), groups=groups, top_groups=top, normalise=False,
                        gating=wq.WQ_GATE_SOFTMAX if gating == "softmax" else wq.WQ_GATE_SIGMOID)
    torch.cuda.synchronize()
    x = np.arange(8) / 4
    p = np.exp(x) / np.exp(x).sum() if gating == "softmax" else 1 / (1 + np.exp(-x))
    assert got[0].tolist() == ids
    assert (np.abs(w[0].double().cpu().numpy() - p[ids]) <= (2.0 ** -24 + 1e-12) * p[ids]).all()  # one rounding of fp64
