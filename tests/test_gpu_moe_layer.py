"""The example layer with a mixture of experts against the same layer in 64 bits on the CPU: prompts of several lengths eagerly,
decode steps as replays of one captured graph.

The reference rounds keys and values to the cache's format as the definition has it, and takes the experts that the definition
chooses by the scores of the GPU (which are compared by themselves): a score next to another's could else choose differently.
Where an fp32 key and its 64-bit value fall on two sides of a rounding border, an element differs by one step (f16 2^-11 of the
value, int8 1/127 of the row's largest, int4 1/7); few do. The products' contract is 1e-5, and norms, softmax and experts each
pass a relative difference on at most a few times larger: stream and norm agree within 2^-10 in the root mean square for f16
and int8, and within 2^-6 for int4.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

import decoder_ref as dref
import moe_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_layer  # noqa: E402


def reference(layer, kind, calls):
    H, K, D, G, eps = layer.heads, layer.kv_heads, layer.dim, layer.heads // layer.kv_heads, layer.eps
    w = [t.cpu().numpy().astype(np.float64) for t in layer.w]
    bias = layer.bias.cpu().numpy()
    norm = lambda x, w: x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * w  # noqa: E731
    kept = None
    for new, x, scores, _, _ in calls:
        x = x.cpu().numpy().astype(np.float64)
        if kept is None:
            kept = [[np.zeros((0, K, D)), np.zeros((0, K, D))] for _ in new]
        at = np.cumsum([0] + list(new))
        pos = np.concatenate([np.arange(len(kept[b][0]), len(kept[b][0]) + n) for b, n in enumerate(new)])[None]
        qkv = (norm(x, w[0]) @ layer.host["qkv"].T).reshape(len(x), H + 2 * K, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        q, k = (dref.rope(t.copy(), pos, D, 0, 1e4, [D // 2]) for t in (q, k))
        o = np.zeros_like(q)
        for b, n in enumerate(new):
            for side, t in enumerate((k, v)):
                rows, scales = dref.quantise(t[at[b]:at[b + 1]].astype(np.float32), kind)
                kept[b][side] = np.concatenate([kept[b][side], dref.open_rows(rows, kind) * scales.astype(np.float64)[..., None]])
            for i in range(n):
                last = len(kept[b][0]) - n + i + 1
                for h in range(H):
                    s = kept[b][0][:last, h // G] @ q[at[b] + i, h] * D ** -0.5
                    p = np.exp(s - s.max())
                    o[at[b] + i, h] = p / p.sum() @ kept[b][1][:last, h // G]
        mid = x + layer.alpha * norm(o.reshape(len(x), -1) @ layer.host["out"].T, w[1])
        y = norm(mid, w[2])
        got = scores.cpu().numpy().astype(np.float64)
        ids, share = ref.route(got, layer.k, bias, "sigmoid", 4, 2)
        f = np.zeros_like(x)
        for t in range(len(x)):
            for e, s in list(zip(ids[t], share[t])) + [(layer.experts, 1.0)]:
                g, u = (layer.host["%s%d" % (n, e)] @ y[t] for n in ("gate", "up"))
                f[t] += s * (layer.host["down%d" % e] @ (ref.silu(g) * u))
        out = mid + layer.alpha * f
        yield y @ layer.host["router"].T, out, norm(out, w[3])


@pytest.mark.parametrize("kind,tol", [(dref.F16, 2.0 ** -10), (dref.I8, 2.0 ** -10), (dref.I4, 2.0 ** -6)])
def test_layer(kind, tol):
    layer = moe_layer.MoeLayer(kind=kind, seed=kind)
    try:
        calls = moe_layer.run(layer)
        for (new, _, *got), want in zip(calls, reference(layer, kind, calls)):
            for g, v in zip(got, want):
                g = g.cpu().numpy().astype(np.float64)
                assert np.sqrt(((g - v) ** 2).mean()) <= tol * np.sqrt((v ** 2).mean()), new
    finally:
        layer.close()
