"""The example layer (norm, products, rotary positions, quantised cache, attention, gated feed-forward) against the same
layer in 64 bits on the CPU, prompts of several lengths and decode steps in one run.

The reference rounds keys and values to the cache's format as the definition has it; where an fp32 key and its 64-bit
value fall on two sides of a rounding border, an element differs by one step (f16 2^-11 of the value, int8 1/127 of the
row's largest, int4 1/7). The products' contract is 1e-5. Softmax, norms and the feed-forward each pass a relative
difference on at most a few times larger, and few elements meet a border: the stream (residual included) agrees within
2^-10 in the root mean square for f16 and int8, and within 2^-6 for int4.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import pytest

import decoder_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - CPU hosts
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import decoder_layer  # noqa: E402


def reference(layer, kind, calls):
    H, K, D, G = layer.heads, layer.kv_heads, layer.dim, layer.heads // layer.kv_heads
    w1, w2 = (w.cpu().numpy().astype(np.float64) for w in (layer.w1, layer.w2))
    norm = lambda x, w: x / np.sqrt((x * x).mean(1, keepdims=True) + layer.eps) * w  # noqa: E731
    kept = None
    for new, x, _ in calls:
        x = x.cpu().numpy().astype(np.float64)
        if kept is None:
            kept = [[np.zeros((0, K, D)), np.zeros((0, K, D))] for _ in new]
        at = np.cumsum([0] + list(new))
        pos = np.concatenate([np.arange(len(kept[b][0]), len(kept[b][0]) + n) for b, n in enumerate(new)])[None]
        qkv = (norm(x, w1) @ layer.host["qkv"].T).reshape(len(x), H + 2 * K, D)
        q, k, v = qkv[:, :H], qkv[:, H:H + K], qkv[:, H + K:]
        q, k = (ref.rope(t.copy(), pos, D, 0, 1e4, [D // 2]) for t in (q, k))
        o = np.zeros_like(q)
        for b, n in enumerate(new):
            for side, t in enumerate((k, v)):
                rows, scales = ref.quantise(t[at[b]:at[b + 1]].astype(np.float32), kind)
                kept[b][side] = np.concatenate([kept[b][side], ref.open_rows(rows, kind) * scales.astype(np.float64)[..., None]])
            for i in range(n):
                last = len(kept[b][0]) - n + i + 1
                for h in range(H):
                    s = kept[b][0][:last, h // G] @ q[at[b] + i, h] * D ** -0.5
                    w = np.exp(s - s.max())
                    o[at[b] + i, h] = w / w.sum() @ kept[b][1][:last, h // G]
        stream = x + o.reshape(len(x), -1) @ layer.host["out"].T
        y = norm(stream, w2)
        g, u = y @ layer.host["gate"].T, y @ layer.host["up"].T
        yield stream + (g / (1 + np.exp(-g)) * u) @ layer.host["down"].T


@pytest.mark.parametrize("kind,tol", [(ref.F16, 2.0 ** -10), (ref.I8, 2.0 ** -10), (ref.I4, 2.0 ** -6)])
def test_layer(kind, tol):
    layer = decoder_layer.DecoderLayer(kind=kind, seed=kind)
    try:
        calls = decoder_layer.run(layer)
        torch.cuda.synchronize()
        for (new, _, got), want in zip(calls, reference(layer, kind, calls)):
            got = got.cpu().numpy().astype(np.float64)
            assert np.sqrt(((got - want) ** 2).mean()) <= tol * np.sqrt((want ** 2).mean()), new
    finally:
        layer.close()
