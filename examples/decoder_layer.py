"""One decoder layer over the weight-only quantised products: norm, fused q/k/v product, rotary positions, quantised
paged cache, attention, output product, norm with the residual, gated feed-forward. Prompts of several lengths go
through it in one batch, then each sequence decodes a few tokens.

    python examples/decoder_layer.py

Weights are random int4 codes with a scale a row; activations are fp32.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_matmul_amd as wq  # noqa: E402

ROW_BYTES = {wq.WQ_KV_F16: lambda d: 2 * d, wq.WQ_KV_I8: lambda d: d, wq.WQ_KV_I4: lambda d: d // 2}


class DecoderLayer:
    def __init__(self, hidden=512, heads=8, kv_heads=2, dim=64, inter=1024, kind=wq.WQ_KV_I8, page=16, pages=64, seed=0):
        rng = np.random.default_rng(seed)
        wq.wq_init([0])
        self.hidden, self.heads, self.kv_heads, self.dim, self.page, self.eps = hidden, heads, kv_heads, dim, page, 1e-6
        self.host = {}

        def weights(name, O, I):
            codes = rng.integers(1, 16, (O, I), dtype=np.uint8)  # nibble - 8: -7 .. 7
            scales = (rng.uniform(0.5, 1.5, O) / (4.5 * np.sqrt(I))).astype(np.float32)
            self.host[name] = (codes.astype(np.float64) - 8) * scales[:, None]
            packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
            return wq.wq_tensor_upload(None, 0, wq.WQ_I4, O, I, packed, scales)

        self.qkv = weights("qkv", (heads + 2 * kv_heads) * dim, hidden)
        self.out = weights("out", hidden, heads * dim)
        self.gate, self.up = weights("gate", inter, hidden), weights("up", inter, hidden)
        self.down = weights("down", hidden, inter)
        self.gated, self.plain = wq.wq_swiglu_create([self.gate], [self.up]), wq.wq_grouped_create([self.down])
        self.w1, self.w2 = (torch.from_numpy((1 + 0.1 * rng.normal(size=hidden)).astype(np.float32)).cuda() for _ in range(2))
        self.rope = wq.wq_rope_create(dim, 0, 1e4, [dim // 2])
        shape = (pages, kv_heads, page)
        pools = [torch.zeros(shape + (ROW_BYTES[kind](dim),), dtype=torch.uint8, device="cuda") for _ in "kv"]
        scales = [torch.zeros(shape, device="cuda") for _ in "kv"]
        self.cache = wq.KvCache(kind, *pools, *scales)

    def __call__(self, x, batch, pos):
        """x float32 [T, hidden] (the residual stream), batch of its tokens, pos int32 [1, T]; returns the new stream."""
        T, H, K, D = x.shape[0], self.heads, self.kv_heads, self.dim
        new = lambda *shape: torch.empty(shape, device="cuda")  # noqa: E731
        y, qkv = new(T, self.hidden), new(T, (H + 2 * K) * D)
        wq.wq_rmsnorm_dev(x, self.w1, self.eps, y)
        wq.wq_matmul_dev(self.qkv, y, qkv)
        q, k, v = qkv.unflatten(1, (H + 2 * K, D)).split([H, K, K], dim=1)  # views: no copies
        wq.wq_rope_dev(self.rope, q, pos, q)
        wq.wq_rope_dev(self.rope, k, pos, k)
        wq.wq_kv_append_dev(self.cache, batch, k, v)
        o, a = new(T, H, D), new(T, self.hidden)
        wq.wq_attn_paged_dev(self.cache, batch, q, o, scale=D ** -0.5)
        wq.wq_matmul_dev(self.out, o.flatten(1), a)
        stream, h, f = new(T, self.hidden), new(T, self.gate.O), new(T, self.hidden)
        wq.wq_rmsnorm_dev(a, self.w2, self.eps, y, residual=x, sum_out=stream)
        wq.wq_swiglu_ffn_dev(self.gated, self.plain, [y], [h], [f])
        return stream + f

    def close(self):
        wq.wq_grouped_free(self.gated)
        wq.wq_grouped_free(self.plain)
        for t in (self.qkv, self.out, self.gate, self.up, self.down):
            wq.wq_tensor_free(t)
        wq.wq_rope_free(self.rope)


class Pages:
    """Hands out pages of the cache to sequences as they grow."""

    def __init__(self, pages, page, sequences, width):
        self.free, self.page = list(range(pages))[::-1], page
        self.table = np.full((sequences, width), -1, dtype=np.int32)
        self.len = np.zeros(sequences, dtype=np.int32)

    def extend(self, new):
        """(batch, positions) of new[b] more tokens for every sequence b."""
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        pos = np.concatenate([np.arange(n, n + m) for n, m in zip(self.len, new)]).astype(np.int32)
        for b, m in enumerate(new):
            for i in range(-(-int(self.len[b]) // self.page), -(-int(self.len[b] + m) // self.page)):
                self.table[b, i] = self.free.pop()
        self.len += np.asarray(new, dtype=np.int32)
        dev = [torch.from_numpy(a.copy()).cuda() for a in (start, self.len, self.table, pos[None])]
        return wq.KvBatch(*dev[:3], int(start[-1]), max_q=int(max(new)), max_kv=int(self.len.max())), dev[3]


def run(layer, prompts=(37, 1, 90), steps=4, seed=1):
    """The layer over the prompts in one batch, then `steps` tokens a sequence; inputs and outputs of every call."""
    rng = np.random.default_rng(seed)
    pages = Pages(64, layer.page, len(prompts), 16)
    calls = []
    for new in [list(prompts)] + [[1] * len(prompts)] * steps:
        x = torch.from_numpy(rng.normal(size=(sum(new), layer.hidden)).astype(np.float32)).cuda()
        batch, pos = pages.extend(new)
        calls.append((new, x, layer(x, batch, pos)))
    return calls


if __name__ == "__main__":
    layer = DecoderLayer()
    for new, x, y in run(layer):
        torch.cuda.synchronize()
        print("new tokens %s: output %s, rms %.4f" % (new, tuple(y.shape), y.square().mean().sqrt()))
    layer.close()
