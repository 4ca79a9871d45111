"""One decoder layer with a mixture of experts, from the residual stream to the residual stream without the host in between:
norm, fused q/k/v product, rotary positions with the append to the quantised cache, attention, output product, the norms around
the block, the router's product and choice, the experts with a shared one among them, and the norm behind them. Prompts go
through it in one batch; the decode steps after them are one graph that is captured once and replayed.

    python examples/moe_layer.py

Weights are random int4 codes with a scale a row, the router's are fp32; activations are fp32.
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_matmul_amd as wq  # noqa: E402
from decoder_layer import ROW_BYTES, Pages  # noqa: E402


class MoeLayer:
    def __init__(self, hidden=512, heads=8, kv_heads=2, dim=64, inter=256, experts=16, k=4, kind=wq.WQ_KV_I8, page=16, pages=64, seed=0):
        rng = np.random.default_rng(seed)
        wq.wq_init([0])
        self.hidden, self.heads, self.kv_heads, self.dim, self.page, self.eps = hidden, heads, kv_heads, dim, page, 1e-6
        self.experts, self.k, self.alpha = experts, k, 0.5
        self.host, self.tensors = {}, []

        def weights(name, O, I):
            codes = rng.integers(1, 16, (O, I), dtype=np.uint8)  # nibble - 8: -7 .. 7
            scales = (rng.uniform(0.5, 1.5, O) / (4.5 * np.sqrt(I))).astype(np.float32)
            self.host[name] = (codes.astype(np.float64) - 8) * scales[:, None]
            self.tensors.append(wq.wq_tensor_upload(None, 0, wq.WQ_I4, O, I, codes[:, 0::2] | (codes[:, 1::2] << 4), scales))
            return self.tensors[-1]

        self.qkv = weights("qkv", (heads + 2 * kv_heads) * dim, hidden)
        self.out = weights("out", hidden, heads * dim)
        # the last of the experts is the shared one: every token has it, with weight 1
        sets = [[weights("%s%d" % (name, e), *shape) for e in range(experts + 1)]
                for name, shape in (("gate", (inter, hidden)), ("up", (inter, hidden)), ("down", (hidden, inter)))]
        self.moe = wq.wq_moe_create(*sets)
        router = (rng.normal(size=(experts, hidden)) / np.sqrt(hidden) * 2).astype(np.float32)
        self.host["router"] = router.astype(np.float64)
        self.tensors.append(wq.wq_tensor_upload(None, 0, wq.WQ_F32, experts, hidden, router.view(np.uint8), None))
        self.router = self.tensors[-1]
        self.w = [torch.from_numpy((1 + 0.1 * rng.normal(size=hidden)).astype(np.float32)).cuda() for _ in range(4)]
        self.bias = torch.from_numpy((0.02 * rng.normal(size=experts)).astype(np.float32)).cuda()
        self.rope = wq.wq_rope_create(dim, 0, 1e4, [dim // 2])
        shape = (pages, kv_heads, page)
        pools = [torch.zeros(shape + (ROW_BYTES[kind](dim),), dtype=torch.uint8, device="cuda") for _ in "kv"]
        scales = [torch.zeros(shape, device="cuda") for _ in "kv"]
        self.cache = wq.KvCache(kind, *pools, *scales)

    def buffers(self, T):
        """What a call for T tokens writes; a captured call keeps it."""
        H, K, D = self.heads, self.kv_heads, self.dim
        new = lambda *shape: torch.empty(shape, device="cuda")  # noqa: E731
        b = {"y": new(T, self.hidden), "qkv": new(T, (H + 2 * K) * D), "o": new(T, H, D), "a": new(T, self.hidden), "mid": new(T, self.hidden),
             "scores": new(T, self.experts), "f": new(T, self.hidden), "stream": new(T, self.hidden), "next": new(T, self.hidden)}
        b["chosen"] = torch.empty((T, self.k), dtype=torch.int32, device="cuda")
        b["share"] = new(T, self.k)
        b["ids"] = torch.full((T, self.k + 1), self.experts, dtype=torch.int32, device="cuda")
        b["weights"] = torch.ones((T, self.k + 1), device="cuda")
        return b

    def __call__(self, x, batch, b, stream=None):
        """x float32 [T, hidden] (the residual stream); leaves the new stream in b["stream"] and its norm in b["next"]."""
        H, K, D = self.heads, self.kv_heads, self.dim
        s = dict(stream=stream)
        wq.wq_rmsnorm_dev(x, self.w[0], self.eps, b["y"], **s)
        wq.wq_matmul_dev(self.qkv, b["y"], b["qkv"], **s)
        q, k, v = b["qkv"].unflatten(1, (H + 2 * K, D)).split([H, K, K], dim=1)  # views: no copies
        wq.wq_kv_append_rope_dev(self.cache, batch, self.rope, k, v, q=q, q_out=q, **s)
        wq.wq_attn_paged_dev(self.cache, batch, q, b["o"], scale=D ** -0.5, **s)
        wq.wq_matmul_dev(self.out, b["o"].flatten(1), b["a"], **s)
        wq.wq_rmsnorm_block_dev(b["a"], x, self.eps, w_post=self.w[1], alpha=self.alpha, w_pre=self.w[2], y=b["y"], sum_out=b["mid"], **s)
        wq.wq_matmul_dev(self.router, b["y"], b["scores"], **s)
        wq.wq_moe_route_dev(b["scores"], b["chosen"], b["share"], bias=self.bias, gating=wq.WQ_GATE_SIGMOID, groups=4, top_groups=2, **s)
        with torch.cuda.stream(stream):  # torch's copies belong between the choice and the experts (None: the current stream)
            b["ids"][:, :self.k].copy_(b["chosen"])
            b["weights"][:, :self.k].copy_(b["share"])
        wq.wq_moe_ffn_dev(self.moe, b["y"], b["ids"], b["weights"], b["f"], **s)
        wq.wq_rmsnorm_block_dev(b["f"], b["mid"], self.eps, alpha=self.alpha, w_pre=self.w[3], y=b["next"], sum_out=b["stream"], **s)

    def close(self):
        torch.cuda.synchronize()
        wq.wq_moe_free(self.moe)
        for t in self.tensors:
            wq.wq_tensor_free(t)
        wq.wq_rope_free(self.rope)


def run(layer, prompts=(37, 1, 90), steps=4, seed=1):
    """The layer over the prompts in one batch, then `steps` tokens a sequence by replays of one graph: (new tokens, input,
    scores, new stream, its norm) of every call."""
    rng = np.random.default_rng(seed)
    pages = Pages(64, layer.page, len(prompts), 16)
    side = torch.cuda.Stream()
    inputs = lambda T: torch.from_numpy(rng.normal(size=(T, layer.hidden)).astype(np.float32)).cuda()  # noqa: E731
    keep = lambda b: tuple(b[n].clone() for n in ("scores", "stream", "next"))  # noqa: E731
    x, b = inputs(sum(prompts)), layer.buffers(sum(prompts))
    batch, _ = pages.extend(list(prompts))
    layer(x, batch, b)
    torch.cuda.synchronize()
    calls = [(list(prompts), x, *keep(b))]
    B, graph = len(prompts), None
    x, b = inputs(B), layer.buffers(B)
    for _ in range(steps):
        now, _ = pages.extend([1] * B)
        x.copy_(inputs(B))
        torch.cuda.synchronize()
        if graph is None:
            # an eager step first, which makes the stream's workspace as large as the graph needs it. It writes the new tokens'
            # rows of the cache, as the first replay does again.
            batch = wq.KvBatch(*(t.clone() for t in now.tensors), now.T, max_q=1, max_kv=256)
            with torch.cuda.stream(side):
                layer(x, batch, b, stream=side)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                layer(x, batch, b, stream=side)
        for kept, new in zip(batch.tensors, now.tensors):
            kept.copy_(new)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        calls.append(([1] * B, x.clone(), *keep(b)))
    return calls


if __name__ == "__main__":
    layer = MoeLayer()
    for new, x, scores, y, _ in run(layer):
        print("new tokens %s: output %s, rms %.4f" % (new, tuple(y.shape), y.square().mean().sqrt()))
    layer.close()
