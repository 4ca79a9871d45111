"""Cases for measuring the operators of a mixture-of-experts decoder layer, with their plain forms.

Four operators: the choice of each token's experts from the router's scores ("route"), the whole gated
feed-forward layer of the experts that were chosen ("moe"), rotary positions applied to queries and keys
while the keys and values go into the paged cache ("append"), and the norms after a block and before the
next one with the block's gate and the residual between them ("norms").

The plain forms are elementary torch operations in 32 bits (64 where 32 lose what matters: the angles of far
positions, scores that decide a choice, values next to a rounding border). With `own` set, run() makes the
calls of weight_only_quantized_matmul_amd instead, on the same inputs.

Expert weights, as both sides have them: codes uint8 [E, rows, row bytes] and scales float32 [E, rows] or
[E, rows, groups of columns]; int8, int4 (two a byte, the even element in the low half, value code - 8) or
int2 (four a byte, lowest bits first, value code - 2). The cache is that of perf/operators.py: pools k, v
uint8 [pages, kv heads, page, row bytes] and k_scale, v_scale float32 [pages, kv heads, page].
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
I8, I4, I2 = 1, 2, 3  # formats of weights
BITS = {I8: 8, I4: 4, I2: 2}
KV_F16, KV_I8, KV_I4 = 0, 1, 2  # cache kinds
TINY = 2.0 ** -100  # a cache row whose largest magnitude is below this is stored as zeros
EPS = 1e-6


def _route(name, **kw):
    c = {"name": name, "op": "route", "T": 1, "E": 256, "k": 8, "dtype": "f32", "gating": "sigmoid", "bias": True, "groups": 1,
         "top_groups": 1, "normalise": True, "scale": 2.5}
    c.update(kw)
    return c


def _moe(name, **kw):
    c = {"name": name, "op": "moe", "T": 1, "E": 16, "k": 8, "D": 6144, "F": 2048, "fmt": I4, "gs": 0, "dtype": "f32", "pad": False, "add": False}
    c.update(kw)
    return c


def _append(name, **kw):
    c = {"name": name, "op": "append", "H": 48, "Hkv": 8, "D": 128, "rot": 128, "pairing": 0, "axes": 0, "far": 0, "page": 64, "kind": KV_I8,
         "dtype": "f32", "B": 64, "q_max": 1, "kv_max": 2000, "lens": 1}
    c.update(kw)
    return c


def _norms(name, **kw):
    c = {"name": name, "op": "norms", "rows": 1, "n": 6144, "dtype": "f32", "out": "f32", "post": True, "gate": "row"}
    c.update(kw)
    return c


def listed():
    # hidden size 6144 and expert width 2048 as in the repository's benchmark; 48 query heads of 128 over 8 key/value heads
    return [
        # one user's next token: 8 of 256 experts in groups, with the bias that evens out the experts' load
        _route("route_one", groups=8, top_groups=4),
        # a prompt's tokens in 16 bits, softmax gating
        _route("route_prompt", T=8191, E=128, dtype="bf16", gating="softmax", bias=False, scale=1.0),
        # one user's next token through 8 of 16 experts: the latency of a step, and the stream of their weights
        _moe("moe_one"),
        # a serving batch in 16 bits over many small experts, one or two tokens each; some places of the batch are empty
        _moe("moe_batch", T=17, E=64, D=2048, F=768, dtype="bf16", pad=True),
        # a few tokens checked at once (drafted ones), experts in 2 bits
        _moe("moe_drafted", T=5, E=8, k=2, fmt=I2, dtype="f16", add=True),
        # a larger serving batch on few experts in 8 bits: about 16 tokens each
        _moe("moe_wide", T=64, E=8, k=2, fmt=I8),
        # group-wise scales, odd sizes
        _moe("moe_groups", T=33, E=12, k=3, D=1001, F=525, gs=128, dtype="bf16"),
        # a decode step's queries, keys and values of 64 users
        _append("append_decode", lens=6),
        # a prefill of four prompts in 16 bits into a 4-bit cache; time, height and width as positions, half of each head turned
        _append("append_prompt", B=4, q_max=2048, kv_max=3000, kind=KV_I4, dtype="bf16", axes=3, far=4096, rot=64, pairing=1, lens=7),
        # one token between two blocks
        _norms("norms_one"),
        # a prefill's rows in 16 bits, a gate value for each of them
        _norms("norms_prompt", rows=8191, dtype="bf16", out="bf16", gate="all"),
        # an odd row length, no norm after the block
        _norms("norms_odd", rows=509, n=5001, dtype="f16", post=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "moe", "append", "norms"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(2, _log(rng, 4, 512) // groups)
        top = rng.randint(1, groups)
        k = rng.randint(1, min(16, E // groups * top))
        return _route("", T=_log(rng, 1, 8192), E=E, k=k, dtype=dtype, gating=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                      groups=groups, top_groups=top, normalise=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
    if op == "moe":
        fmt = rng.choice([I8, I4, I4, I2])
        D, F, E = _log(rng, 64, 6144), _log(rng, 64, 2048), _log(rng, 2, 128)
        E = max(2, min(E, 604_000_000 // (3 * D * F * BITS[fmt] // 4)))
        k = rng.randint(1, min(8, E))
        T = max(1, min(_log(rng, 1, 128), 2_000_000_000 // (D * F * k)))
        return _moe("", T=T, E=E, k=k, D=D, F=F, fmt=fmt, gs=rng.choice([0, 0, 64, 128]), dtype=dtype, pad=rng.random() < 0.3, add=rng.random() < 0.3)
    if op == "append":
        D = rng.choice([64, 128, 128, 256])
        Hkv, G = rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 6, 8])
        B, q_max = _log(rng, 1, 128), _log(rng, 1, 4096)
        q_max = max(1, min(q_max, 40_000_000 // (B * Hkv * (G + 2) * D)))
        return _append("", H=Hkv * G, Hkv=Hkv, D=D, rot=rng.choice([D, D, D // 2]), pairing=rng.choice([0, 1]), axes=rng.choice([0, 0, 1, 2, 3]),
                       far=_log(rng, 100, 1_000_000), page=rng.choice([16, 32, 64, 128]), kind=rng.choice([KV_F16, KV_I8, KV_I4]), dtype=dtype, B=B,
                       q_max=q_max, kv_max=q_max + rng.randint(0, 4000), lens=rng.randrange(1 << 30))
    n = _log(rng, 64, 16384)
    return _norms("", rows=min(_log(rng, 1, 16384), 31_000_000 // n), n=n, dtype=dtype, out=rng.choice(["f32", "bf16", "f16"]),
                  post=rng.random() < 0.7, gate=rng.choice(["none", "row", "all"]))


# ---------------------------------------------------------------------------------------
# inputs


def _lens(c):
    """(q_len, kv_len) of every sequence: by the case alone."""
    rng = random.Random(c["lens"])
    q, kv = [], []
    for b in range(c["B"]):
        n = c["q_max"] if b == 0 or c["q_max"] == 1 else rng.choice([1, rng.randint(1, c["q_max"]), c["q_max"]])
        q.append(n)
        kv.append(c["kv_max"] if b == 0 else rng.randint(min(n, c["kv_max"]), c["kv_max"]))
    return q, kv


def _sections(c):
    """Pairs for each axis: the first takes what the others leave. Positions by the cache's lengths are one axis."""
    half, axes = c["rot"] // 2, max(1, c["axes"])
    rest = [half * 3 // 8] * (axes - 1)
    return [half - sum(rest)] + rest


def _row_bytes(kind, D):
    return 2 * D if kind == KV_F16 else D if kind == KV_I8 else D // 2


def _groups(c, cols):
    return -(-cols // c["gs"]) if c["gs"] else 1


class _Experts:
    """The resident experts of one state; they go when it goes."""

    def __init__(self, wq, c, mats):
        sets = []
        for rows, cols, codes, scales in mats:
            codes, scales = codes.cpu().numpy(), scales.cpu().numpy()
            if c["gs"]:
                sets.append([wq.wq_tensor_upload_gs(None, 0, c["fmt"], rows, cols, c["gs"], codes[e], scales[e]) for e in range(c["E"])])
            else:
                sets.append([wq.wq_tensor_upload(None, 0, c["fmt"], rows, cols, codes[e], scales[e]) for e in range(c["E"])])
        self.wq, self.sets, self.moe = wq, sets, wq.wq_moe_create(*sets)

    def __del__(self):
        self.wq.wq_moe_free(self.moe)
        for t in sum(self.sets, []):
            self.wq.wq_tensor_free(t)


def prepare(case, seed):
    c, dt = dict(case), DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    def rand(*shape):
        return torch.rand(shape, device="cuda", generator=g)

    wq = None
    if own:
        import weight_only_quantized_matmul_amd as wq
        wq.wq_init([0])
    s = {"c": c}
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        s["scores"] = (randn(T, E) * 1.5 + randn(E) * 0.7).to(dt)
        s["bias"] = randn(E) * 0.05 if c["bias"] else None
        s["ids"] = torch.empty((T, c["k"]), dtype=torch.int32, device="cuda")
        s["w"] = torch.empty((T, c["k"]), device="cuda")
    elif c["op"] == "moe":
        T, E, k, D, F = (c[n] for n in ("T", "E", "k", "D", "F"))
        mats = []
        for rows, cols in ((F, D), (F, D), (D, F)):
            codes = torch.randint(0, 256, (E, rows, -(-cols * BITS[c["fmt"]] // 8)), device="cuda", generator=g, dtype=torch.uint8)
            spread = {I8: 74.0, I4: 4.6, I2: 1.2}[c["fmt"]]
            shape = (E, rows, _groups(c, cols)) if c["gs"] else (E, rows)
            mats.append((rows, cols, codes, (0.5 + rand(*shape)) / (spread * math.sqrt(cols))))
        s["mats"] = mats
        s["x"] = randn(T, D).to(dt)
        like = randn(T, E) + randn(E) * 0.5  # some experts are liked more than others
        top, ids = like.topk(k, 1)
        s["ids"], s["w"] = ids.to(torch.int32), top.softmax(1)
        if c["pad"]:  # places of a batch without a token: no expert
            s["ids"][rand(T) < 0.15] = -1
        s["add"] = randn(T, D).to(dt) if c["add"] else None
        if own:
            s["experts"], s["y"] = _Experts(wq, c, mats), torch.empty_like(s["x"])
    elif c["op"] == "append":
        q, kv = _lens(c)
        need = [-(-n // c["page"]) for n in kv]
        pages = sum(need) + 3
        order = torch.randperm(pages, device="cuda", generator=g)[: sum(need)].to(torch.int32)
        first = torch.tensor([0] + need, device="cuda").cumsum(0)
        at = torch.arange(max(need), device="cuda")
        have = at[None, :] < torch.tensor(need, device="cuda")[:, None]
        s["table"] = torch.where(have, order[(first[:-1, None] + at).clamp(max=len(order) - 1)], torch.full((), -1, device="cuda", dtype=torch.int32))
        s["start"] = torch.tensor([0] + q, device="cuda", dtype=torch.int32).cumsum(0).to(torch.int32)
        s["kv_len"] = torch.tensor(kv, device="cuda", dtype=torch.int32)
        T, D = sum(q), c["D"]
        shape = (pages, c["Hkv"], c["page"])
        s["k"], s["v"] = (torch.zeros(shape + (_row_bytes(c["kind"], D),), dtype=torch.uint8, device="cuda") for _ in "kv")
        s["ks"], s["vs"] = (torch.zeros(shape, device="cuda") for _ in "kv")
        loud = 1 + 7 * (rand(c["Hkv"], D) < 0.04)  # keys have a few channels much larger than the others
        s["q"], s["new_k"], s["new_v"] = randn(T, c["H"], D).to(dt), (randn(T, c["Hkv"], D) * loud).to(dt), randn(T, c["Hkv"], D).to(dt)
        s["pos"] = torch.randint(0, c["far"] + 1, (c["axes"], T), device="cuda", generator=g, dtype=torch.int32) if c["axes"] else None
        if own:
            s["cache"] = wq.KvCache(c["kind"], s["k"], s["v"], s["ks"], s["vs"])
            s["batch"] = wq.KvBatch(s["start"], s["kv_len"], s["table"], T, max_q=max(q), max_kv=max(kv))
            s["rope"] = wq.wq_rope_create(c["rot"], c["pairing"], 1e6, _sections(c))
            s["q_out"] = torch.empty_like(s["q"])
            s["out_k"], s["out_v"] = (torch.empty((T, c["Hkv"], D), device="cuda") for _ in "kv")
    else:
        rows, n = c["rows"], c["n"]
        s["x"], s["res"] = (randn(rows, n) * 0.7).to(dt), (randn(rows, n) * 2).to(dt)
        s["w_post"] = 0.3 + 0.1 * randn(n) if c["post"] else None
        s["w_pre"] = 1 + 0.2 * randn(n)
        s["gate"] = None if c["gate"] == "none" else rand(1 if c["gate"] == "row" else rows, n).to(dt)
        if own:
            s["y"], s["sum"] = torch.empty((rows, n), dtype=DTYPES[c["out"]], device="cuda"), torch.empty_like(s["x"])
    return s


# ---------------------------------------------------------------------------------------
# one pass

ALPHA = 0.21875  # scale of a block's output as it joins the residual


def run(s):
    c = s["c"]
    if own:
        import weight_only_quantized_matmul_amd as wq
        if c["op"] == "route":
            wq.wq_moe_route_dev(s["scores"], s["ids"], s["w"], bias=s["bias"], gating=wq.WQ_GATE_SOFTMAX if c["gating"] == "softmax" else wq.WQ_GATE_SIGMOID,
                                groups=c["groups"], top_groups=c["top_groups"], normalise=c["normalise"], scale=c["scale"])
            return {"ids": s["ids"], "w": s["w"]}
        if c["op"] == "moe":
            wq.wq_moe_ffn_dev(s["experts"].moe, s["x"], s["ids"], s["w"], s["y"], add=s["add"])
            return {"y": s["y"]}
        if c["op"] == "append":
            wq.wq_kv_append_rope_dev(s["cache"], s["batch"], s["rope"], s["new_k"], s["new_v"], q=s["q"], q_out=s["q_out"], pos=s["pos"])
            wq.wq_kv_read_dev(s["cache"], s["batch"], s["out_k"], s["out_v"])
            return {"q": s["q_out"], "k": s["out_k"], "v": s["out_v"]}
        wq.wq_rmsnorm_block_dev(s["x"], s["res"], EPS, w_post=s["w_post"], gate=s["gate"], alpha=ALPHA, w_pre=s["w_pre"], y=s["y"], sum_out=s["sum"])
        return {"y": s["y"], "sum": s["sum"]}
    return {"route": _plain_route, "moe": _plain_moe, "append": _plain_append, "norms": _plain_norms}[c["op"]](s)


def _plain_route(s):
    c, x = s["c"], s["scores"].double()
    T, E = x.shape
    if c["gating"] == "softmax":
        p = (x - x.amax(1, keepdim=True)).exp()
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + (-x).exp())
    choice = p if s["bias"] is None else p + s["bias"].double()
    if c["groups"] > 1:
        g = choice.view(T, c["groups"], -1)
        best = g.sort(dim=-1, descending=True)[0][..., :2].sum(-1)
        kept = best.sort(dim=1, descending=True, stable=True)[1][:, : c["top_groups"]]
        mask = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(mask[..., None], g, torch.full((), -math.inf, device="cuda", dtype=torch.float64)).reshape(T, E)
    ids = choice.sort(dim=1, descending=True, stable=True)[1][:, : c["k"]]
    w = p.gather(1, ids)
    if c["normalise"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "w": (w * c["scale"]).float()}


def _open_weights(codes, scales, cols, c):
    """float32 [rows, cols] of one expert's matrix."""
    if c["fmt"] == I8:
        q = codes.view(torch.int8).float()
    elif c["fmt"] == I4:
        q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8
    else:
        q = torch.stack([codes & 3, (codes >> 2) & 3, (codes >> 4) & 3, codes >> 6], -1).flatten(-2).float() - 2
    q = q[:, :cols]
    return q * (scales.repeat_interleave(c["gs"], 1)[:, :cols] if c["gs"] else scales[:, None])


def _plain_moe(s):
    c, x = s["c"], s["x"].float()
    y = torch.zeros_like(x) if s["add"] is None else s["add"].float()
    for e in s["ids"].unique().tolist():
        if e < 0:
            continue
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        gate, up, down = (_open_weights(codes[e], scales[e], cols, c) for _, cols, codes, scales in s["mats"])
        a, b = x[t] @ gate.t(), x[t] @ up.t()
        y.index_add_(0, t, ((a / (1 + (-a).exp()) * b) @ down.t()) * s["w"][t, j][:, None])
    return {"y": y.to(s["x"].dtype)}


def _turn(c, x, phi):
    """x [T, heads, D] in 64 bits with its pairs turned by phi [T, rot / 2], as float32."""
    cos, sin, half = phi.cos()[:, None], phi.sin()[:, None], c["rot"] // 2
    x = x.double()
    r = x[..., : c["rot"]]
    if c["pairing"] == 0:
        a, b = r[..., :half], r[..., half:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, x[..., c["rot"] :]], -1).float()


def _places(s):
    """Position, page and slot of every new token."""
    at = torch.arange(s["q"].shape[0], device="cuda")
    b = torch.searchsorted(s["start"][1:].long(), at, right=True)
    p = s["kv_len"].long()[b] - (s["start"][1:].long()[b] - at)
    return p, s["table"][b, p // s["c"]["page"]].long(), p % s["c"]["page"]


def _open_rows(rows, kind):
    """The codes of cache rows, as float32."""
    if kind == KV_F16:
        return rows.view(torch.float16).float()
    if kind == KV_I8:
        return rows.view(torch.int8).float()
    return torch.stack([(rows & 15).float() - 8, (rows >> 4).float() - 8], -1).flatten(-2)


def _quantise(x, kind):
    """(rows of codes, scales) of x [..., D]; codes next to a border are decided in 64 bits."""
    x = x.float()
    top = x.abs().amax(-1)
    zero = top < TINY
    if kind == KV_F16:
        scale = top / torch.frexp(top)[0] * 2.0 ** -15  # a power of two: the largest magnitude becomes [2^14, 2^15)
        rows = (x.double() / scale.double()[..., None]).float().half().view(torch.uint8)
    else:
        scale = (top.double() / (127 if kind == KV_I8 else 7)).float()
        code = torch.where(zero[..., None], torch.zeros((), device="cuda", dtype=torch.float64), (x.double() / scale.double()[..., None]).round())
        if kind == KV_I8:
            rows = code.to(torch.int8).view(torch.uint8)
        else:
            rows = (code + 8).to(torch.uint8)
            rows = rows[..., 0::2] | (rows[..., 1::2] << 4)
    return torch.where(zero[..., None], torch.full((), 0x88 if kind == KV_I4 else 0, device="cuda", dtype=torch.uint8), rows), torch.where(zero, torch.zeros_like(scale), scale)


def _plain_append(s):
    c = s["c"]
    p, page, slot = _places(s)
    pos = p[None] if s["pos"] is None else s["pos"]
    i = torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64)
    sec = _sections(c)
    axis = torch.repeat_interleave(torch.arange(len(sec), device="cuda"), torch.tensor(sec, device="cuda"), output_size=c["rot"] // 2)
    phi = pos[axis].double().t() * (1e6 ** (-2 * i / c["rot"]))
    at = (page[:, None], torch.arange(c["Hkv"], device="cuda")[None, :], slot[:, None])
    back = []
    for x, rows, scales in ((_turn(c, s["new_k"], phi), s["k"], s["ks"]), (s["new_v"], s["v"], s["vs"])):
        rows[at], scales[at] = _quantise(x, c["kind"])
        back.append(_open_rows(rows[at], c["kind"]) * scales[at][..., None])
    return {"q": _turn(c, s["q"], phi).to(s["q"].dtype), "k": back[0], "v": back[1]}


def _plain_norms(s):
    z = s["x"].float()
    if s["w_post"] is not None:
        z = z * torch.rsqrt(z.square().mean(1, keepdim=True) + EPS) * s["w_post"]
    if s["gate"] is not None:
        z = z * s["gate"].float()
    r = s["res"].float() + ALPHA * z
    y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + EPS) * s["w_pre"]
    return {"y": y.to(DTYPES[s["c"]["out"]]), "sum": r.to(s["x"].dtype)}


# ---------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    c = case
    if c["op"] == "route":
        e = c["T"] * c["E"]
        return {"bytes": e * SIZE[c["dtype"]] + 8 * c["T"] * c["k"] + (4 * c["E"] if c["bias"] else 0), "flops": 20 * e}
    if c["op"] == "moe":
        T, E, k, D, F = (c[n] for n in ("T", "E", "k", "D", "F"))
        active = E * (1 - (1 - k / E) ** T)  # experts that some token chose, on average
        rows = 2 * F * (-(-D * BITS[c["fmt"]] // 8) + 4 * _groups(c, D)) + D * (-(-F * BITS[c["fmt"]] // 8) + 4 * _groups(c, F))
        return {"bytes": int(active * rows) + T * D * SIZE[c["dtype"]] * (3 if c["add"] else 2) + 8 * T * k, "flops": 6 * T * k * D * F}
    if c["op"] == "append":
        T, row = sum(_lens(c)[0]), _row_bytes(c["kind"], c["D"]) + 4
        # queries read and written; keys and values read, written as codes, read back and written as values
        e = T * c["D"] * (2 * c["H"] * SIZE[c["dtype"]] + 2 * c["Hkv"] * (SIZE[c["dtype"]] + 4))
        return {"bytes": e + 4 * T * c["Hkv"] * row + 4 * T * max(1, c["axes"]), "flops": T * (3 * (c["H"] + c["Hkv"]) * c["rot"] + 8 * c["Hkv"] * c["D"])}
    e = c["rows"] * c["n"]
    return {"bytes": e * (3 * SIZE[c["dtype"]] + SIZE[c["out"]]) + (e if c["gate"] == "all" else c["n"] if c["gate"] == "row" else 0) * SIZE[c["dtype"]]
            + 4 * c["n"] * (2 if c["post"] else 1), "flops": 12 * e}


# ---------------------------------------------------------------------------------------
# from the definitions, in 64 bits


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "route":
        x = s["scores"].double()
        p = torch.softmax(x, 1) if c["gating"] == "softmax" else torch.sigmoid(x)
        pick = p.clone() if s["bias"] is None else p + s["bias"].double()
        T, E, n = c["T"], c["E"], c["E"] // c["groups"]
        if c["groups"] > 1:
            value = torch.stack([pick[:, i * n : (i + 1) * n].topk(min(2, n), 1)[0].sum(1) for i in range(c["groups"])], 1)
            open_ = torch.zeros((T, c["groups"]), dtype=torch.bool, device="cuda")
            for _ in range(c["top_groups"]):
                best = value.masked_fill(open_, -math.inf)
                # the lowest index among the largest
                first = (best == best.amax(1, keepdim=True)).int().argmax(1)
                open_[torch.arange(T, device="cuda"), first] = True
            pick = pick.masked_fill(~open_.repeat_interleave(n, 1), -math.inf)
        ids = torch.empty((T, c["k"]), dtype=torch.int64, device="cuda")
        for j in range(c["k"]):
            ids[:, j] = (pick == pick.amax(1, keepdim=True)).int().argmax(1)
            pick[torch.arange(T, device="cuda"), ids[:, j]] = -math.inf
        w = p[torch.arange(T, device="cuda")[:, None], ids]
        return {"ids": ids.to(torch.int32), "w": w * (c["scale"] / w.sum(1, keepdim=True) if c["normalise"] else c["scale"])}
    if c["op"] == "moe":
        step = {I8: 1, I4: 2, I2: 4}[c["fmt"]]

        def matrix(m, e):
            rows, cols, codes, scales = s["mats"][m]
            q = torch.empty((rows, codes.shape[2] * step), dtype=torch.float64, device="cuda")
            byte = codes[e].long()
            for i in range(step):
                part = byte // 2 ** (BITS[c["fmt"]] * i) % 2 ** BITS[c["fmt"]]
                q[:, i::step] = (torch.where(part > 127, part - 256, part) if c["fmt"] == I8 else part - 2 ** (BITS[c["fmt"]] - 1)).double()
            q = q[:, :cols]
            if c["gs"]:
                return q * scales[e].double()[:, torch.arange(cols, device="cuda") // c["gs"]]
            return q * scales[e].double()[:, None]

        y = torch.zeros((c["T"], c["D"]), dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()
        x, w = s["x"].double(), s["w"].double()
        for e in range(c["E"]):
            share = torch.where(s["ids"] == e, w, torch.zeros_like(w)).sum(1)
            has = (s["ids"] == e).any(1).nonzero()[:, 0]
            if len(has):
                g = x[has] @ matrix(0, e).T
                y[has] += share[has, None] * ((g * torch.sigmoid(g) * (x[has] @ matrix(1, e).T)) @ matrix(2, e).T)
        return {"y": y}
    if c["op"] == "append":
        q_lens, kv_lens = _lens(c)
        place = torch.cat([torch.arange(kv - n, kv, device="cuda") for n, kv in zip(q_lens, kv_lens)])

        def turned(x):
            x, first = x.double(), 0
            y = x.clone()
            for axis, n in enumerate(_sections(c)):
                at = place if s["pos"] is None else s["pos"][axis]
                for i in range(first, first + n):
                    phi = at.double() * math.exp(-2 * i / c["rot"] * math.log(1e6))
                    a, b = (i, i + c["rot"] // 2) if c["pairing"] == 0 else (2 * i, 2 * i + 1)
                    z = torch.complex(x[..., a], x[..., b]) * torch.polar(torch.ones_like(phi), phi)[:, None]
                    y[..., a], y[..., b] = z.real, z.imag
                first += n
            return y

        def nearest(x):
            x = x.float().double()  # what is quantised is a 32-bit value by definition
            top = x.abs().amax(-1, keepdim=True)
            if c["kind"] == KV_F16:  # 11 significant bits, down to 2^-24 of the scale
                scale = torch.exp2(torch.floor(torch.log2(top)) - 14)
                z = x / scale
                step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -14))) - 10)
                return torch.round(z / step) * step * scale
            scale = (top / (127 if c["kind"] == KV_I8 else 7)).float().double()  # a 32-bit value by definition
            return torch.round(x / scale) * scale
        return {"q": turned(s["q"]), "k": nearest(turned(s["new_k"])), "v": nearest(s["new_v"])}
    z = s["x"].double()
    if c["post"]:
        z = z / (z.pow(2).mean(1, keepdim=True) + EPS).sqrt() * s["w_post"].double()
    r = s["res"].double() + ALPHA * (z if s["gate"] is None else z * s["gate"].double())
    return {"y": r / (r.pow(2).mean(1, keepdim=True) + EPS).sqrt() * s["w_pre"].double(), "sum": r}
