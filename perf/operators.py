"""Cases for measuring the operators between a decoder layer's products, with their plain forms.

Four operators: the root-mean-square norm with the residual's addition ("norm"), rotary positions
with several axes ("rope"), a key/value cache that is quantised as it is written and read back
("kv_write", "kv_read"), and the attention of new tokens over that paged cache ("attn").

The plain forms are elementary torch operations in 32 bits (64 where 32 lose what matters: angles of
far positions, values next to a rounding border). With `own` set, run() makes the calls of
weight_only_quantized_matmul_amd instead, on the same inputs.

The cache, as both sides have it: pools k, v uint8 [pages, kv heads, page, row bytes] and k_scale,
v_scale float32 [pages, kv heads, page]; a row holds D codes of one token and head (float16, int8, or
two 4-bit codes a byte, the even element in the low half, stored as code + 8) and stands for code * scale.
Sequence b's position t lies in slot t % page of page table[b, t // page]; its q_len[b] =
q_start[b+1] - q_start[b] new tokens are the last of its kv_len[b] positions.
"""
import math
import random

import torch

own = False

F16, I8, I4 = 0, 1, 2  # cache kinds
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "i8": 1}
TINY = 2.0 ** -100  # a row whose largest magnitude is below this is stored as zeros


def _attn(name, **kw):
    c = {"name": name, "op": "attn", "H": 48, "Hkv": 8, "D": 128, "page": 64, "kind": I8, "dtype": "f32", "B": 1,
         "q_max": 1, "kv_max": 1500, "ragged": False, "causal": True, "window": 0, "lens": 1}
    c.update(kw)
    return c


def _kv(name, op, **kw):
    c = {"name": name, "op": op, "Hkv": 8, "D": 128, "page": 64, "kind": I8, "dtype": "f32", "B": 64, "q_max": 1,
         "kv_max": 2000, "ragged": True, "lens": 1}
    c.update(kw)
    return c


def listed():
    # hidden size 6144 as in the repository's benchmark: 48 query heads of 128, here over 8 key/value heads
    return [
        # one user, one token, a short context: the latency of a step
        _attn("attn_decode_one"),
        # a serving batch of 64 users with contexts of all lengths up to 8192, one token each
        _attn("attn_decode_batch", B=64, kv_max=8192, ragged=True, lens=2),
        # four long documents in a 4-bit cache
        _attn("attn_decode_long", B=4, kv_max=131072, kind=I4, page=128, lens=3),
        # chunked prefill beside decode: ragged chunks of up to 511 new tokens on contexts up to 5000, odd sizes, sliding window
        _attn("attn_chunk_mixed", B=8, q_max=511, kv_max=5000, ragged=True, window=4096, page=16, lens=4),
        # the prefill of one prompt in 16-bit activations and a 16-bit cache
        _attn("attn_prefill", H=32, q_max=4096, kv_max=4096, kind=F16, dtype="bf16", lens=5),
        # a decode step's new keys and values of 64 users go into the cache, and come back as the values they stand for
        _kv("kv_write_decode", "kv_write", lens=6),
        # a prefill's 8191 new tokens in bf16 go into a 4-bit cache
        _kv("kv_write_prefill", "kv_write", B=4, q_max=4096, kv_max=6000, kind=I4, dtype="bf16", lens=7),
        # whole contexts are read back in bf16 (to move them or to check them)
        _kv("kv_read_context", "kv_read", B=4, q_max=32768, kv_max=32768, dtype="bf16", ragged=False, lens=8),
        # one token's norm before a product
        {"name": "norm_decode", "op": "norm", "rows": 1, "n": 6144, "dtype": "f32", "out": "f32", "res": True},
        # a prefill's rows, out in 8 bits
        {"name": "norm_prefill_8bit", "op": "norm", "rows": 8191, "n": 6144, "dtype": "bf16", "out": "i8", "res": True},
        # a decode step's queries and keys (48 + 8 heads), positions up to a million
        {"name": "rope_decode", "op": "rope", "T": 64, "H": 56, "D": 128, "rot": 128, "pairing": 0, "axes": 1, "far": 1000000, "dtype": "f32"},
        # an image's or a video's tokens: time, height and width
        {"name": "rope_video", "op": "rope", "T": 8191, "H": 40, "D": 128, "rot": 128, "pairing": 0, "axes": 3, "far": 4096, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "kv_write", "kv_read", "norm", "rope"])
    dtype = rng.choice(["f32", "f32", "bf16", "f16"])
    if op == "norm":
        n = _log(rng, 64, 16384)
        rows = min(_log(rng, 1, 16384), 50_000_000 // n)
        return {"op": op, "rows": rows, "n": n, "dtype": dtype, "out": rng.choice(["f32", "bf16", "f16", "i8"]), "res": rng.random() < 0.7}
    D = rng.choice([64, 128, 128, 256])
    if op == "rope":
        rot = rng.choice([D, D, D // 2])
        H = rng.randint(1, 64)
        T = min(_log(rng, 1, 16384), 40_000_000 // (H * D))
        return {"op": op, "T": max(1, T), "H": H, "D": D, "rot": rot, "pairing": rng.choice([0, 1]), "axes": rng.choice([1, 2, 3, 4]),
                "far": _log(rng, 100, 2_000_000), "dtype": dtype}
    kind, page = rng.choice([F16, I8, I4]), rng.choice([16, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    if op != "attn":
        B, q_max = _log(rng, 1, 256), _log(rng, 1, 8192)
        q_max = max(1, min(q_max, 30_000_000 // (B * Hkv * D)))
        return {"op": op, "Hkv": Hkv, "D": D, "page": page, "kind": kind, "dtype": dtype, "B": B, "q_max": q_max,
                "kv_max": q_max + rng.randint(0, 4000), "ragged": True, "lens": rng.randrange(1 << 30)}
    G = rng.choice([1, 2, 3, 4, 6, 8, 12])
    if rng.random() < 0.5:  # decode, or a few tokens at a time
        B, q_max = _log(rng, 1, 128), rng.choice([1, 1, 1, 2, 5])
        kv_max = max(q_max + 1, min(_log(rng, 1, 100_000), 40_000_000 // (B * Hkv * D), 400_000_000 // (B * Hkv * G * q_max)))
    else:
        B, q_max = _log(rng, 1, 16), _log(rng, 6, 2048)
        kv_max = q_max + _log(rng, 1, 8000)
        q_max = max(1, min(q_max, 300_000_000 // (B * Hkv * G * kv_max)))
    causal = rng.random() < 0.85
    return {"op": op, "H": Hkv * G, "Hkv": Hkv, "D": D, "page": page, "kind": kind, "dtype": dtype, "B": B, "q_max": q_max, "kv_max": kv_max,
            "ragged": True, "causal": causal, "window": rng.choice([0, 0, 0, rng.randint(1, kv_max)]) if causal else 0, "lens": rng.randrange(1 << 30)}


# ---------------------------------------------------------------------------------------
# inputs


def _lens(c):
    """(q_len, kv_len) of every sequence: by the case alone."""
    rng = random.Random(c["lens"])
    q, kv = [], []
    for b in range(c["B"]):
        n = c["q_max"] if b == 0 or not c["ragged"] or c["q_max"] == 1 else rng.choice([1, rng.randint(1, c["q_max"]), c["q_max"]])
        q.append(n)
        kv.append(c["kv_max"] if b == 0 or not c["ragged"] else rng.randint(min(n, c["kv_max"]), c["kv_max"]))
    return q, kv


def _row_bytes(kind, D):
    return 2 * D if kind == F16 else D if kind == I8 else D // 2


def _codes(shape, kind, g):
    """A pool of codes as a written cache holds them: bell-shaped, the largest of a row near the end of the range."""
    x = torch.randn(shape, device="cuda", generator=g)
    if kind == F16:
        return (x * 8000.0).clamp_(-32000, 32000).half().view(torch.uint8)
    if kind == I8:
        return (x * 40).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
    n = (x * 2.5).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _unit(kind):
    """The scale with which such codes have a spread of about 1."""
    return 1 / 8000 if kind == F16 else 1 / 40 if kind == I8 else 1 / 2.5


def _paging(c, g):
    """A pool's size and a page table with its pages in no order; entries past a sequence's end are -1."""
    q, kv = _lens(c)
    need = [-(-n // c["page"]) for n in kv]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, device="cuda", generator=g)[: sum(need)].to(torch.int32)
    wide = max(need)
    first = torch.tensor([0] + need, device="cuda").cumsum(0)
    at = torch.arange(wide, device="cuda")
    have = at[None, :] < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(have, order[(first[:-1, None] + at).clamp(max=len(order) - 1)], torch.full((), -1, device="cuda", dtype=torch.int32))
    start = torch.tensor([0] + q, device="cuda", dtype=torch.int32).cumsum(0).to(torch.int32)
    return n_pages, table.contiguous(), start, torch.tensor(kv, device="cuda", dtype=torch.int32), sum(q)


def prepare(case, seed):
    c, dt = dict(case), DTYPES[case["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def randn(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    s = {"c": c}
    if c["op"] == "norm":
        rows, n = c["rows"], c["n"]
        s["x"] = (randn(rows, n) * 0.7).to(dt)
        s["res"] = (randn(rows, n) * 2).to(dt) if c["res"] else None
        s["w"] = 1 + 0.2 * randn(n)
        if own:
            import weight_only_quantized_matmul_amd as wq
            wq.wq_init([0])
            out = torch.int8 if c["out"] == "i8" else DTYPES[c["out"]]
            s["y"] = torch.empty((rows, n), dtype=out, device="cuda")
            s["scale"] = torch.empty(rows, device="cuda") if c["out"] == "i8" else None
            s["sum"] = torch.empty((rows, n), dtype=dt, device="cuda") if c["res"] else None
    elif c["op"] == "rope":
        s["x"] = randn(c["T"], c["H"], c["D"]).to(dt)
        s["pos"] = torch.randint(0, c["far"] + 1, (c["axes"], c["T"]), device="cuda", generator=g, dtype=torch.int32)
        s["sections"] = _sections(c)
        if own:
            import weight_only_quantized_matmul_amd as wq
            wq.wq_init([0])
            s["rope"] = wq.wq_rope_create(c["rot"], c["pairing"], 1e6, s["sections"])
            s["y"] = torch.empty_like(s["x"])
    else:
        n_pages, s["table"], s["start"], s["kv_len"], T = _paging(c, g)
        shape = (n_pages, c["Hkv"], c["page"])
        if c["op"] == "kv_write":
            rb = _row_bytes(c["kind"], c["D"])
            s["k"], s["v"] = (torch.zeros(shape + (rb,), dtype=torch.uint8, device="cuda") for _ in "kv")
            s["ks"], s["vs"] = (torch.zeros(shape, device="cuda") for _ in "kv")
            # keys have a few channels much larger than the others
            loud = 1 + 7 * (torch.rand(c["Hkv"], c["D"], device="cuda", generator=g) < 0.04)
            s["new_k"], s["new_v"] = (randn(T, c["Hkv"], c["D"]) * loud).to(dt), randn(T, c["Hkv"], c["D"]).to(dt)
        else:
            s["k"], s["v"] = (_codes(shape + (c["D"],), c["kind"], g) for _ in "kv")
            s["ks"], s["vs"] = ((0.5 + torch.rand(shape, device="cuda", generator=g)) * _unit(c["kind"]) for _ in "kv")
        if c["op"] == "attn":
            s["q"] = (randn(T, c["H"], c["D"]) * 2.5).to(dt)
        if own:
            import weight_only_quantized_matmul_amd as wq
            wq.wq_init([0])
            s["cache"] = wq.KvCache(c["kind"], s["k"], s["v"], s["ks"], s["vs"])
            s["batch"] = wq.KvBatch(s["start"], s["kv_len"], s["table"], T, max_q=max(_lens(c)[0]), max_kv=max(_lens(c)[1]))
            if c["op"] == "attn":
                s["o"], s["lse"] = torch.empty_like(s["q"]), torch.empty((T, c["H"]), device="cuda")
            else:
                back = torch.float32 if c["op"] == "kv_write" else dt
                s["out_k"], s["out_v"] = (torch.empty((T, c["Hkv"], c["D"]), dtype=back, device="cuda") for _ in "kv")
    return s


def _sections(c):
    """Frequencies for each axis: the first axis takes what the others leave."""
    half = c["rot"] // 2
    rest = [half * 3 // 8] * (c["axes"] - 1) if c["axes"] <= 3 else [half // 4] * 3
    return [half - sum(rest)] + rest


# ---------------------------------------------------------------------------------------
# one pass


def run(s):
    c = s["c"]
    if own:
        import weight_only_quantized_matmul_amd as wq
        if c["op"] == "norm":
            wq.wq_rmsnorm_dev(s["x"], s["w"], 1e-6, s["y"], residual=s["res"], sum_out=s["sum"], y_scale=s["scale"])
            y = s["y"] if s["scale"] is None else s["y"] * s["scale"][:, None]
            return {"y": y, "sum": s["sum"]}
        if c["op"] == "rope":
            wq.wq_rope_dev(s["rope"], s["x"], s["pos"], s["y"])
            return {"y": s["y"]}
        if c["op"] == "attn":
            wq.wq_attn_paged_dev(s["cache"], s["batch"], s["q"], s["o"], scale=c["D"] ** -0.5, causal=c["causal"], window=c["window"], lse=s["lse"])
            return {"o": s["o"], "lse": s["lse"]}
        if c["op"] == "kv_write":
            wq.wq_kv_append_dev(s["cache"], s["batch"], s["new_k"], s["new_v"])
        wq.wq_kv_read_dev(s["cache"], s["batch"], s["out_k"], s["out_v"])
        return {"k": s["out_k"], "v": s["out_v"]}
    return {"norm": _norm, "rope": _rope, "attn": _attention, "kv_write": _write, "kv_read": _read}[c["op"]](s)


def _norm(s):
    c = s["c"]
    r = s["x"].float() if s["res"] is None else s["x"].float() + s["res"].float()
    rstd = torch.rsqrt(r.square().mean(1, keepdim=True) + 1e-6)
    if c["out"] == "i8":
        t = r.double() * s["w"].double()  # codes next to a border
        top = t.abs().amax(1, keepdim=True)
        y = ((t * 127) / top).round().float() * (top * rstd / 127).float()
    else:
        y = (r * rstd * s["w"]).to(DTYPES[c["out"]])
    return {"y": y, "sum": None if s["res"] is None else r.to(s["x"].dtype)}


def _angles(c, pos, sections):
    i = torch.arange(c["rot"] // 2, device=pos.device, dtype=torch.float64)
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=pos.device), torch.tensor(sections, device=pos.device))
    return pos[axis].double().t() * (1e6 ** (-2 * i / c["rot"]))  # [T, rot/2]


def _rope(s):
    c, x = s["c"], s["x"].float()
    phi = _angles(c, s["pos"], s["sections"])
    cos, sin = phi.cos().float()[:, None], phi.sin().float()[:, None]
    turned, half = x[..., : c["rot"]], c["rot"] // 2
    if c["pairing"] == 0:
        a, b = turned[..., :half], turned[..., half:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return {"y": torch.cat([y, x[..., c["rot"] :]], -1).to(s["x"].dtype)}


def _places(s):
    """Page and slot of every new token."""
    at = torch.arange(sum(_lens(s["c"])[0]), device="cuda")
    b = torch.searchsorted(s["start"][1:].long(), at, right=True)
    p = s["kv_len"].long()[b] - (s["start"][1:] - s["start"][:-1]).long()[b] + at - s["start"].long()[b]
    return s["table"][b, p // s["c"]["page"]].long(), p % s["c"]["page"]


def _open(rows, kind):
    """The codes of cache rows, as float32."""
    if kind == F16:
        return rows.view(torch.float16).float()
    if kind == I8:
        return rows.view(torch.int8).float()
    return torch.stack([(rows & 15).float() - 8, (rows >> 4).float() - 8], -1).flatten(-2)


def _quantise(x, kind):
    """(rows of codes, scales) of x [..., D]."""
    x = x.float()
    top = x.abs().amax(-1)
    if kind == F16:
        scale = top / torch.frexp(top)[0] * 2.0 ** -15  # a power of two: the largest magnitude becomes [2^14, 2^15)
        rows = (x.double() / scale.double()[..., None]).float().half().view(torch.uint8)
    else:
        scale = (top.double() / (127 if kind == I8 else 7)).float()
        code = torch.where(top[..., None] < TINY, torch.zeros((), device="cuda", dtype=torch.float64), (x.double() / scale.double()[..., None]).round())
        rows = code.to(torch.int8).view(torch.uint8)
        if kind == I4:
            rows = (code + 8).to(torch.uint8)
            rows = rows[..., 0::2] | (rows[..., 1::2] << 4)
    zero = top < TINY
    return torch.where(zero[..., None], torch.full((), 0x88 if kind == I4 else 0, device="cuda", dtype=torch.uint8), rows), torch.where(zero, torch.zeros_like(scale), scale)


def _write(s):
    c = s["c"]
    page, slot = _places(s)
    head = torch.arange(c["Hkv"], device="cuda")[None, :]
    for x, rows, scales in ((s["new_k"], s["k"], s["ks"]), (s["new_v"], s["v"], s["vs"])):
        got = _quantise(x, c["kind"])
        rows[page[:, None], head, slot[:, None]], scales[page[:, None], head, slot[:, None]] = got
    return _read(s, torch.float32)


def _read(s, dtype=None):
    c = s["c"]
    page, slot = _places(s)
    at = (page[:, None], torch.arange(c["Hkv"], device="cuda")[None, :], slot[:, None])
    k, v = (_open(rows[at], c["kind"]) * scales[at][..., None] for rows, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])))
    dtype = dtype or DTYPES[c["dtype"]]
    return {"k": k.to(dtype), "v": v.to(dtype)}


def _attention(s):
    c = s["c"]
    B, H, Hkv, D, G = c["B"], c["H"], c["Hkv"], c["D"], c["H"] // c["Hkv"]
    table = s["table"].long().clamp(min=0)
    k, v = ((_open(rows[table], c["kind"]) * scales[table][..., None]).transpose(2, 3).reshape(B, -1, Hkv, D).transpose(1, 2).contiguous()
            for rows, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])))  # [B, Hkv, positions, D]
    start, kv_len = s["start"].long(), s["kv_len"].long()
    q_len = start[1:] - start[:-1]
    i = torch.arange(max(_lens(c)[0]), device="cuda")
    token = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)  # [B, q]
    q = s["q"].float()[token].reshape(B, -1, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)
    score = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(D ** -0.5)  # [B, Hkv, q * G, positions]
    t = torch.arange(k.shape[2], device="cuda")
    p = (kv_len - q_len)[:, None] + i  # [B, q]
    seen = (t < kv_len[:, None])[:, None, :].expand(B, len(i), -1)
    if c["causal"]:
        seen = seen & (t <= p[..., None])
    if c["window"]:
        seen = seen & (t > p[..., None] - c["window"])
    seen = seen.repeat_interleave(G, 1)[:, None]
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    score = score.sub_(top).exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score, v) / torch.where(total == 0, torch.ones_like(total), total)
    lse = total.log() + top
    o = o.reshape(B, Hkv, len(i), G, D).permute(0, 2, 1, 3, 4).reshape(B, len(i), H, D)
    lse = lse.reshape(B, Hkv, len(i), G).permute(0, 2, 1, 3).reshape(B, len(i), H)
    real = i < q_len[:, None]
    return {"o": o[real].to(s["q"].dtype), "lse": lse[real]}


# ---------------------------------------------------------------------------------------
# what a pass cannot do without


def _pairs(c):
    """(query, key) pairs that are seen, and keys that some query of the sequence sees, over all sequences."""
    pairs = keys = 0
    for q, kv in zip(*_lens(c)):
        low = kv
        for i in range(q):
            p = kv - q + i
            hi = min(p + 1, kv) if c["causal"] else kv
            lo = max(0, p + 1 - c["window"]) if c["window"] else 0
            pairs += max(0, hi - lo)
            low = min(low, lo)
        keys += kv - low
    return pairs, keys


def work(case):
    c = case
    if c["op"] == "norm":
        e, moved = c["rows"] * c["n"], SIZE[c["dtype"]] * (3 if c["res"] else 1)
        return {"bytes": e * (moved + SIZE[c["out"]]) + 4 * c["n"] + (4 * c["rows"] if c["out"] == "i8" else 0), "flops": 6 * e}
    if c["op"] == "rope":
        e = c["T"] * c["H"] * c["D"]
        return {"bytes": 2 * e * SIZE[c["dtype"]] + 4 * c["axes"] * c["T"], "flops": 3 * c["T"] * c["H"] * c["rot"]}
    row = _row_bytes(c["kind"], c["D"]) + 4
    T = sum(_lens(c)[0])
    if c["op"] == "attn":
        pairs, keys = _pairs(c)
        return {"bytes": 2 * T * c["H"] * c["D"] * SIZE[c["dtype"]] + 4 * T * c["H"] + 2 * keys * c["Hkv"] * row, "flops": 4 * pairs * c["H"] * c["D"]}
    rows = 2 * T * c["Hkv"]
    if c["op"] == "kv_write":  # read, write the codes, read them back, write the values
        return {"bytes": rows * (c["D"] * SIZE[c["dtype"]] + 2 * row + 4 * c["D"]), "flops": 4 * rows * c["D"]}
    return {"bytes": rows * (row + c["D"] * SIZE[c["dtype"]]), "flops": rows * c["D"]}


# ---------------------------------------------------------------------------------------
# from the definitions, in 64 bits


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "norm":
        # the residual's sum is a 32-bit value by definition; what follows is exact
        r = (s["x"].float() + (0 if s["res"] is None else s["res"].float())).double()
        y = r / (r.pow(2).mean(1, keepdim=True) + 1e-6).sqrt() * s["w"].double()
        if c["out"] == "i8":
            t = r * s["w"].double()
            step = y.abs().amax(1, keepdim=True) / 127
            y = torch.round(127 * t / t.abs().amax(1, keepdim=True)) * step
        return {"y": y, "sum": None if s["res"] is None else r}
    if c["op"] == "rope":
        x, half = s["x"].double(), c["rot"] // 2
        y, first = x.clone(), 0
        for axis, n in enumerate(s["sections"]):
            for i in range(first, first + n):
                phi = s["pos"][axis].double() * math.exp(-2 * i / c["rot"] * math.log(1e6))
                turn = torch.polar(torch.ones_like(phi), phi)[:, None]
                a, b = (i, i + half) if c["pairing"] == 0 else (2 * i, 2 * i + 1)
                z = torch.complex(x[..., a], x[..., b]) * turn
                y[..., a], y[..., b] = z.real, z.imag
            first += n
        return {"y": y}
    q_lens, kv_lens = _lens(c)
    table = s["table"].tolist()

    def positions(b, first):
        t = torch.arange(first, kv_lens[b], device="cuda")
        return torch.tensor(table[b], device="cuda")[t // c["page"]], t % c["page"]

    def values(rows, scales, b, first, h=None):
        page, slot = positions(b, first)
        rows, scales = (rows[page, :, slot], scales[page, :, slot]) if h is None else (rows[page, h, slot], scales[page, h, slot])
        if c["kind"] == F16:
            codes = rows.view(torch.float16).double()
        elif c["kind"] == I8:
            codes = rows.view(torch.int8).double()
        else:
            codes = torch.empty(rows.shape[:-1] + (c["D"],), dtype=torch.float64, device="cuda")
            codes[..., 0::2], codes[..., 1::2] = (rows % 16).double() - 8, (rows // 16).double() - 8
        return codes * scales.double()[..., None]

    if c["op"] == "kv_write":
        def nearest(x):
            x = x.double()
            top = x.abs().amax(-1, keepdim=True)
            if c["kind"] == F16:  # 11 significant bits, down to 2^-24 of the scale
                scale = torch.exp2(torch.floor(torch.log2(top)) - 14)
                z = x / scale
                step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -14))) - 10)
                return torch.round(z / step) * step * scale
            n = 127 if c["kind"] == I8 else 7
            scale = (top / n).float().double()  # a 32-bit value by definition
            return torch.round(x / scale) * scale
        return {"k": nearest(s["new_k"]), "v": nearest(s["new_v"])}
    if c["op"] == "kv_read":
        return {n: torch.cat([values(s[n], s[n + "s"], b, kv_lens[b] - q_lens[b]) for b in range(c["B"])]) for n in "kv"}
    T, H, G, D = sum(q_lens), c["H"], c["H"] // c["Hkv"], c["D"]
    if 4 * _pairs(c)[0] * H * D > 2e12:
        return None
    o = torch.zeros((T, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for b in range(c["B"]):
        n, kv = q_lens[b], kv_lens[b]
        if kv > 0 and n > 0:
            p = kv - n + torch.arange(n, device="cuda")[:, None]
            t = torch.arange(kv, device="cuda")[None, :]
            hidden = torch.zeros((n, kv), dtype=torch.bool, device="cuda")
            if c["causal"]:
                hidden |= t > p
            if c["window"]:
                hidden |= t <= p - c["window"]
            for h in range(c["Hkv"]):
                kk, vv = values(s["k"], s["ks"], b, 0, h), values(s["v"], s["vs"], b, 0, h)
                for j in range(h * G, h * G + G):
                    z = (s["q"][first : first + n, j].double() @ kk.t()) / math.sqrt(D)
                    z = torch.where(hidden, torch.full((), -math.inf, device="cuda", dtype=torch.float64), z)
                    l = torch.logsumexp(z, 1)
                    w = torch.where(hidden, torch.zeros((), device="cuda", dtype=torch.float64), (z - l[:, None]).exp())
                    o[first : first + n, j], lse[first : first + n, j] = w @ vv, l
        first += n
    return {"o": o, "lse": lse}
