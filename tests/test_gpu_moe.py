"""The choice of experts and the expert layer against their plain forms in 64 bits."""
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

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LOWEST = {"f32": -3.4028234663852886e38, "bf16": -3.3895313892515355e38, "f16": -65504.0}


@pytest.fixture(autouse=True)
def _init():
    gu.reinit_with_env(WQ_FAULT=None, WQ_MEM_LIMIT_BYTES=None)
    yield
    torch.cuda.synchronize()


def run_route(scores, k, bias=None, stream=None, **kw):
    T = scores.shape[0]
    ids = torch.full((T + 2, k), -77, dtype=torch.int32, device="cuda")
    w = torch.full((T + 2, k), -77.0, device="cuda")
    kw["gating"] = wq.WQ_GATE_SOFTMAX if kw.get("gating", "softmax") == "softmax" else wq.WQ_GATE_SIGMOID
    wq.wq_moe_route_dev(scores, ids[1:T + 1], w[1:T + 1], bias=bias, stream=stream, **kw)
    torch.cuda.synchronize()
    for t in (ids, w):
        assert (t[0] == -77).all() and (t[T + 1] == -77).all(), "a row outside the tokens was written"
    return ids[1:T + 1].cpu().numpy(), w[1:T + 1].cpu().numpy()


def check_route(scores, k, bias=None, **kw):
    gu.banner("route %s k=%d %s" % (tuple(scores.shape), k, kw))
    ids, w = run_route(scores, k, None if bias is None else torch.from_numpy(bias).cuda(), **kw)
    want_ids, want_w = ref.route(scores.double().cpu().numpy(), k, bias, **kw)
    assert (ids == want_ids).all()
    # one rounding to fp32 of a value whose fp64 sums and exponentials are within 1e-12
    assert (np.abs(w - want_w) <= (2.0 ** -24 + 1e-12) * np.abs(want_w) + 2.0 ** -149).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k,kw", [
    (1, 1, 1, {}), (1, 8, 2, {}), (3, 7, 7, dict(gating="sigmoid")), (5, 60, 4, dict(normalise=False)), (2, 64, 6, dict(scale=2.5)),
    (9, 65, 32, {}), (4, 128, 8, dict(gating="sigmoid", groups=8, top_groups=3)), (6, 256, 8, dict(gating="sigmoid", groups=8, top_groups=4, scale=2.5)),
    (3, 320, 6, dict(groups=64, top_groups=5)), (2, 1000, 11, dict(groups=4, top_groups=1)), (2, 1024, 32, dict(gating="sigmoid")),
    (130, 160, 6, dict(groups=20, top_groups=20)), (3, 6, 2, dict(groups=6, top_groups=2)), (3, 9, 3, dict(groups=3, top_groups=1))])
@pytest.mark.parametrize("bias", [False, True])
def test_route(dtype, T, E, k, kw, bias):
    rng = np.random.default_rng(E + T)
    s = torch.from_numpy(rng.normal(0, 1.5, (T, E)).astype(np.float32)).cuda().to(DT[dtype])
    check_route(s, k, rng.normal(0, 0.05, E).astype(np.float32) if bias else None, **kw)


@pytest.mark.parametrize("gating", ["softmax", "sigmoid"])
def test_route_ties_go_to_the_lowest(gating):
    rng = np.random.default_rng(3)
    s = torch.from_numpy(rng.integers(0, 3, (17, 130)).astype(np.float32)).cuda()
    check_route(s, 9, gating=gating)
    check_route(s, 9, gating=gating, groups=10, top_groups=3)
    check_route(torch.zeros((2, 512), device="cuda"), 32, gating=gating, groups=16, top_groups=7)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gating", ["softmax", "sigmoid"])
def test_route_masked_infinite_and_nan_scores(dtype, gating):
    inf, nan, low = float("inf"), float("nan"), LOWEST[dtype]
    rows = [[-inf] * 5 + [1.0, 2.0, -inf], [low] * 8, [low] * 7 + [0.0], [-inf] * 8, [nan] * 8, [nan, 1.0, -inf, 2.0, nan, 0.0, -1.0, low],
            [inf, 1.0, inf, 0.0, -inf, nan, 2.0, 3.0], [-low, low, 0.0, 1.0, 2.0, 3.0, -low, 4.0]]
    s = torch.tensor(rows, dtype=torch.float32).to(DT[dtype]).cuda()
    for norm in (True, False):
        check_route(s, 3, gating=gating, normalise=norm)
        check_route(s, 8, gating=gating, normalise=norm)
        check_route(s, 2, gating=gating, normalise=norm, groups=4, top_groups=2)


def test_route_strides_and_nothing():
    big = torch.randn((40, 3 * 77 + 1), device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    check_route(big[::2, 5:82], 5)
    check_route(big.to(torch.bfloat16)[1::3, 1:64], 5)
    wq.wq_moe_route_dev(big[:0, :64], torch.empty((0, 4), dtype=torch.int32, device="cuda"), torch.empty((0, 4), device="cuda"))


def test_route_more_tokens_than_a_launch_has_threads():
    T = (1 << 32) // 64 + 7  # a wave a token
    ids, w = torch.full((T, 1), -77, dtype=torch.int32, device="cuda"), torch.zeros((T, 1), device="cuda")
    gu.banner("route (%d, 1)" % T)
    wq.wq_moe_route_dev(torch.ones((T, 1), dtype=torch.bfloat16, device="cuda"), ids, w, scale=0.5)
    torch.cuda.synchronize()
    assert int(ids.abs().max()) == 0 and float(w.min()) == 0.5 and float(w.max()) == 0.5


def test_route_refusals_of_the_binding():
    s = torch.zeros((2, 8), device="cuda")
    ids, w = torch.empty((2, 4), dtype=torch.int32, device="cuda"), torch.empty((2, 4), device="cuda")
    for args in ((s, ids.long(), w), (s, ids, w.double()), (s, ids[:1], w), (s, ids, w[:, :2]), (s.cpu(), ids, w),
                 (s, torch.empty((2, 8), dtype=torch.int32, device="cuda")[:, ::2], w), (s.t(), ids, w)):
        with pytest.raises(ValueError):
            wq.wq_moe_route_dev(*args)
    with pytest.raises(ValueError):
        wq.wq_moe_route_dev(s, ids, w, bias=torch.zeros(7, device="cuda"))
    with pytest.raises(wq.WqError):
        wq.wq_moe_route_dev(s, ids, w, groups=3)


# ---------------------------------------------------------------------------------------


class Layer:
    def __init__(self, rng, fmt, E, D, F, O=None, gs=0, spread=1.0):
        O = D if O is None else O
        self.E, self.D, self.F, self.O = E, D, F, O
        handles, self.mats = [], []
        opened = []
        for rows, cols in ((F, D), (F, D), (O, F)):
            hs, ms = [], []
            for _ in range(E):
                codes = rng.integers(0, 256, (rows, -(-cols * ref.BITS[fmt] // 8)), dtype=np.uint8)
                shape = (rows, -(-cols // gs)) if gs else (rows,)
                scales = (rng.uniform(0.5, 1.5, shape) * spread / ({1: 74, 2: 4.6, 3: 1.2}[fmt] * np.sqrt(cols))).astype(np.float32)
                if gs:
                    hs.append(wq.wq_tensor_upload_gs(None, 0, fmt, rows, cols, gs, codes, scales))
                else:
                    hs.append(wq.wq_tensor_upload(None, 0, fmt, rows, cols, codes, scales))
                ms.append(ref.open_matrix(codes, scales, cols, fmt, gs))
            handles.append(hs)
            opened.append(ms)
        self.handles = handles
        self.mats = list(zip(*opened))
        self.moe = wq.wq_moe_create(*handles)

    def free(self):
        torch.cuda.synchronize()
        wq.wq_moe_free(self.moe)
        for t in sum(self.handles, []):
            wq.wq_tensor_free(t)


def choose(rng, T, E, k):
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    return ids, rng.uniform(0.1, 1.0, (T, k)).astype(np.float32)


def check_moe(layer, x, ids, w, dtype, add=None, what=""):
    """x, add: tensors on the GPU in their type; ids, w numpy."""
    T = x.shape[0]
    gu.banner("moe %s T=%d k=%d E=%d D=%d F=%d O=%d %s" % (what, T, ids.shape[1], layer.E, layer.D, layer.F, layer.O, dtype))
    room = torch.full((T + 2, layer.O + 3), 7.0, dtype=x.dtype, device="cuda")
    y = room[1:T + 1, 1:layer.O + 1]
    wq.wq_moe_ffn_dev(layer.moe, x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), y, add=add)
    torch.cuda.synchronize()
    edge = room.clone()
    edge[1:T + 1, 1:layer.O + 1] = 7.0
    assert (edge == 7.0).all(), "written outside of y"
    want, bound = ref.moe(x.double().cpu().numpy(), ids, w, layer.mats, None if add is None else add.double().cpu().numpy())
    bound = bound + ref.HALF[dtype] * (np.abs(want) + bound) + ref.TINY[dtype]
    err = np.abs(y.double().cpu().numpy() - want)
    assert (err <= bound).all(), "worst err/bound %.3g" % (err / bound).max()
    return y.clone()


def rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((rng.normal(0, scale, shape)).astype(np.float32)).cuda().to(DT[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", [ref.I8, ref.I4, ref.I2])
@pytest.mark.parametrize("E,D,F,T,k", [(4, 64, 64, 1, 2), (1, 1, 1, 1, 1), (3, 5, 3, 2, 3), (2, 130, 77, 3, 1), (8, 512, 96, 5, 4),
                                       (2, 2048, 300, 2, 2), (2, 260, 2050, 3, 1), (2, 4100, 33, 1, 2), (2, 33, 4200, 1, 2)])
def test_moe_sizes(fmt, dtype, E, D, F, T, k):
    rng = np.random.default_rng(E * D + F)
    layer = Layer(rng, fmt, E, D, F)
    ids, w = choose(rng, T, E, k)
    check_moe(layer, rand(rng, (T, D), dtype), ids, w, dtype)
    layer.free()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", [ref.I8, ref.I4, ref.I2])
def test_moe_many_rows_an_expert(fmt, dtype):
    """From one row to more than any operand holds, also with a few left over."""
    rng = np.random.default_rng(17)
    layer = Layer(rng, fmt, 3, 200, 100, O=70)
    for T in (3, 4, 5, 8, 9, 15, 16, 17, 20, 33, 64, 65, 70, 131):
        ids = np.zeros((T, 2), dtype=np.int32)
        ids[:, 1] = np.where(np.arange(T) % 3 == 0, 2, -1)
        check_moe(layer, rand(rng, (T, 200), dtype), ids, rng.uniform(0, 1, (T, 2)).astype(np.float32), dtype)
    layer.free()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("gs", [64, 128, 192, 256, 512])
@pytest.mark.parametrize("fmt", [ref.I8, ref.I4, ref.I2])
def test_moe_group_scales(fmt, gs, dtype):
    rng = np.random.default_rng(gs)
    layer = Layer(rng, fmt, 3, 1001, 525, gs=gs)
    for T, k in ((1, 2), (7, 2), (40, 1)):
        ids, w = choose(rng, T, 3, k)
        check_moe(layer, rand(rng, (T, 1001), dtype), ids, w, dtype)
    layer.free()


def test_moe_ids_outside_and_twice():
    rng = np.random.default_rng(5)
    layer = Layer(rng, ref.I4, 4, 192, 96)
    ids = np.array([[-1, 0, 4, 2], [3, 3, 3, 3], [-(1 << 31), (1 << 31) - 1, -5, 1024], [1, 1, -1, 0], [2, 0, 1, 3]], dtype=np.int32)
    w = rng.normal(0, 1, ids.shape).astype(np.float32)
    w[4, 1] = 0.0
    x, add = rand(rng, (5, 192), "f32"), rand(rng, (5, 192), "f32")
    y = check_moe(layer, x, ids, w, "f32")
    assert (y[2] == 0).all()
    y = check_moe(layer, x, ids, w, "f32", add=add)
    assert torch.equal(y[2], add[2])
    none = np.full((3, 2), -1, dtype=np.int32)
    y = check_moe(layer, x[:3], none, w[:3, :2].copy(), "f32")
    assert (y == 0).all()
    layer.free()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_moe_strides_and_overlaps(dtype):
    rng = np.random.default_rng(6)
    layer = Layer(rng, ref.I4, 4, 131, 96)
    T = 6
    ids, w = choose(rng, T, 4, 2)
    wide = rand(rng, (2 * T, 200), dtype)
    x = wide[::2, 3:134]
    add = rand(rng, (T, 150), dtype)[:, 7:138]
    y = check_moe(layer, x, ids, w, dtype, add=add)
    di, dw = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    same = add.contiguous()
    wq.wq_moe_ffn_dev(layer.moe, x, di, dw, same, add=same)  # y is add
    torch.cuda.synchronize()
    assert torch.equal(same, y)
    own = x.contiguous()
    wq.wq_moe_ffn_dev(layer.moe, own, di, dw, own, add=add.contiguous())  # y is x
    torch.cuda.synchronize()
    assert torch.equal(own, y)
    broadcast = rand(rng, (1, 131), dtype).expand(T, 131)  # one row for all tokens
    check_moe(layer, broadcast, ids, w, dtype)
    layer.free()


def test_moe_bad_rows_stay_their_own():
    """A token with infinities or NaN spoils its own row only, and one whose place is empty spoils none."""
    rng = np.random.default_rng(7)
    layer = Layer(rng, ref.I4, 3, 192, 96)
    for dtype in ("f32", "bf16", "f16"):
        x = rand(rng, (9, 192), dtype)
        ids, w = choose(rng, 9, 3, 2)
        clean = check_moe(layer, x, ids, w, dtype)
        bad = x.clone()
        bad[2, 5], bad[4], bad[7, 0] = float("nan"), float("inf"), float("-inf")
        ids[4] = -1
        y = torch.empty_like(x)
        wq.wq_moe_ffn_dev(layer.moe, bad, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), y)
        torch.cuda.synchronize()
        for t in range(9):
            if t in (2, 7):
                assert not torch.isfinite(y[t]).any()
            elif t == 4:
                assert (y[t] == 0).all()
            else:
                assert torch.equal(y[t], clean[t])
    layer.free()


def test_moe_far_values():
    """Activations over a wide range, tiny ones among huge ones."""
    rng = np.random.default_rng(8)
    layer = Layer(rng, ref.I8, 2, 256, 64, spread=1e-3)
    x = torch.from_numpy((rng.normal(0, 1, (5, 256)) * 10.0 ** rng.uniform(-12, 3, (5, 256))).astype(np.float32)).cuda()
    ids, w = choose(rng, 5, 2, 1)
    check_moe(layer, x, ids, w, "f32")
    zero = torch.zeros((2, 256), device="cuda")
    assert (check_moe(layer, zero, ids[:2], w[:2], "f32") == 0).all()
    layer.free()


def test_moe_largest_number_of_rows():
    rng = np.random.default_rng(9)
    layer = Layer(rng, ref.I4, 40, 64, 32)
    T = wq.WQ_MOE_MAX_ROWS // 8
    ids, w = choose(rng, T, 40, 8)
    check_moe(layer, rand(rng, (T, 64), "bf16"), ids, w, "bf16")
    x = torch.zeros((T + 1, 64), device="cuda")
    with pytest.raises(wq.WqError) as e:
        wq.wq_moe_ffn_dev(layer.moe, x, torch.zeros((T + 1, 8), dtype=torch.int32, device="cuda"), torch.zeros((T + 1, 8), device="cuda"), x)
    assert e.value.code == wq.WQ_E_UNSUPPORTED
    wq.wq_moe_ffn_dev(layer.moe, x[:0], torch.zeros((0, 8), dtype=torch.int32, device="cuda"), torch.zeros((0, 8), device="cuda"), x[:0])
    layer.free()


def test_moe_many_experts():
    rng = np.random.default_rng(10)
    layer = Layer(rng, ref.I8, wq.WQ_MOE_MAX_EXPERTS, 16, 8)
    for T in (3, 200):
        ids, w = choose(rng, T, wq.WQ_MOE_MAX_EXPERTS, 12)
        check_moe(layer, rand(rng, (T, 16), "f32"), ids, w, "f32")
    layer.free()


def test_moe_refusals():
    rng = np.random.default_rng(11)
    a, b = Layer(rng, ref.I4, 2, 64, 32), Layer(rng, ref.I8, 2, 64, 32)
    c, d = Layer(rng, ref.I4, 2, 64, 48), Layer(rng, ref.I4, 2, 64, 32, gs=64)
    g, u, n = a.handles
    f32 = wq.wq_tensor_upload(None, 0, wq.WQ_F32, 32, 64, np.zeros(32 * 64 * 4, dtype=np.uint8), None)
    for sets, code in (((g, b.handles[1], n), wq.WQ_E_INVAL), ((g, u, b.handles[2]), wq.WQ_E_INVAL), ((g, c.handles[1], n), wq.WQ_E_INVAL),
                       ((g, u, c.handles[2]), wq.WQ_E_INVAL), ((g, d.handles[1], n), wq.WQ_E_INVAL), (([g[0], c.handles[0][0]], u, n), wq.WQ_E_INVAL),
                       ((g, u, [n[0], d.handles[2][0]]), wq.WQ_E_INVAL)):
        with pytest.raises(wq.WqError) as e:
            wq.wq_moe_create(*sets)
        assert e.value.code == code
    down = wq.wq_tensor_upload(None, 0, wq.WQ_F32, 64, 32, np.zeros(32 * 64 * 4, dtype=np.uint8), None)
    with pytest.raises(wq.WqError) as e:
        wq.wq_moe_create([f32], [f32], [down])
    assert e.value.code == wq.WQ_E_UNSUPPORTED
    wq.wq_moe_free(wq.wq_moe_create([g[0], g[0]], [u[1], u[1]], [n[0], n[0]]))  # a tensor in several places
    x = torch.zeros((3, 64), device="cuda")
    ids, w = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.zeros((3, 2), device="cuda")
    for args in ((x[:, :63], ids, w, x), (x, ids.long(), w, x), (x, ids, w[:2], x), (x, ids, w.double(), x), (x, ids, w, x[:, :60]),
                 (x, ids, w, x.to(torch.bfloat16)), (x.double(), ids, w, x), (x, ids[:, 0], w, x)):
        with pytest.raises(ValueError):
            wq.wq_moe_ffn_dev(a.moe, *args)
    with pytest.raises(ValueError):
        wq.wq_moe_ffn_dev(a.moe, x, ids, w, x, add=x.to(torch.bfloat16))
    # one tensor of 2^18 + 16 rows as each of 1024 experts: the products' blocks could have 2^32 threads
    F, zeros = (1 << 18) + 16, np.zeros
    wide = [wq.wq_tensor_upload(None, 0, wq.WQ_I2, rows, cols, zeros(rows * cols // 4, dtype=np.uint8), zeros(rows, dtype=np.float32)) for rows, cols in ((F, 16), (16, F))]
    many = wq.wq_moe_create([wide[0]] * 1024, [wide[0]] * 1024, [wide[1]] * 1024)
    y = torch.zeros((1024, 16), device="cuda")
    with pytest.raises(wq.WqError) as e:
        wq.wq_moe_ffn_dev(many, y, torch.zeros((1024, 1), dtype=torch.int32, device="cuda"), torch.zeros((1024, 1), device="cuda"), y)
    assert e.value.code == wq.WQ_E_UNSUPPORTED
    wq.wq_moe_free(many)
    for t in wide:
        wq.wq_tensor_free(t)
    gu.reinit_with_env(WQ_FAULT="launch")
    for call in (lambda: wq.wq_moe_ffn_dev(a.moe, x, ids, w, x), lambda: wq.wq_moe_route_dev(x, ids, w)):
        with pytest.raises(wq.WqError) as e:
            call()
        assert e.value.code == wq.WQ_E_FAULT
    gu.reinit_with_env(WQ_FAULT=None)
    for layer in (a, b, c, d):
        layer.free()
    for t in (f32, down):
        wq.wq_tensor_free(t)


def test_moe_two_streams_and_repeats():
    """Calls on two streams at once do not share a workspace; equal calls give equal bits."""
    rng = np.random.default_rng(12)
    layer = Layer(rng, ref.I4, 8, 1024, 512)
    sets = []
    for T in (9, 33):
        ids, w = choose(rng, T, 8, 3)
        x = rand(rng, (T, 1024), "f32")
        sets.append((x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), check_moe(layer, x, ids, w, "f32")))
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[torch.empty_like(s[0]) for _ in range(8)] for s in sets]
    torch.cuda.synchronize()
    for i in range(8):
        for (x, ids, w, _), st, out in zip(sets, streams, outs):
            wq.wq_moe_ffn_dev(layer.moe, x, ids, w, out[i], stream=st)
    torch.cuda.synchronize()
    for (_, _, _, want), out in zip(sets, outs):
        assert all(torch.equal(o, want) for o in out)
    layer.free()


@pytest.mark.parametrize("T", [1, 3, 40])
def test_route_and_moe_in_a_graph(T):
    """Replays follow the scores and activations of the moment, whichever experts they choose."""
    rng = np.random.default_rng(13)
    E, D, k = 16, 512, 4
    layer = Layer(rng, ref.I4, E, D, 256)
    x, scores = torch.empty((T, D), device="cuda"), torch.empty((T, E), device="cuda")
    ids, w, y = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda"), torch.empty((T, D), device="cuda")
    side = torch.cuda.Stream()

    def step():
        wq.wq_moe_route_dev(scores, ids, w, gating=wq.WQ_GATE_SIGMOID, stream=side)
        wq.wq_moe_ffn_dev(layer.moe, x, ids, w, y, add=x, stream=side)

    x.normal_(), scores.normal_()
    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    for _ in range(5):
        x.normal_(), scores.normal_(), y.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = (ids.clone(), w.clone(), y.clone())
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (ids, w, y)))
    layer.free()


@pytest.mark.parametrize("T,D,k", [(2, 256, 2), (9, 250, 3), (64, 256, 6), (90, 258, 3), (70, 256, 1)])
@pytest.mark.parametrize("fmt,gs", [(ref.I4, 0), (ref.I8, 64), (ref.I2, 0)])
def test_moe_calls_with_nothing_between(T, D, k, fmt, gs):
    """Two layers in turn on one stream leave each other's results, and their own inputs, as they are."""
    rng = np.random.default_rng(15)
    states = []
    for n in range(2):
        layer = Layer(rng, fmt, 70 + 3 * n, D, 100, gs=gs)
        ids, w = choose(rng, T, layer.E, k)
        x, add = rand(rng, (T, D), "f32"), rand(rng, (T, D), "f32")
        states.append((layer, x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), add, add.clone(), check_moe(layer, x, ids, w, "f32", add=add)))
    outs = []
    for n in (0, 1, 0, 0, 1):
        layer, x, ids, w, add, _, _ = states[n]
        outs.append((n, torch.empty_like(x)))
        wq.wq_moe_ffn_dev(layer.moe, x, ids, w, outs[-1][1], add=add)
    torch.cuda.synchronize()
    for n, y in outs:
        assert torch.equal(y, states[n][6]) and torch.equal(states[n][4], states[n][5])
    for s in states:
        s[0].free()


def test_moe_capture_needs_a_workspace():
    rng = np.random.default_rng(14)
    # 4 GiB for the experts' rows alone: more than any stream's workspace, which a captured call could use instead, has grown to
    layer = Layer(rng, ref.I4, 2, 64, 64, O=1 << 16)
    T = wq.WQ_MOE_MAX_ROWS // 2
    x, y = torch.zeros((T, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, 1 << 16), dtype=torch.bfloat16, device="cuda")
    ids, w = torch.zeros((T, 2), dtype=torch.int32, device="cuda"), torch.zeros((T, 2), device="cuda")
    side, codes = torch.cuda.Stream(), []
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        try:
            wq.wq_moe_ffn_dev(layer.moe, x, ids, w, y, stream=side)
        except wq.WqError as e:
            codes.append(e.code)
        torch.zeros(1, device="cuda")
    assert codes == [wq.WQ_E_UNSUPPORTED]
    layer.free()
